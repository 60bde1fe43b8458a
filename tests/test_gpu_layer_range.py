"""GPU tests of the layer operators where a plain bound says little: infinities are
compared as such, a 16-bit result's last place counts below its normal range, and only
what is summed over rows may carry a row's roundings.
"""
import numpy as np
import pytest
import torch

import layer_ref as ref
from tensor_gemm_reduce_amd import layer
from test_gpu_layer import BF16, F16, F32, W4_WIDTHS, gen, w4_case, wgrad_case, wgrad_exact
from test_layer_plan import WGRAD_PLANS

pytestmark = pytest.mark.gpu

HALF_STEP = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}  # of the smallest subnormals


def assert_within(got, want, mag, roundings, what="", step=2.0 ** -150):
    """|got - want| <= half a last place of the output (a subnormal's where it is one) + `roundings` FP32 roundings, each of
    2^-24 of the magnitude and, among FP32's subnormals, of `step`.  Infinities, and what rounds to them, exactly."""
    dtype = got.dtype
    g = got.detach().cpu().to(torch.float64).numpy()
    assert g.shape == want.shape, (what, g.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(g), nan), f"{what}: NaN in other places"
    u = ref.UNIT[dtype]
    with np.errstate(invalid="ignore"):
        bound = u * np.abs(want) + HALF_STEP[dtype] + (1 + u) * roundings * (ref.U32 * mag + step)
        # a result this far past the largest value is an infinity, this far below it none
        top = float(torch.finfo(dtype).max) * (1 + u / 2)
        inf, finite = np.abs(want) - bound > top, np.abs(want) + bound < top
        assert np.array_equal(g[inf], np.copysign(np.inf, want[inf])), f"{what}: infinities"
        assert np.all(np.isfinite(g[finite])), f"{what}: not finite"
        bad = finite & (np.abs(g - want) > bound)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - want) / bound, 0)), bad.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} beyond the bound; at {i} got {g[i]!r}, want {want[i]!r}, "
                             f"bound {bound[i]:.3g}")


# ---- 4-bit weights -----------------------------------------------------------------

W4_RANGE = [(1, 40, 300), (3, 4200, 256), (12, 40, 640), (12, 4200, 300), (30, 100, 256), (30, 4200, 384), (70, 40, 514)] + [
    (1000, N, 300) for N in W4_WIDTHS]


@pytest.mark.parametrize("M,N,K", W4_RANGE)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_largest_bf16_inputs(M, N, K, group, zeros):
    """Inputs of the type's largest value, of one sign in even rows, and scales that bring the results back into range:
    whatever is summed on the way is no reason for an infinity."""
    x, q, s, z = w4_case(M, N, K, group, BF16, zeros, seed=M + N + K + group)
    big = torch.finfo(BF16).max
    x = torch.where(x < 0, -big, big).to(BF16)
    x[::2] = big
    s = s * 2.0 ** -9   # at most 3/2 2^-13, and 15 x 640 inputs are below 2^13.3
    w, terms = ref.w4_weights(q, s, z, group)
    xd = ref.f64(x)
    got = layer.w4_linear(x, layer.w4_pack(q, s, z, group=group))
    assert_within(got, xd @ w.T, np.abs(xd) @ terms.T, 2 * -(-K // 32) + 40, f"{M}x{N}x{K}/{group}")


@pytest.mark.parametrize("M,N,K", W4_RANGE)
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_small_bf16_inputs(M, N, K, zeros):
    """Inputs just above and below the type's normal range, results too.  Results are summed at 2^-12 of their size, where
    FP32's last subnormal place is 2^-149: a rounding there is one of 2^-138."""
    x, q, s, z = w4_case(M, N, K, 64, BF16, zeros, seed=M + N + K)
    x = (x.double() * 2.0 ** -125).to(BF16)
    w, terms = ref.w4_weights(q, s, z, 64)
    xd = ref.f64(x)
    got = layer.w4_linear(x, layer.w4_pack(q, s, z, group=64))
    assert_within(got, xd @ w.T, np.abs(xd) @ terms.T, 2 * -(-K // 32) + 40, f"{M}x{N}x{K}", step=2.0 ** -138)


@pytest.mark.parametrize("M,N,K", W4_RANGE)
def test_w4_results_past_the_largest(M, N, K):
    """Finite results past the output type's range are infinities of their sign."""
    for dtype, scale in ((F16, 2.0 ** 14), (BF16, 2.0 ** 126)):
        x, q, s, z = w4_case(M, N, K, 64, dtype, True, seed=M + N)
        x = (x.double() * scale / 64).clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype)
        w, terms = ref.w4_weights(q, s, z, 64)
        xd = ref.f64(x)
        got = layer.w4_linear(x, layer.w4_pack(q, s, z, group=64))
        assert_within(got, xd @ w.T, np.abs(xd) @ terms.T, 2 * -(-K // 32) + 40, f"{dtype} {M}x{N}x{K}")


def test_w4_rows_do_not_depend_on_the_number_of_rows():
    """Counts of rows that take different kernels agree to their roundings, row by row, with the whole product's."""
    x, q, s, z = w4_case(300, 100, 512, 128, F16, True, seed=5)
    weight = layer.w4_pack(q, s, z, group=128)
    w, terms = ref.w4_weights(q, s, z, 128)
    xd = ref.f64(x)
    whole = layer.w4_linear(x, weight)
    for M in (1, 16, 17, 32, 33, 64, 65, 128, 300):
        got = layer.w4_linear(x[:M], weight)
        assert_within(got, xd[:M] @ w.T, np.abs(xd[:M]) @ terms.T, 2 * 16 + 40, f"M={M}")
        far = (got.double() - whole[:M].double()).abs().cpu().numpy()
        assert np.all(far <= 2 * ref.UNIT[F16] * np.abs(xd[:M] @ w.T) + 2.0 ** -24 + 2 * 72 * ref.U32 * (np.abs(xd[:M]) @ terms.T))


# ---- weight gradient -----------------------------------------------------------------

PLANS = [shape for shape, _ in WGRAD_PLANS]


@pytest.mark.parametrize("M,N,K", PLANS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_wgrad_of_every_plan(M, N, K, dtype):
    """Integers: sums of at most 72 M, multiples of 1/2, below 2^23, so exact in FP32 whatever their order, and the only
    rounding is the output's.  Every way the work is cut, with either output and with and without a running sum."""
    dy, kept = wgrad_case(M, N, K, dtype, seed=M, integer=True)
    add = torch.randint(-50, 50, (N, K), generator=gen(1)).float().cuda()
    sums = dy.double().t().contiguous() @ layer.ckpt_unpack(kept).double()
    for a in (None, add):
        want = sums if a is None else sums + a
        assert torch.equal(layer.ckpt_wgrad(dy, kept, add=a).double(), want)
        assert torch.equal(layer.ckpt_wgrad(dy, kept, add=a, dtype=dtype), want.to(dtype))
    main = add.clone()
    assert torch.equal(layer.ckpt_wgrad(dy, kept, add=main, out=main).double(), sums + add)


@pytest.mark.parametrize("M,N,K", [s for s in PLANS if s[1] * s[2] <= 1 << 21])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_wgrad_of_every_plan_random(M, N, K, dtype):
    dy, kept = wgrad_case(M, N, K, dtype, seed=N)
    for out in (F32, dtype):
        assert_within(layer.ckpt_wgrad(dy, kept, dtype=out), *wgrad_exact(dy, kept), -(-M // 16) + 40, f"{out}")
