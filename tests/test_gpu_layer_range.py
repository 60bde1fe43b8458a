"""GPU tests of the layer operators where a plain bound says little: infinities are
compared as such, a 16-bit result's last place counts below its normal range, and only
what is summed over rows may carry a row's roundings.
"""
import numpy as np
import pytest
import torch

import layer_ref as ref
from tensor_gemm_reduce_amd import layer
from test_gpu_layer import (BF16, F16, F32, GRAD_ROUNDINGS, NORM_ROUNDINGS, W4_WIDTHS, gen, grad_case, norm_case, run_grad,
                            run_norm, w4_case, wgrad_case, wgrad_exact)
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


# ---- block norm -----------------------------------------------------------------------

PER_ROW = ("residual", "y")


def check_grad_rows(got, c, a=0.7, b=-0.9):
    """As check_grad, but only what is summed over rows carries a row's roundings."""
    want = ref.block_norm_backward(c["dz"], c["dh"], c["h"], c["y"], c["rstd"], c["pre"], c["post"], c["gate"], a, b)
    rows = c["y"].shape[0]
    for k, (value, mag) in want.items():
        t = getattr(got, k)
        summed = k not in PER_ROW and (k != "gate" or c["gate"].dim() == 1)
        assert_within(t, value, mag, GRAD_ROUNDINGS + (rows if summed else 0), k)


# Rows wider than a workgroup's registers, with one to three rows per workgroup (256 of them): two and four chunks of
# columns per thread, the last one ragged or whole
@pytest.mark.parametrize("S,N", [(600, 8200), (700, 16384), (600, 20001), (290, 32768)])
@pytest.mark.parametrize("dtype,rdtype,post,gate", [(BF16, F32, True, "channel"), (F16, F16, False, "channel"), (F32, F32, True, "token"),
                                                    (BF16, BF16, True, "full"), (F16, F32, False, "none")])
def test_wide_rows_repeat(S, N, dtype, rdtype, post, gate):
    c = grad_case(S, N, dtype, rdtype, post, gate, seed=S + N)
    got = run_grad(c)
    check_grad_rows(got, c)
    again = run_grad(c)
    for k in got.__slots__:
        t = getattr(got, k)
        assert t is None or torch.equal(t, getattr(again, k)), k


@pytest.mark.parametrize("S,N", [(700, 264), (513, 2050), (1300, 1000), (64, 8192)])
@pytest.mark.parametrize("dtype,rdtype,post,gate", [(F16, F16, True, "full"), (BF16, F32, True, "token"), (F32, F32, False, "channel")])
def test_block_norm_rows_by_themselves(S, N, dtype, rdtype, post, gate):
    c = grad_case(S, N, dtype, rdtype, post, gate, seed=S * N)
    check_grad_rows(run_grad(c), c)


def check_norm_within(out, c, a, b):
    want = ref.block_norm(c["parts"], c["residual"], c["pre"], c["post"], c["gate"], a, b, 1e-5)
    for k in ("y", "h", "z"):
        assert_within(getattr(out, k), *want[k], NORM_ROUNDINGS[k], k)


@pytest.mark.parametrize("N", [100, 2056, 8192, 9000, 20001])
def test_block_norm_results_past_the_largest(N):
    """A sum or a residual past half precision's range is an infinity in y or h, while z comes from the FP32 values."""
    c = norm_case(3, 6, N, F16, F16, False, "none", seed=N)
    c["parts"][:, 1] *= 2.0 ** 15
    c["parts"][:, 4] *= 2.0 ** 13
    c["residual"][2] *= 2.0 ** 14
    out = run_norm(c, a=3.0, b=-2.0, save=True)
    check_norm_within(out, c, 3.0, -2.0)
    # (some inputs are infinities at the larger widths)
    finite = torch.isfinite(c["parts"]).all(2).all(0) & torch.isfinite(c["residual"]).all(1)
    assert torch.isinf(out.y[1]).any() and torch.isinf(out.h[2]).any() and torch.isfinite(out.z[finite]).all()


@pytest.mark.parametrize("N", [100, 2056, 8192, 9000, 20001])
@pytest.mark.parametrize("scale", [2.0 ** 40, 2.0 ** -40])
def test_block_norm_small_and_large_results(N, scale):
    """Values far from one whose squares FP32 still holds."""
    for dtype in (BF16, F32):
        c = norm_case(2, 5, N, dtype, F32, True, "channel", seed=N)
        c["parts"] *= scale
        c["residual"] *= scale
        check_norm_within(run_norm(c, save=True), c, 0.7, -0.9)
    c = norm_case(2, 5, N, F16, F16, False, "full", seed=N)   # results below half precision's normal range
    c["parts"] *= 2.0 ** -13
    c["residual"] *= 2.0 ** -14
    check_norm_within(run_norm(c, save=True), c, 0.7, -0.9)


@pytest.mark.parametrize("N", [72, 2056, 8192, 9000, 20001])
def test_block_norm_rows_whose_squares_overflow(N):
    """Statistics are FP32: a row of values from 2^64 on has a mean square of infinity, so 1 / rms is 0, its norm 0, and
    nothing of another row changes.  h keeps the values."""
    c = norm_case(2, 6, N, BF16, F32, False, "none", seed=N)
    clean = run_norm(c, save=True)
    c["residual"][3] = 2.0 ** 100
    out = run_norm(c, save=True)
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(out.h[keep], clean.h[keep]) and torch.equal(out.z[keep], clean.z[keep])
    assert torch.allclose(out.h[3], torch.full_like(out.h[3], -0.9 * 2.0 ** 100), rtol=2.0 ** -22)
    assert torch.all(out.z[3] == 0) and out.rstd[1, 3] == 0
