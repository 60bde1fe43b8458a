"""GPU tests of the layer operators against plain 64-bit implementations
(layer_ref.py): shapes from one row or column up, odd widths, strides, types,
special values, gradients against differences, refusals, streams, graphs and
offsets past 32 bits.

Tolerances: one rounding to the output's type, plus the FP32 roundings on the
longest path from an input to an output times the terms' magnitudes.  An MFMA
of 16 or 32 terms counts as one step of its accumulator; 40 cover what happens
inside and after it.  A row's sum of squares is a chain of at most 54 additions
(32 in a thread, 6 in a wave, 16 over the waves).
"""
import numpy as np
import pytest
import torch

import layer_ref as ref
from tensor_gemm_reduce_amd import layer

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NORM_ROUNDINGS = {"y": 8, "h": 128, "z": 384}
GRAD_ROUNDINGS = 384


def randn(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(dtype).cuda()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def strided(t, pad, offset=0, fill=float("nan")):
    """The same rows inside a wider buffer, `offset` elements in, `fill` around them."""
    S, N = t.shape
    buf = torch.full((S, N + pad), fill, dtype=t.dtype, device=t.device)
    view = buf[:, offset:offset + N]
    view.copy_(t)
    return view


# ---- 4-bit weights -----------------------------------------------------------------

def w4_case(M, N, K, group, dtype, zeros, seed=0, integer=False):
    g = gen(seed)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    G = -(-K // group)
    if integer:
        x = torch.randint(-2, 3, (M, K), generator=g).to(dtype)
        s = torch.exp2(torch.randint(-1, 2, (N, G), generator=g).float()).to(dtype)
    else:
        x = torch.randn((M, K), generator=g).to(dtype)
        s = (torch.rand((N, G), generator=g) + 0.5).to(dtype) / 16
    z = torch.randint(0, 16, (N, G), generator=g, dtype=torch.uint8) if zeros else None
    return x.cuda(), q.cuda(), s.cuda(), None if z is None else z.cuda()


def check_w4(y, x, q, s, z, group, what):
    w, terms = ref.w4_weights(q, s, z, group)
    xd = ref.f64(x)
    K = x.shape[1]
    ref.assert_close(y, xd @ w.T, np.abs(xd) @ terms.T, 2 * -(-K // 32) + 40, what)


W4_SHAPES = [  # M, N, K, group
    (1, 1, 2, 32), (1, 16, 128, 128), (1, 17, 130, 32), (2, 33, 62, 62), (3, 100, 1000, 1000), (16, 64, 256, 64),
    (17, 250, 384, 32), (31, 128, 1024, 128), (33, 48, 2050, 96), (64, 1024, 128, 128), (65, 72, 320, 64),
    (129, 257, 514, 256), (300, 96, 2048, 128), (1, 8192, 1024, 128), (5, 4096, 3584, 64),
]


@pytest.mark.parametrize("M,N,K,group", W4_SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_linear(M, N, K, group, dtype, zeros):
    x, q, s, z = w4_case(M, N, K, group, dtype, zeros, seed=M + N + K)
    weight = layer.w4_pack(q, s, z, group=group)
    check_w4(layer.w4_linear(x, weight), x, q, s, z, group, f"{M}x{N}x{K}/{group}")


@pytest.mark.parametrize("M,N,K,group", [(1, 40, 256, 32), (20, 300, 512, 64), (70, 130, 640, 128), (200, 64, 256, 32)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_w4_integers_are_exact(M, N, K, group, dtype):
    """Every sum is an integer multiple of 1/2 far below 2^24, so the only rounding is the output's."""
    x, q, s, z = w4_case(M, N, K, group, dtype, True, seed=7, integer=True)
    w, _ = ref.w4_weights(q, s, z, group)
    want = torch.from_numpy(ref.f64(x) @ w.T).to(dtype)
    got = layer.w4_linear(x, layer.w4_pack(q, s, z, group=group)).cpu()
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [1, 16, 48, 150])
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (3, 1), (1, 1)])
def test_w4_strides_and_alignment(M, pad, offset):
    x, q, s, z = w4_case(M, 80, 384, 128, BF16, True, seed=3)
    weight = layer.w4_pack(q, s, z, group=128)
    want = layer.w4_linear(x, weight)
    out = strided(torch.zeros((M, 80), dtype=BF16, device="cuda"), pad, offset, fill=7.0)
    got = layer.w4_linear(strided(x, pad, offset), weight, out)   # NaN around the rows must not be read into them
    assert torch.equal(got, want) and got.data_ptr() == out.data_ptr()
    assert torch.all(out._base[:, :offset] == 7.0) and torch.all(out._base[:, offset + 80:] == 7.0)


def test_w4_special_values_stay_in_their_row():
    x, q, s, z = w4_case(9, 64, 256, 64, BF16, False, seed=4)
    weight = layer.w4_pack(q, s, group=64)
    clean = layer.w4_linear(x, weight)
    x[2, 5] = float("nan")
    x[7, 255] = float("inf")
    got = layer.w4_linear(x, weight)
    keep = [0, 1, 3, 4, 5, 6, 8]
    assert torch.equal(got[keep], clean[keep])
    assert torch.all(torch.isnan(got[[2, 7]]))


def test_w4_no_rows_and_rows_split_alike():
    x, q, s, z = w4_case(300, 100, 512, 128, F16, True, seed=5)
    weight = layer.w4_pack(q, s, z, group=128)
    assert layer.w4_linear(x[:0], weight).shape == (0, 100)
    for M in (1, 16, 17, 32, 33, 64, 65, 128, 300):
        check_w4(layer.w4_linear(x[:M], weight), x[:M], q, s, z, 128, f"M={M}")


# Widths that put 1000 rows through each shape of workgroup: 16 and 32 columns, then 64, 128, 192 and 256 with the rows
# in LDS; and few rows of weights with more tiles than compute units.
W4_WIDTHS = [250, 500, 700, 1590, 2390, 3190]


@pytest.mark.parametrize("N", W4_WIDTHS)
@pytest.mark.parametrize("K,group", [(2, 32), (200, 64), (384, 128), (514, 32), (1154, 64), (1408, 128)])
@pytest.mark.parametrize("dtype,zeros", [(BF16, False), (BF16, True), (F16, False), (F16, True)])
def test_w4_linear_many_rows(N, K, group, dtype, zeros):
    x, q, s, z = w4_case(1000, N, K, group, dtype, zeros, seed=N + K)
    weight = layer.w4_pack(q, s, z, group=group)
    check_w4(layer.w4_linear(x, weight), x, q, s, z, group, f"{N}x{K}/{group}")


@pytest.mark.parametrize("M", [1, 3, 4, 12, 30])
@pytest.mark.parametrize("K,group", [(514, 32), (400, 64), (1152, 128)])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_linear_wide_weights(M, K, group, zeros):
    x, q, s, z = w4_case(M, 4200, K, group, F16, zeros, seed=M + K)
    check_w4(layer.w4_linear(x, layer.w4_pack(q, s, z, group=group)), x, q, s, z, group, f"{M} rows")


@pytest.mark.parametrize("N", W4_WIDTHS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_integers_are_exact_many_rows(N, dtype, group):
    """As above: multiples of 1/2, the sums of inputs for the zero points among them."""
    x, q, s, z = w4_case(1000, N, 640, group, dtype, True, seed=11, integer=True)
    w, _ = ref.w4_weights(q, s, z, group)
    got = layer.w4_linear(x, layer.w4_pack(q, s, z, group=group)).cpu()
    assert torch.equal(got, torch.from_numpy(ref.f64(x) @ w.T).to(dtype))


@pytest.mark.parametrize("M,N", [(1, 40), (20, 40), (70, 40)] + [(1000, N) for N in W4_WIDTHS])
def test_w4_subnormal_inputs(M, N):
    """Inputs of a few times 2^-24, below half precision's normal range, times scales of 2^9 .. 2^11: exact in FP32."""
    x, q, s, z = w4_case(M, N, 256, 64, F16, True, seed=13, integer=True)
    x, s = x * 2.0**-24, s * 2.0**10
    w, _ = ref.w4_weights(q, s, z, 64)
    got = layer.w4_linear(x, layer.w4_pack(q, s, z, group=64)).cpu()
    assert torch.equal(got, torch.from_numpy(ref.f64(x) @ w.T).to(F16))


@pytest.mark.parametrize("M,N", [(1, 40), (20, 40), (70, 40), (1000, 700), (1000, 3190)])
def test_w4_subnormal_inputs_bf16(M, N):
    """The same in BF16, inputs of a few times 2^-133 and scales that bring the results back."""
    x, q, s, z = w4_case(M, N, 256, 64, BF16, True, seed=13, integer=True)
    x, s = (x.double() * 2.0**-133).to(BF16), (s.double() * 2.0**40).to(BF16)
    w, _ = ref.w4_weights(q, s, z, 64)
    got = layer.w4_linear(x, layer.w4_pack(q, s, z, group=64)).cpu()
    assert torch.equal(got, torch.from_numpy(ref.f64(x) @ w.T).to(BF16))


@pytest.mark.parametrize("N", W4_WIDTHS)
@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 1)])
def test_w4_many_rows_strides_and_special_values(N, pad, offset):
    x, q, s, z = w4_case(1000, N, 386, 128, BF16, True, seed=3)
    weight = layer.w4_pack(q, s, z, group=128)
    want = layer.w4_linear(x, weight)
    out = strided(torch.zeros((1000, N), dtype=BF16, device="cuda"), pad, offset, fill=7.0)
    assert torch.equal(layer.w4_linear(strided(x, pad, offset), weight, out), want)
    assert torch.all(out._base[:, :offset] == 7.0) and torch.all(out._base[:, offset + N:] == 7.0)
    x[2, 5], x[700, 385], x[999, 0] = float("nan"), float("inf"), float("nan")
    got = layer.w4_linear(x, weight)
    bad = torch.zeros(1000, dtype=torch.bool, device="cuda")
    bad[[2, 700, 999]] = True
    assert torch.equal(got[~bad], want[~bad]) and torch.all(torch.isnan(got[bad]))


# ---- block norm -----------------------------------------------------------------------

def gate_shape(kind, S, N):
    return {"none": None, "channel": (N,), "token": (S, 1), "full": (S, N)}[kind]


def norm_case(P, S, N, dtype, rdtype, post, gate, pre=True, seed=0, residual=True):
    g = gen(seed)
    return dict(parts=randn(g, (P, S, N), dtype, 0.5), residual=randn(g, (S, N), rdtype) if residual else None,
                pre=1 + randn(g, (N,), dtype, 0.2) if pre else None, post=1 + randn(g, (N,), dtype, 0.2) if post else None,
                gate=randn(g, gate_shape(gate, S, N), dtype) if gate != "none" else None)


def run_norm(c, a=0.7, b=-0.9, eps=1e-5, **kw):
    return layer.block_norm(c["parts"], c["residual"], pre_weight=c["pre"], post_weight=c["post"], gate=c["gate"],
                            block_scale=a, residual_scale=b, eps=eps, **kw)


def check_norm(out, c, a=0.7, b=-0.9, eps=1e-5, what=""):
    want = ref.block_norm(c["parts"], c["residual"], c["pre"], c["post"], c["gate"], a, b, eps)
    for k in ("y", "h", "z"):
        got = getattr(out, k)
        assert (got is None) == (k not in want or (k == "y" and out.rstd is None)), k
        if got is not None:
            ref.assert_close(got, *want[k], NORM_ROUNDINGS[k], f"{what} {k}")
    if out.rstd is not None:
        np.testing.assert_allclose(out.rstd.cpu().numpy(), want["rstd"], rtol=256 * ref.U32)


@pytest.mark.parametrize("S,N", [(1, 1), (3, 7), (2, 8), (5, 9), (4, 100), (3, 1000), (2, 2048), (7, 2056), (2, 4095),
                                 (3, 4104), (1, 8192), (2, 8200), (2, 16384), (1, 20001), (1, 32768)])
@pytest.mark.parametrize("dtype,rdtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
def test_block_norm_shapes_and_types(S, N, dtype, rdtype):
    P, post, gate = [(1, True, "channel"), (8, False, "none"), (3, True, "full"), (2, True, "token")][(S + N) % 4]
    c = norm_case(P, S, N, dtype, rdtype, post, gate, seed=S * N)
    check_norm(run_norm(c, save=True), c)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_block_norm_forms(post, gate, pre, residual):
    for P in (1, 5, 8):
        c = norm_case(P, 6, 520, BF16, F32, post, gate, pre, seed=P, residual=residual)
        check_norm(run_norm(c), c)


def test_block_norm_sums_the_parts_in_order():
    """The sum of the partials is the slice sum of the fused layer: FP32, in order, one rounding."""
    g = gen(11)
    parts = [randn(g, (9, 264), BF16, 10.0 ** (i % 3)) for i in range(8)]
    s = torch.zeros((9, 264), dtype=F32, device="cuda")
    for p in parts:
        s = s + p.float()
    out = layer.block_norm(parts, save=True)
    assert torch.equal(out.h, s.to(BF16)) and torch.equal(out.y, s.to(BF16)) and out.z is None


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 1)])
def test_block_norm_strides_in_place_and_lists(pad, offset):
    c = norm_case(3, 10, 300, BF16, BF16, True, "full", seed=2)
    want = run_norm(c, save=True)
    parts = [strided(p, pad, offset) for p in c["parts"]]
    resid = strided(c["residual"], pad, offset, fill=7.0)
    z = strided(torch.zeros_like(c["residual"]), pad, offset, fill=7.0)
    out = layer.block_norm(parts, resid, pre_weight=c["pre"], post_weight=c["post"], gate=strided(c["gate"], pad, offset),
                           block_scale=0.7, residual_scale=-0.9, h=resid, z=z)
    assert out.h is resid and torch.equal(resid, want.h) and torch.equal(z, want.z)
    for t in (resid, z):
        assert torch.all(t._base[:, :offset] == 7.0) and torch.all(t._base[:, offset + 300:] == 7.0)


def test_block_norm_special_rows():
    """A row of zeros, an infinity, a NaN and huge values change no other row; eps = 0 gives what the formula gives."""
    c = norm_case(1, 6, 640, F32, F32, True, "none", seed=9)
    clean = run_norm(c)
    c["parts"][0, 1] = 0
    c["residual"][1] = 0
    c["parts"][0, 3, 17] = float("inf")
    c["residual"][5, 600] = float("nan")
    out = run_norm(c)
    assert torch.equal(out.z[[0, 2, 4]], clean.z[[0, 2, 4]])
    assert torch.all(out.h[1] == 0) and torch.all(out.z[1] == 0)
    check_norm(out, c)
    check_norm(run_norm(c, eps=0.0), c, eps=0.0)


def test_block_norm_no_rows():
    e = torch.empty((0, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, dtype=BF16, device="cuda")
    assert layer.block_norm(e, e, pre_weight=w).z.shape == (0, 64)
    g = layer.block_norm_backward(e, e, e, e, torch.empty((2, 0), device="cuda"), pre_weight=w, post_weight=w, gate=w)
    for t in (g.pre_weight, g.post_weight, g.gate):
        assert torch.equal(t, torch.zeros(64, device="cuda"))
    assert g.y.shape == (0, 64)


def grad_case(S, N, dtype, rdtype, post, gate, seed=0, pre=True, dh=True):
    g = gen(seed)
    c = norm_case(1, S, N, dtype, rdtype, post, gate, pre, seed)
    c["y"] = c["parts"][0]
    c["h"] = randn(g, (S, N), rdtype, 1.3)
    c["rstd"] = torch.stack([torch.rsqrt(t.double().square().mean(1) + 1e-5).float() for t in (c["y"], c["h"])])
    c["dz"] = randn(g, (S, N), dtype, 0.3) if pre else None
    c["dh"] = randn(g, (S, N), rdtype, 0.3) if dh else None
    return c


def run_grad(c, a=0.7, b=-0.9, **kw):
    return layer.block_norm_backward(c["dz"], c["dh"], c["h"], c["y"], c["rstd"], pre_weight=c["pre"], post_weight=c["post"],
                                     gate=c["gate"], block_scale=a, residual_scale=b, **kw)


def check_grad(got, c, a=0.7, b=-0.9):
    want = ref.block_norm_backward(c["dz"], c["dh"], c["h"], c["y"], c["rstd"], c["pre"], c["post"], c["gate"], a, b)
    rows = c["y"].shape[0]
    for k in ("residual", "y", "pre_weight", "post_weight", "gate"):
        t = getattr(got, k)
        assert (t is None) == (k not in want), k
        if t is not None:
            ref.assert_close(t, *want[k], GRAD_ROUNDINGS + rows, k)


@pytest.mark.parametrize("S,N", [(1, 1), (3, 7), (2, 8), (5, 9), (130, 100), (3, 1000), (2, 2048), (700, 264), (2, 4095),
                                 (3, 4104), (1, 8192), (600, 8192), (2, 8200), (3, 16384), (600, 8320), (1, 32768)])
@pytest.mark.parametrize("dtype,rdtype", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
def test_block_norm_backward_shapes_and_types(S, N, dtype, rdtype):
    post, gate = [(True, "channel"), (False, "none"), (True, "full"), (True, "token"), (False, "channel")][(S + N) % 5]
    c = grad_case(S, N, dtype, rdtype, post, gate, seed=S + N)
    check_grad(run_grad(c), c)


# Rows and widths of every count of threads; one, two and more rows per workgroup; partial rows of one batch and more.
@pytest.mark.parametrize("S,N", [(257, 520), (511, 1025), (513, 2050), (300, 2504), (300, 4100), (1300, 5000), (5, 6144),
                                 (2100, 1000)])
@pytest.mark.parametrize("dtype,rdtype,post,gate", [(BF16, F32, True, "channel"), (F16, F16, False, "token"),
                                                    (F32, F32, True, "none")])
def test_block_norm_rows_and_widths(S, N, dtype, rdtype, post, gate):
    c = grad_case(S, N, dtype, rdtype, post, gate, seed=S + N)
    check_norm(run_norm(c, save=True), c)
    got = run_grad(c)
    check_grad(got, c)
    again = run_grad(c)
    assert torch.equal(got.pre_weight, again.pre_weight)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("dh", [False, True])
def test_block_norm_backward_forms(post, gate, pre, dh):
    c = grad_case(20, 520, BF16, F32, post, gate, seed=3, pre=pre, dh=dh)
    if not pre:
        c["h"] = torch.empty((20, 520), device="cuda")
    check_grad(run_grad(c), c)


@pytest.mark.parametrize("post,gate", [(True, "channel"), (True, "token"), (False, "full"), (False, "none")])
def test_block_norm_backward_against_differences(post, gate):
    """The derivative of L = <z, dz> + <h, dh> along random directions, from central differences of the 64-bit forward
    pass.  Their error: (1e-4)^2 times third derivatives of order one, and 2^-52 / 1e-4 of cancellation."""
    S, N = 5, 72
    c = norm_case(1, S, N, F32, F32, post, gate, seed=6)
    g = gen(8)
    dz, dh = randn(g, (S, N), F32), randn(g, (S, N), F32)
    out = run_norm(c, save=True)
    grads = layer.block_norm_backward(dz, dh, out.h, out.y, out.rstd, pre_weight=c["pre"], post_weight=c["post"],
                                      gate=c["gate"], block_scale=0.7, residual_scale=-0.9)
    names = {"parts": "y", "residual": "residual", "pre": "pre_weight", "post": "post_weight", "gate": "gate"}
    for name, field in names.items():
        if c[name] is None:
            continue
        d = torch.randn(c[name].shape, generator=g, dtype=torch.float64)
        vals = []
        for step in (1e-4, -1e-4):
            moved = {k: None if v is None else v.double().cpu() for k, v in c.items()}
            moved[name] = moved[name] + step * d
            w = ref.block_norm(moved["parts"], moved["residual"], moved["pre"], moved["post"], moved["gate"], 0.7, -0.9, 1e-5)
            vals.append((w["z"][0] * ref.f64(dz)).sum() + (w["h"][0] * ref.f64(dh)).sum())
        diff = (vals[0] - vals[1]) / 2e-4
        got = (ref.f64(getattr(grads, field)).reshape(d.shape) * d.numpy()).sum()
        size = np.abs(ref.f64(getattr(grads, field)).reshape(d.shape) * d.numpy()).sum()
        assert abs(got - diff) <= 1e-5 * max(size, 1.0), (name, got, diff)


def test_block_norm_backward_strides_and_repeats():
    c = grad_case(700, 1000, BF16, F32, True, "channel", seed=12)
    want = run_grad(c)
    for _ in range(3):
        again = run_grad(c)
        for k in ("residual", "y", "pre_weight", "post_weight", "gate"):
            assert torch.equal(getattr(want, k), getattr(again, k)), k
    s = dict(c, **{k: strided(c[k], 5, 3) for k in ("dz", "dh", "h", "y")})
    got = run_grad(s)
    for k in ("residual", "y", "pre_weight", "post_weight", "gate"):
        assert torch.equal(getattr(want, k), getattr(got, k)), k


def test_block_norm_backward_nan_row_spoils_only_its_own():
    c = grad_case(8, 264, F32, F32, True, "token", seed=13)
    clean = run_grad(c)
    c["dz"][3, 100] = float("nan")
    got = run_grad(c)
    keep = [0, 1, 2, 4, 5, 6, 7]
    for k in ("residual", "y", "gate"):
        assert torch.equal(getattr(got, k)[keep], getattr(clean, k)[keep]), k
        assert torch.all(torch.isnan(getattr(got, k)[3])), k
    assert torch.isnan(got.pre_weight[100]) and torch.isnan(got.pre_weight).sum() == 1


# ---- 8-bit checkpoints -------------------------------------------------------------------

def check_ckpt(x):
    kept = layer.ckpt_pack(x)
    q, e = ref.ckpt_pack(x)
    assert np.array_equal(kept.exps.cpu().numpy(), e)
    assert np.array_equal(kept.q.cpu().numpy(), q)
    back = layer.ckpt_unpack(kept)
    assert back.dtype == x.dtype
    np.testing.assert_array_equal(ref.f64(back), ref.ckpt_value(q, e, x.shape[1]))
    return kept


@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (1, 31), (2, 32), (5, 33), (130, 100), (4, 1000), (64, 3584), (1000, 40)])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_ckpt_is_exact(M, K, dtype):
    g = gen(M + K)
    check_ckpt((torch.randn((M, K), generator=g) * torch.exp(torch.randn((M, K), generator=g))).to(dtype).cuda())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_ckpt_extremes(dtype):
    """Every power of two the type holds as a block's maximum, ties, subnormals, the largest values, zeros."""
    info = torch.finfo(dtype)
    low, high = int(np.log2(info.tiny)) - 30, int(np.floor(np.log2(info.max)))
    p = torch.arange(max(low, -149), high + 1)
    f = torch.tensor([1.0, 127 / 128, 0.5 + 1 / 256, 63.5 / 64, 1 / 128, 3 / 128, 1 / 64, 5 / 128] * 4)
    x = (torch.ldexp(torch.ones(len(p), 1, dtype=torch.float64), p[:, None]) * f.double() * 1.99).to(dtype)
    x = torch.where(torch.isfinite(x), x, torch.full_like(x, info.max))
    x[:, 1::2] *= -1
    check_ckpt(x.cuda())
    y = torch.zeros((6, 64), dtype=dtype)
    y[0, :32] = -0.0
    y[1, 40] = info.max
    y[2, 3] = -info.max
    y[3, 5] = info.tiny
    y[4] = info.max
    check_ckpt(y.cuda())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_ckpt_marks_blocks_that_are_not_finite(dtype):
    g = gen(1)
    x = torch.randn((4, 96), generator=g).to(dtype).cuda()
    x[0, 33] = float("inf")
    x[1, 0] = float("nan")
    x[3, 95] = float("-inf")
    kept = check_ckpt(x)
    assert (kept.exps == layer.CKPT_NAN).sum() == 3
    back = layer.ckpt_unpack(kept)
    assert torch.isnan(back).sum() == 96 and torch.all(torch.isnan(back[0, 32:64]))


@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 1), (5, 2)])
def test_ckpt_strides(pad, offset):
    g = gen(2)
    x = torch.randn((37, 200), generator=g).to(BF16).cuda()
    want = layer.ckpt_pack(x)
    kept = layer.ckpt_pack(strided(x, pad, offset))
    assert torch.equal(kept.q, want.q) and torch.equal(kept.exps, want.exps)
    out = strided(torch.zeros_like(x), pad, offset, fill=7.0)
    assert torch.equal(layer.ckpt_unpack(kept, out), layer.ckpt_unpack(want))
    assert torch.all(out._base[:, :offset] == 7.0) and torch.all(out._base[:, offset + 200:] == 7.0)


def wgrad_case(M, N, K, dtype, seed=0, integer=False):
    g = gen(seed)
    blocks = -(-K // 32)
    if integer:
        dy = torch.randint(-2, 3, (M, N), generator=g).to(dtype)
        q = torch.randint(-9, 10, (M, blocks * 32), generator=g, dtype=torch.int8)
        e = torch.randint(-1, 3, (M, blocks), generator=g, dtype=torch.int8)
    else:
        dy = torch.randn((M, N), generator=g).to(dtype)
        q = torch.randint(-127, 128, (M, blocks * 32), generator=g, dtype=torch.int8)
        e = torch.randint(-9, -4, (M, blocks), generator=g, dtype=torch.int8)
    q[:, K:] = 0
    return dy.cuda(), layer.Checkpoint(q.cuda(), e.cuda(), K, dtype)


def wgrad_exact(dy, kept, add=None):
    v = torch.from_numpy(ref.ckpt_value(kept.q.cpu().numpy(), kept.exps.cpu().numpy(), kept.K))
    d = dy.double().cpu().t()
    w, m = (d @ v).numpy(), (d.abs() @ v.abs()).numpy()
    if add is not None:
        w, m = w + ref.f64(add), m + np.abs(ref.f64(add))
    return w, m


WGRAD_SHAPES = [(1, 1, 1), (1, 8, 32), (2, 33, 31), (31, 128, 128), (32, 129, 130), (33, 100, 1000), (64, 256, 256),
                (65, 264, 72), (257, 520, 264), (512, 1024, 128), (1000, 300, 200), (4100, 136, 96), (128, 1000, 1037),
                (300, 776, 520), (2570, 1030, 1000)]


@pytest.mark.parametrize("M,N,K", WGRAD_SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_wgrad(M, N, K, dtype):
    dy, kept = wgrad_case(M, N, K, dtype, seed=M + N)
    add = randn(gen(3), (N, K), F32)
    for out_dtype, a in ((F32, None), (F32, add), (dtype, None), (dtype, add)):
        got = layer.ckpt_wgrad(dy, kept, add=a, dtype=out_dtype)
        ref.assert_close(got, *wgrad_exact(dy, kept, a), -(-M // 16) + 40, f"{out_dtype} add={a is not None}")


@pytest.mark.parametrize("M,N,K", [(40, 130, 70), (512, 1024, 256), (2048, 512, 520), (777, 264, 1000),
                                   # tiles of 256 x 256: 16 tiles in shares, an odd number of steps, ragged in every
                                   # direction; one whole round and a rest; a rest too short to cut
                                   (2624, 1024, 1024), (2570, 1030, 1000), (2560, 4104, 4130), (2700, 4096, 4096)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_wgrad_integers_are_exact(M, N, K, dtype):
    """Every sum is a multiple of 1/2 below 2^23, so FP32 holds it exactly whatever the order."""
    dy, kept = wgrad_case(M, N, K, dtype, seed=5, integer=True)
    add = torch.randint(-50, 50, (N, K), generator=gen(1)).float().cuda()
    want, _ = wgrad_exact(dy, kept, add)
    assert torch.equal(layer.ckpt_wgrad(dy, kept, add=add).double().cpu(), torch.from_numpy(want))


# Tiles of 128 x 128 in many pieces; tiles of 256 x 256 all cut, one whole round and a rest in few pieces, and two
# whole rounds but for a rest too short to cut
LONG_WGRADS = [(4100, 300, 200), (16390, 100, 60), (12300, 1030, 1000), (2840, 4104, 4130), (2850, 8190, 4090)]


@pytest.mark.parametrize("M,N,K", LONG_WGRADS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_wgrad_integers_are_exact_long(M, N, K, dtype):
    """Sums of at most 72 M, multiples of 1/2: below 2^23, so exact in FP32."""
    dy, kept = wgrad_case(M, N, K, dtype, seed=6, integer=True)
    add = torch.randint(-50, 50, (N, K), generator=gen(1)).float().cuda()
    v = layer.ckpt_unpack(kept).double()
    want = dy.double().t().contiguous() @ v + add
    assert torch.equal(layer.ckpt_wgrad(dy, kept, add=add).double(), want)


@pytest.mark.parametrize("M,N,K", LONG_WGRADS[:3])
def test_wgrad_long_random_and_special_values(M, N, K):
    dy, kept = wgrad_case(M, N, K, BF16, seed=8)
    clean = layer.ckpt_wgrad(dy, kept, dtype=F32)
    ref.assert_close(clean, *wgrad_exact(dy, kept), -(-M // 16) + 40, "f32")
    assert torch.equal(clean, layer.ckpt_wgrad(dy, kept, dtype=F32))
    kept.exps[M - 3, 1] = layer.CKPT_NAN
    dy[M // 2, 7] = float("nan")
    got = layer.ckpt_wgrad(dy, kept, dtype=F32)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[:, 32:64] = True
    bad[7] = True
    assert torch.all(torch.isnan(got[bad])) and torch.equal(got[~bad], clean[~bad])


def test_wgrad_in_place_strides_and_no_rows():
    dy, kept = wgrad_case(100, 136, 72, BF16, seed=6)
    add = randn(gen(4), (136, 72), F32)
    want = layer.ckpt_wgrad(dy, kept, add=add)
    main = add.clone()
    assert layer.ckpt_wgrad(dy, kept, add=main, out=main) is main and torch.equal(main, want)
    for pad, offset in ((8, 8), (4, 0), (3, 1)):
        out = strided(torch.zeros_like(add), pad, offset, fill=7.0)
        got = layer.ckpt_wgrad(strided(dy, pad, offset), kept, add=strided(add, pad, offset), out=out)
        assert torch.equal(got, want), (pad, offset)
        assert torch.all(out._base[:, :offset] == 7.0) and torch.all(out._base[:, offset + 72:] == 7.0)
    none = layer.Checkpoint(kept.q[:0], kept.exps[:0], 72, BF16)
    assert torch.equal(layer.ckpt_wgrad(dy[:0], none, add=add), add)
    assert torch.equal(layer.ckpt_wgrad(dy[:0], none), torch.zeros_like(add))


@pytest.mark.parametrize("M,N,K", [(70, 140, 200), (2600, 1000, 1000)])
def test_wgrad_special_values(M, N, K):
    """A NaN block reaches its 32 columns of every row, a NaN in dy its row of dw; nothing else changes."""
    dy, kept = wgrad_case(M, N, K, BF16, seed=8)
    clean = layer.ckpt_wgrad(dy, kept)
    kept.exps[13, 2] = layer.CKPT_NAN
    dy[50, 7] = float("nan")
    got = layer.ckpt_wgrad(dy, kept)
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[:, 64:96] = True
    bad[7] = True
    assert torch.all(torch.isnan(got[bad])) and torch.equal(got[~bad], clean[~bad])


def test_wgrad_is_the_gradient_of_the_layer():
    """L(w) = <dy, x^ w^T> is linear in w, so its difference along any direction is <dw, direction> exactly."""
    M, N, K = 60, 40, 50
    g = gen(9)
    x = torch.randn((M, K), generator=g).to(BF16).cuda()
    kept = layer.ckpt_pack(x)
    dy = randn(g, (M, N), BF16)
    dw = ref.f64(layer.ckpt_wgrad(dy, kept))
    v = ref.f64(layer.ckpt_unpack(kept))
    d = np.random.default_rng(1).standard_normal((N, K))
    size = np.abs(dw * d).sum()
    assert abs((ref.f64(dy) * (v @ d.T)).sum() - (dw * d).sum()) <= 64 * ref.U32 * M * size
    # and the checkpoint itself is within half a step (a whole one at the limit) of the activation
    step = np.exp2(kept.exps.cpu().numpy().astype(np.float64)).repeat(32, 1)[:, :K]
    assert np.all(np.abs(v - ref.f64(x)) <= step)


# ---- all of them ---------------------------------------------------------------------------

def all_ops():
    """name -> (call, outputs of a plain run)"""
    x, q, s, z = w4_case(20, 200, 512, 128, BF16, True, seed=1)
    weight = layer.w4_pack(q, s, z, group=128)
    n = norm_case(8, 40, 1000, BF16, F32, True, "channel", seed=1)
    gr_ = grad_case(600, 1000, BF16, F32, True, "channel", seed=2)
    act = randn(gen(5), (300, 200), BF16)
    kept = layer.ckpt_pack(act)
    dy = randn(gen(6), (300, 264), BF16)
    big = wgrad_case(2048, 512, 512, BF16, seed=3)
    tup = lambda o: tuple(getattr(o, k) for k in o.__slots__ if isinstance(getattr(o, k), torch.Tensor))  # noqa: E731
    return {
        "w4_pack": lambda **kw: (layer.w4_pack(q, s, z, group=128, **kw).packed,),
        "w4_linear": lambda **kw: (layer.w4_linear(x, weight, **kw),),
        "block_norm": lambda **kw: tup(run_norm(n, save=True, **kw)),
        "block_norm_backward": lambda **kw: tup(run_grad(gr_, **kw)),
        "ckpt_pack": lambda **kw: tup(layer.ckpt_pack(act, **kw)),
        "ckpt_unpack": lambda **kw: (layer.ckpt_unpack(kept, **kw),),
        "ckpt_wgrad": lambda **kw: (layer.ckpt_wgrad(dy, kept, **kw),),
        "ckpt_wgrad long": lambda **kw: (layer.ckpt_wgrad(*big, **kw),),
    }


@pytest.mark.parametrize("name", ["w4_pack", "w4_linear", "block_norm", "block_norm_backward", "ckpt_pack", "ckpt_unpack",
                                  "ckpt_wgrad", "ckpt_wgrad long"])
def test_streams_and_graphs(name):
    call = all_ops()[name]
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = call(stream=stream)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        captured = call()
    for _ in range(3):
        for t in captured:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
        assert all(torch.equal(a, b) for a, b in zip(call(), want))   # eager work between replays
        torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Three rows 2^30 + 8 elements apart: the last one starts past 4 GiB (and past 2^31 elements)."""
    S, N, far = 3, 96, (1 << 30) + 8
    buf = torch.zeros(2 * far + N, dtype=BF16, device="cuda")
    wide = buf.as_strided((S, N), (far, 1))
    t = randn(gen(1), (S, N), BF16)

    def put(v):
        wide.copy_(v)
        return wide

    w = torch.ones(N, dtype=BF16, device="cuda")
    near = layer.block_norm(t, t, pre_weight=w, post_weight=w, save=True)
    got = layer.block_norm(put(t), t, pre_weight=w, post_weight=w, save=True)
    assert torch.equal(near.h, got.h) and torch.equal(near.z, got.z)
    layer.block_norm(t, t, pre_weight=w, post_weight=w, z=wide)
    assert torch.equal(wide, near.z)
    a = layer.block_norm_backward(t, near.h, near.h, near.y, near.rstd, pre_weight=w, post_weight=w)
    b = layer.block_norm_backward(put(t), near.h, near.h, near.y, near.rstd, pre_weight=w, post_weight=w)
    assert torch.equal(a.y, b.y) and torch.equal(a.pre_weight, b.pre_weight)
    kept = layer.ckpt_pack(t)
    far_kept = layer.ckpt_pack(put(t))
    assert torch.equal(kept.q, far_kept.q) and torch.equal(kept.exps, far_kept.exps)
    assert torch.equal(layer.ckpt_unpack(kept, put(torch.zeros_like(t))), layer.ckpt_unpack(kept))
    assert torch.equal(layer.ckpt_wgrad(put(t), kept), layer.ckpt_wgrad(t, kept))
    x, q, s, z = w4_case(S, N, N, 32, BF16, True, seed=2)
    weight = layer.w4_pack(q, s, z, group=32)
    want = layer.w4_linear(x, weight)
    assert torch.equal(layer.w4_linear(put(x), weight), want)
    assert torch.equal(layer.w4_linear(x, weight, put(torch.zeros_like(want))), want)


@pytest.mark.parametrize("S,N", [(9, 520), (5, 9000), (3, 20000)])
def test_block_norm_backward_in_place(S, N):
    """The C call may write the residual's gradient over dh and y's over dz."""
    import ctypes
    c = grad_case(S, N, BF16, BF16, True, "none", seed=21)
    want = run_grad(c)
    dz, dh = c["dz"].clone(), c["dh"].clone()
    sums = torch.empty((2, N), device="cuda")
    cfg = layer.gemm_rs_norm_config(N, layer.DTYPE_BF16, layer.DTYPE_BF16, 1, layer.GATE_NONE, 1, 1, 1e-5, 0.7, -0.9)
    a = layer.gemm_rs_norm_grad_args(
        dz.data_ptr(), N, dh.data_ptr(), N, c["h"].data_ptr(), N, c["y"].data_ptr(), N, c["rstd"].data_ptr(),
        c["post"].data_ptr(), None, c["pre"].data_ptr(), 0, dh.data_ptr(), N, dz.data_ptr(), N, sums[0].data_ptr(),
        sums[1].data_ptr(), None, 0)
    L = layer.lib()
    size = L.gemm_rs_block_norm_workspace(ctypes.byref(cfg), S)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    call = lambda n: L.gemm_rs_block_norm_backward(ctypes.byref(cfg), S, ctypes.byref(a), ws.data_ptr(), n,  # noqa: E731
                                                   torch.cuda.current_stream().cuda_stream)
    assert call(size - 1) == -8  # the workspace's size is checked
    assert call(size) == 0
    assert torch.equal(dz, want.y) and torch.equal(dh, want.residual)
    assert torch.equal(sums[0], want.pre_weight) and torch.equal(sums[1], want.post_weight)


@pytest.mark.parametrize("name,tokens", [("tiny", 1), ("tiny", 16), ("o_proj", 5)])
def test_example_runs_them_together(name, tokens):
    """The example's training step and decode: the operators on the layer's own buffers.  BF16 roundings (2^-9 rms) of
    h's or z's terms; 8-bit inputs: half a step of at most 2^-6 of a block's largest of 32 normal values; 4-bit
    weights: half of a fifteenth of a group's range, uniform."""
    import os
    import sys

    import synthetic
    from conftest import ROOT
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import layer_block

    found = layer_block.run(synthetic.CONFIGS[name], tokens, verbose=False)
    for k, limit in {"h": 4e-3, "z": 8e-3, "weight gradient (8-bit input)": 2e-2, "4-bit partial": 0.15, "decode h": 4e-3,
                     "decode z": 8e-3}.items():
        assert found[k] <= limit, (k, found[k])


def test_refusals():
    x, q, s, z = w4_case(4, 64, 128, 64, BF16, True, seed=1)
    weight = layer.w4_pack(q, s, z, group=64)
    for bad in (x.half(), x.float()):
        with pytest.raises(TypeError):
            layer.w4_linear(bad, weight)
    for bad in (x[:, :64], x.t(), x[0], x.cpu(), x.expand(4, 4, 128)):
        with pytest.raises(ValueError):
            layer.w4_linear(bad, weight)
    with pytest.raises(ValueError):
        layer.w4_linear(x[:1].expand(4, 128), weight)   # rows on top of each other
    with pytest.raises(ValueError):
        layer.w4_linear(x, weight, torch.empty((4, 63), dtype=BF16, device="cuda"))
    with pytest.raises(ValueError):
        layer.w4_pack(q, s[:, :1].contiguous(), z, group=64)
    with pytest.raises(TypeError):
        layer.w4_pack(q.to(torch.int32), s, z, group=64)
    c = norm_case(2, 4, 64, BF16, F32, True, "full", seed=1)
    with pytest.raises(TypeError):
        layer.block_norm(c["parts"].half(), c["residual"].to(BF16))
    with pytest.raises(TypeError):
        layer.block_norm(c["parts"], c["residual"], pre_weight=c["pre"].float())
    with pytest.raises(ValueError):
        layer.block_norm(c["parts"], c["residual"], gate=c["gate"][:3])
    with pytest.raises(ValueError):
        layer.block_norm(c["parts"], c["residual"][:3])
    with pytest.raises(ValueError):
        layer.block_norm([c["parts"][0], strided(c["parts"][1], 8)])
    with pytest.raises(ValueError):
        layer.block_norm(c["parts"], z=torch.empty((4, 64), dtype=BF16, device="cuda"))
    with pytest.raises(layer.GemmRSLayerError):
        layer.block_norm(c["parts"], eps=float("nan"))
    with pytest.raises(layer.GemmRSLayerError):
        layer.block_norm(torch.zeros((1, 32776), dtype=BF16, device="cuda"))
    gc = grad_case(4, 64, BF16, F32, True, "channel")
    for drop in ("dz", "h", "y", "rstd"):
        with pytest.raises(ValueError):
            run_grad(dict(gc, **{drop: None}))
    with pytest.raises(ValueError):
        run_grad(dict(gc, rstd=gc["rstd"][:1]))
    with pytest.raises(TypeError):
        run_grad(dict(gc, dz=gc["dz"].half()))
    kept = layer.ckpt_pack(x)
    with pytest.raises(TypeError):
        layer.ckpt_wgrad(x.float(), kept)
    with pytest.raises(TypeError):
        layer.ckpt_wgrad(x.half(), kept)
    with pytest.raises(ValueError):
        layer.ckpt_wgrad(x[:3], kept)
    with pytest.raises(TypeError):
        layer.ckpt_wgrad(x, kept, dtype=F16)
    with pytest.raises(ValueError):
        layer.ckpt_wgrad(x, kept, add=torch.zeros((128, 64), device="cuda"))
    with pytest.raises(ValueError):
        layer.Checkpoint(kept.q, kept.exps, 200, BF16)
    with pytest.raises(ValueError):
        layer.ckpt_pack(torch.zeros((4, 0), dtype=BF16, device="cuda"))
