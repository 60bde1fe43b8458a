"""GPU tests of the experts' operators at the ends of their ranges: buffers of exactly the stated sizes,
FP32 results of blocks whose scales are the lowest and highest, gradients of saturated scores,
biases at the types' ends, and tokens that no plan makes."""
import pytest
import torch

import experts_ref as ref
from experts_ref import f64
from tensor_gemm_reduce_amd import experts as ex
from test_gpu_experts import BF16, F32, gen, integers

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


# ---- buffers of the sizes that the header states ------------------------------------------------------------------

def guarded(size):
    """(buffer of `size` bytes, check that nothing beside it was written)."""
    around = 1024
    buf = torch.full((size + 2 * around,), 0xA5, dtype=torch.uint8, device="cuda")

    def check():
        assert (buf[:around] == 0xA5).all() and (buf[around + size:] == 0xA5).all()
    return buf[around:around + size], check


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 128, 130])
@pytest.mark.parametrize("cols", [100, 256])
def test_calls_write_the_stated_layout_and_nothing_else(rows, cols):
    """q [rows][Kp] and scales [Kp / 128][rows + 3 rounded up to 4], for every call that makes them."""
    x = torch.randn((rows, cols), generator=gen(rows)).cuda()
    kp, rp = (cols + 127) // 128 * 128, (rows + 6) // 4 * 4
    L = ex.lib()
    for E, call in ((1, lambda q, s: L.gemm_rs_fp8_quant(2, rows, cols, x.data_ptr(), cols, q, s, stream())),
                    (1, lambda q, s: L.gemm_rs_fp8_quant_transposed(2, cols, rows, x.t().contiguous().data_ptr(), rows, q, s, stream())),
                    (1, lambda q, s: L.gemm_rs_fp8_pack(2, 1, rows, cols, 0, x.data_ptr(), q, s, stream())),
                    (3, lambda q, s: L.gemm_rs_fp8_pack(2, 3, rows, cols, 0, x.repeat(3, 1).data_ptr(), q, s, stream()))):
        (q, q_check), (s, s_check) = guarded(E * rows * kp), guarded(E * rp * kp // 128)
        assert call(q.data_ptr(), s.data_ptr()) == 0
        torch.cuda.synchronize()
        q_check()
        s_check()
        m = ex.Fp8(q.view(E, rows, kp).view(torch.float8_e4m3fn), s.view(E, kp // 128, rp), rows, cols)
        # quantised to within half a step of e4m3 of its block's largest value
        assert ((m.values() - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -9 * x.abs().max()).all()


# ---- FP32 results at both ends of the scales ------------------------------------------------------------------------

# exponents of blocks: the lowest (where e4m3's values times 2^e are no BF16 numbers), those beside it, and the highest
ENDS = (-126, -125, -124, -120, -117, -110, 0, 113, 119, 120)


def bytes_of(g, rows, K):
    """Finite e4m3 bytes, subnormal ones and zeros among them; zeros past K."""
    q = torch.randint(0, 256, (rows, (K + 127) // 128 * 128), generator=g, dtype=torch.int32)
    q[q % 128 == 127] = 1
    q[:, K:] = 0
    return q.to(torch.uint8)


def operand(g, e, K):
    """(an Fp8 [.., rows][K] with block exponents e [.., rows][blocks], what it stands for in 64 bits); random unused bytes."""
    lead, (rows, blocks) = e.shape[:-2], e.shape[-2:]
    n = max(1, int(torch.tensor(lead).prod())) if lead else 1
    q = bytes_of(g, n * rows, K).view(*lead, rows, blocks * 128)
    s = torch.randint(0, 256, (*lead, blocks, (rows + 6) // 4 * 4), generator=g, dtype=torch.int32).to(torch.uint8)
    s[..., :rows] = (e + 127).transpose(-1, -2).to(torch.uint8)
    q = q.cuda().view(torch.float8_e4m3fn)
    values = q.double() * torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), e.cuda().repeat_interleave(128, -1))
    return ex.Fp8(q, s.cuda(), rows, K), values[..., :K]


def exponents(g, rows, blocks, share=1.0):
    """Exponents of x's blocks: near ENDS in turn for a `share` of the rows, near zero for the others."""
    e = torch.tensor([ENDS[b % len(ENDS)] for b in range(blocks)]) + torch.randint(-2, 3, (rows, blocks), generator=g)
    e = torch.where(torch.rand((rows, 1), generator=g) < share, e, torch.randint(-3, 4, (rows, blocks), generator=g))
    return e.clamp(-126, 120)


def partners(g, rows, blocks, share=1.0):
    """Those of w's: where all of x's rows are at an end, at the other one (products are about one); else part of the way, so
    that no product leaves FP32."""
    c = torch.tensor([ENDS[b % len(ENDS)] for b in range(blocks)])
    e = -c if share == 1 else -20 * c.sign()
    return (e + torch.randint(-2, 3, (rows, blocks), generator=g)).clamp(-126, 120)


def near(got, x, w, add=0.0):
    """Within (K + 2) 2^-24 sum |x| |w|, the stated bound, the rounding of the sum with add, and the rounding of K products to
    multiples of 2^-149."""
    want, mag = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    bound = (x.shape[1] + 2) * 2.0 ** -24 * mag
    off = (got.double() - (want + add)).abs()
    ok = off <= bound + 2.0 ** -24 * (want + add).abs() + x.shape[1] * 2.0 ** -149
    assert ok.all(), (int((~ok).sum()), float((off / (bound + 2.0 ** -149))[~ok].max()))


# few rows, both forms; tiles of 128 x 128; of 256 x 256, one and more for a workgroup
DENSE = [(3, 40, 300), (16, 33, 1300), (20, 40, 600), (130, 150, 1300), (300, 260, 130), (4090, 4096, 384), (8100, 4300, 256)]


@pytest.mark.parametrize("M,N,K", DENSE)
@pytest.mark.parametrize("share", [1.0, 0.003])
def test_fp32_results_of_blocks_at_both_ends(M, N, K, share):
    g = gen(M + N)
    blocks = (K + 127) // 128
    x, xv = operand(g, exponents(g, M, blocks, share), K)
    w, wv = operand(g, partners(g, N, blocks, share), K)
    near(ex.fp8_linear(x, w, dtype=F32), xv, wv)
    add = integers(g, M, N).cuda()
    got = add.clone()
    assert ex.fp8_linear(x, w, add=got, out=got) is got
    near(got, xv, wv, add.double())


@pytest.mark.parametrize("M,N,K", [(5, 40, 200), (17, 40, 200), (200, 130, 384)])
@pytest.mark.parametrize("top", [2.0 ** -118, 2.0 ** -126, 2.0 ** -133, 1.99 * 2.0 ** 127])
def test_fp32_results_of_operands_at_both_ends(M, N, K, top):
    """Matrices whose largest values are at an end of FP32, quantised by the calls, times others that bring them back."""
    g = gen(N)
    x = torch.rand((M, K), generator=g) * (2 * torch.randint(0, 2, (M, K), generator=g) - 1) * top
    w = torch.randn((N, K), generator=g) * (2.0 ** 100 if top < 1 else 2.0 ** -126)
    near(ex.fp8_linear(x.cuda(), ex.fp8_pack(w.cuda())), ref.quantised(x).cuda(), ref.quantised(w, 128, 128).cuda())
    near(ex.fp8_linear(w.cuda(), ex.fp8_pack(x.cuda())), ref.quantised(w).cuda(), ref.quantised(x, 128, 128).cuda())


# T, E, k, N, K: few rows an expert; tiles of 128; of 256, one and more for a workgroup
EXPERTS = [(6, 4, 2, 40, 300), (300, 3, 2, 140, 300), (8192, 2, 1, 1700, 384), (9000, 3, 2, 1700, 256)]


@pytest.mark.parametrize("T,E,k,N,K", EXPERTS)
@pytest.mark.parametrize("rows", [False, True])
@pytest.mark.parametrize("share", [1.0, 0.01])
def test_experts_fp32_results_of_blocks_at_both_ends(T, E, k, N, K, rows, share):
    g = gen(T)
    blocks = (K + 127) // 128
    plan = ex.plan(torch.rand((T, E), generator=g).argsort(1)[:, :k].to(torch.int32).contiguous().cuda(), E)
    at, tokens = plan.offsets.tolist(), plan.tokens.long()
    x, xv = operand(g, exponents(g, T * k if rows else T, blocks, share), K)
    w, wv = operand(g, torch.stack([partners(g, N, blocks, share) for _ in range(E)]), K)
    y = ex.experts_linear(x, w, plan, rows=rows, dtype=F32)
    for e in range(E):
        r = slice(at[e], at[e + 1])
        near(y[r], xv[r] if rows else xv[tokens[r]], wv[e])


@pytest.mark.parametrize("T,E,N,K", [(300, 3, 70, 130), (700, 2, 2100, 2100), (1000, 4, 2750, 2700)])
def test_experts_wgrad_of_operands_at_both_ends(T, E, N, K):
    """Gradients of 2^-128 and inputs of 2^100, in some blocks; FP32 operands."""
    g = gen(E)
    plan = ex.plan(torch.randint(0, E, (T, 1), generator=g, dtype=torch.int32).cuda(), E)
    at, tokens = plan.offsets.tolist(), plan.tokens.long().cpu()
    dy, x = torch.randn((T, N), generator=g), torch.randn((T, K), generator=g)
    dy[:, ::7] *= 2.0 ** -128
    x[:, ::5] *= 2.0 ** 100
    dw = ex.experts_wgrad(dy.cuda(), x.cuda(), plan)
    for e in range(E):
        r = slice(at[e], at[e + 1])
        near(dw[e], ref.quantised(dy[r], 128, 1).t().contiguous().cuda(), ref.quantised(x[tokens[r]], 128, 1).t().contiguous().cuda())


@pytest.mark.parametrize("M,N,K", [(3, 40, 300), (20, 33, 1300), (130, 150, 1300), (200, 120, 384)])
def test_16_bit_results_of_blocks_at_both_ends(M, N, K):
    """The scales are the matrix instruction's own operands there: every byte from 1 on, and what eights of products drop."""
    g = gen(K)
    blocks = (K + 127) // 128
    x, xv = operand(g, exponents(g, M, blocks), K)
    w, wv = operand(g, partners(g, N, blocks), K)
    want, mag, top = (t.cuda() for t in ref.product(xv.cpu(), wv.cpu()))
    sums, drop = (K + 2) * 2.0 ** -24 * mag, 2.0 ** -10 * top
    off = (ex.fp8_linear(x, w, dtype=BF16).double() - want).abs()
    assert not (off > 2.0 ** -8 * (want.abs() + drop + sums) + drop + sums).any()


def test_blocks_of_zeros_beside_others():
    """Zeros at the lowest scale, as a caller's own matrices may have them, change nothing."""
    g = gen(3)
    x, xv = operand(g, torch.zeros((300, 3), dtype=torch.int64), 384)
    w, wv = operand(g, torch.zeros((200, 3), dtype=torch.int64), 384)
    x.q.view(torch.uint8)[::2, 128:256] = 0
    x.scales[1, :300:2] = 1
    xv[::2, 128:256] = 0
    near(ex.fp8_linear(x, w, dtype=F32), xv, wv)


@pytest.mark.parametrize("M,N", [(5, 40), (130, 140)])
def test_fp32_results_below_the_normal_range(M, N):
    g = gen(M)
    x, xv = operand(g, torch.full((M, 2), -90), 256)
    w, wv = operand(g, torch.full((N, 2), -48), 256)
    near(ex.fp8_linear(x, w, dtype=F32), xv, wv)


# ---- the sigmoid's gradient where it saturates -------------------------------------------------------------------------

@pytest.mark.parametrize("E,k", [(6, 2), (40, 5), (300, 8)])
@pytest.mark.parametrize("renormalise", [False, True])
def test_sigmoid_gradient_of_saturated_logits(E, k, renormalise):
    """dl = ds s (1 - s) to a few roundings of each factor, also where s is next to one: 1 - s is 1 / (1 + e^l)."""
    g = gen(E)
    T = 50
    logits = 30 * (2 * torch.rand((T, E), generator=g) - 1)
    logits[0, :4] = torch.tensor([8.0, 12.0, 17.0, 30.0])
    r = ex.route(logits.cuda(), k, score="sigmoid", renormalise=renormalise)
    dw = torch.randn((T, k), generator=g)
    got = f64(ex.route_backward(dw.cuda(), logits.cuda(), r.experts, score="sigmoid", renormalise=renormalise))
    l, e = f64(logits), r.experts.cpu().long()
    s, rest = torch.sigmoid(l), torch.sigmoid(-l)
    ds = f64(dw)
    size = ds.abs()   # the sum of the magnitudes that make ds
    if renormalise:
        se = s.gather(1, e)
        D = se.sum(1, keepdim=True) + 1e-20
        ds, size = (ds - (ds * se).sum(1, keepdim=True) / D) / D, (size + (size * se).sum(1, keepdim=True) / D) / D
    factor = (s * rest).gather(1, e)
    want = torch.zeros_like(l).scatter_(1, e, ds * factor)
    # each of s and 1 - s: exp (2 units), of a logit that is a number; the sum and the quotient: 4; their product, ds: k + 8
    bound = torch.zeros_like(l).scatter_(1, e, (k + 24) * 2.0 ** -24 * size * factor) + 1e-37
    bad = (got - want).abs() > bound
    assert not bad.any(), float(((got - want).abs() / bound).max())
    # against differences of the score, in 64 bits: h^2 / 6 of it and less, and two scores' roundings of 2^-52 each over 2 h
    h = 1e-4
    diff = (torch.sigmoid(l + h) - torch.sigmoid(l - h)) / (2 * h)
    bad = (diff - s * rest).abs() > h * h / 6 * s * rest + 2 * 2.0 ** -52 / (2 * h)
    assert not bad.any()


@pytest.mark.parametrize("E,k", [(2, 1), (2, 2), (6, 2), (40, 5), (300, 8), (1000, 64)])
@pytest.mark.parametrize("renormalise", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_where_one_score_is_nearly_all(E, k, renormalise, score):
    """What is left of the others counts: sums of s_j (g_i - g_j), relative to the terms that are there, not to g_i."""
    g = gen(E + k)
    T = 60
    logits = torch.randn((T, E), generator=g)
    for t in range(T):
        logits[t, t % E] += t / 2   # ahead of the rest by up to 30
    r = ex.route(logits.cuda(), k, score=score, renormalise=renormalise, scale=2.0)
    dw = torch.randn((T, k), generator=g)
    got = f64(ex.route_backward(dw.cuda(), logits.cuda(), r.experts, score=score, renormalise=renormalise, scale=2.0))
    l, e = f64(logits), r.experts.cpu().long()
    s = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l)
    se, ds = s.gather(1, e), 2 * f64(dw)
    size = ds.abs()
    if renormalise:
        D = se.sum(1)[:, None, None] + 1e-20
        apart = ds[:, :, None] - ds[:, None, :]              # [i][j]
        sizes = (ds.abs()[:, :, None] + ds.abs()[:, None, :]) * (1 - torch.eye(k))
        ds, size = (((se[:, None, :] * a).sum(2, keepdim=True) / D / D)[:, :, 0] + 1e-20 * b / D[:, :, 0] ** 2
                    for a, b in ((apart, ds), (sizes, size)))
    full, full_size = (torch.zeros_like(l).scatter_(1, e, v) for v in (ds, size))
    if score == "softmax":
        others = s.sum(1, keepdim=True) - s                  # 1 - s, by what is not s: the largest's is summed without it
        top = s.argmax(1, keepdim=True)
        others.scatter_(1, top, s.scatter(1, top, 0.0).sum(1, keepdim=True))
        rest = lambda v: torch.stack([(s * v).scatter(1, torch.full((T, 1), i), 0.0).sum(1) for i in range(E)], 1)  # noqa: E731
        want, mag = s * (full * others - rest(full)), s * (full_size * others + rest(full_size))
    else:
        want, mag = full * s * torch.sigmoid(-l), full_size * s * torch.sigmoid(-l)
    # in units of 2^-24: a score's exp is of a rounded difference of up to 35 (half of it, and 2), its sum has E / 64 + 6 in a row, and
    # a quotient: 28 + E / 64; a term has up to four of them, two sums over k and one more over E / 64 + 6
    rel = (4 * (28 + E / 64) + 2 * k + E / 64 + 24) * 2.0 ** -24
    bad = (got - want).abs() > rel * mag + 1e-37
    assert not bad.any(), (int(bad.sum()), float(((got - want).abs() / (rel * mag + 1e-37)).max()))


# ---- groups with biases at the types' ends ----------------------------------------------------------------------------

@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [1, 40])
def test_groups_whose_sums_leave_fp32(score, T):
    """Biases of the type's lowest and highest value: sums of two are past FP32, not past 64 bits."""
    low, high = torch.finfo(F32).min, torch.finfo(F32).max
    off = -float("inf")
    l = torch.tensor([0.5, -0.25, 1.0, 0.75, -0.5, 0.25, 2.0, 1.5])
    cases = [
        # a group that is off beside one whose experts are on, at the lowest bias: the latter stays
        ([off, off, 1.0, 0.5, 0.25, 0.75, off, off], [0, 0, 0, 0, low, low, 0, 0], 4, 2),
        # sums past the lowest value, that differ
        (l.tolist(), [low, low, 0, 0, low * 0.75, low * 0.8, 0, 0], 4, 3),
        # and past the highest
        (l.tolist(), [0.6 * high, 0.7 * high, 0.9 * high, high, 0.8 * high, 0.75 * high, 0, 0], 4, 1),
        (l.tolist(), [0.6 * high, 0.7 * high, 0.9 * high, high, 0.8 * high, 0.75 * high, 0, 0], 4, 2),
    ]
    for logits, bias, groups, keep in cases:
        logits, bias = torch.tensor([logits]).repeat(T, 1), torch.tensor(bias)
        for k in (1, 2, 4, 6):
            want = ref.route(logits, k, score, bias, groups, keep, True, 1.0)[1]
            r = ex.route(logits.cuda(), k, score=score, bias=bias.cuda(), groups=groups, keep_groups=keep)
            assert torch.equal(r.experts.cpu(), want), (bias, keep, k, r.experts[0], want[0])


# ---- tokens that no plan makes ----------------------------------------------------------------------------------------

@pytest.mark.parametrize("T,E,N,K,wide", [(6, 3, 20, 130, False), (6, 3, 20, 5000, False), (6, 3, 20, 130, True), (300, 2, 140, 130, False),
                                          (8000, 2, 2100, 130, False)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_token_out_of_range_has_no_input(T, E, N, K, wide, dtype):
    """Its row is zeros in every kernel: for few rows (quantising on the way, or not), and tiles of both sizes."""
    g = gen(T)
    plan = ex.plan((torch.arange(T, dtype=torch.int32) % E)[:, None].contiguous().cuda(), E)
    bad = torch.tensor([-1, T, 1 << 30, -(1 << 31)], dtype=torch.int32).cuda()
    plan.tokens[1::2] = bad.repeat((T + 3) // 4)[:plan.tokens[1::2].numel()]
    x, w = integers(g, T, K, low=-3, high=3).to(dtype), integers(g, E, N, K, low=-3, high=3).to(dtype)
    given = ex.fp8_quant(x.cuda()) if wide else x.cuda()
    y = ex.experts_linear(given, ex.fp8_pack(w.cuda()), plan, dtype=dtype)
    assert (y[1::2] == 0).all()
    at = plan.offsets.tolist()
    for e in range(E):
        r = torch.arange(at[e], at[e + 1], device="cuda")
        r = r[r % 2 == 0]
        want = x.cuda().double()[plan.tokens[r].long()] @ w[e].cuda().double().t().contiguous()
        assert torch.equal(y[r].double(), want.to(dtype).double())
    if dtype is F32:
        add = torch.full((T, N), 5.0, device="cuda")
        assert (ex.experts_linear(given, ex.fp8_pack(w.cuda()), plan, add=add, dtype=F32)[1::2] == 5).all()


@pytest.mark.parametrize("name", ["offsets", "tokens"])
def test_a_plan_with_parts_exchanged_is_refused(name):
    """Parts of other sizes or types, or in host memory, are refused by the calls that read them."""
    plan = ex.plan(torch.zeros((4, 2), dtype=torch.int32, device="cuda"), 3)
    x, dy, w = (torch.ones(s, dtype=BF16, device="cuda") for s in ((4, 16), (8, 8), (3, 8, 16)))
    weight, whole = ex.fp8_pack(w), getattr(plan, name)
    for part, error in ((whole[:-1], ValueError), (whole.long(), TypeError), (whole.cpu(), ValueError), (whole[:, None], ValueError)):
        setattr(plan, name, part)
        for call in (lambda: ex.experts_linear(x, weight, plan), lambda: ex.experts_wgrad(dy, x, plan)):
            with pytest.raises(error, match=name):
                call()
    setattr(plan, name, whole)
    assert (ex.experts_linear(x, weight, plan) == 16).all()
