"""GPU tests of every form of the experts' products (test_experts_plan.py holds which shape reaches which), in all types.

Operands are small integers: their sums are exact in FP32, whatever the order, so results are the 64-bit ones, rounded once."""
import pytest
import torch

import experts_shapes as shapes
from test_gpu_experts import BF16, F16, F32, TYPES, gen, integers, strided
from tensor_gemm_reduce_amd import experts as ex

pytestmark = pytest.mark.gpu


def few(g, *shape):
    return integers(g, *shape, low=-3, high=3).cuda()


def times(x, w):
    """x w^T in 64 bits."""
    return x.double() @ w.double().t().contiguous()


def choices(g, T, E, k, dead):
    s = torch.rand((T, E), generator=g)
    s[:, list(dead)] = -1
    e = s.argsort(1, descending=True)[:, :k]
    if k > E - len(dead):
        e[s.gather(1, e) < 0] = -1   # no expert is left for these
    return e.to(torch.int32).contiguous()


@pytest.mark.parametrize("shape", [s for s, _, _ in shapes.DENSE])
@pytest.mark.parametrize("dtype", TYPES)
def test_dense(shape, dtype):
    M, N, K = shape
    g = gen(M + N)
    x, w = few(g, M, K), few(g, N, K)
    want = times(x, w)
    weight, wide = ex.fp8_pack(w), torch.full((M, N + 5), 99.0, dtype=dtype, device="cuda")
    assert torch.equal(ex.fp8_linear(x.to(dtype), weight), want.to(dtype))
    out = wide[:, 2:N + 2]
    ex.fp8_linear(ex.fp8_quant(x), weight, out=out)
    assert torch.equal(out, want.to(dtype))
    assert (wide[:, :2] == 99).all() and (wide[:, N + 2:] == 99).all()
    if dtype is F32:
        add = few(g, M, N)
        main = add.clone()
        ex.fp8_linear(x, weight, add=main, out=main)
        assert torch.equal(main.double(), want + add)
        assert torch.equal(ex.fp8_linear(x, weight, add=strided(add.cpu()), dtype=F32).double(), want + add)


@pytest.mark.parametrize("shape", [s for s, _, _ in shapes.EXPERTS])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [False, True])
def test_experts(shape, dtype, rows):
    T, E, k, N, K, dead = shape
    g = gen(T + N)
    plan = ex.plan(choices(g, T, E, k, dead).cuda(), E)
    at, tokens = plan.offsets.tolist(), plan.tokens.long()
    n = at[E]
    x, w = few(g, T, K), few(g, E, N, K)
    given = torch.zeros((T * k, K), device="cuda")
    given[:n] = x[tokens[:n]]
    given = given if rows else x
    want = torch.full((T * k, N), 77.0, dtype=torch.float64, device="cuda")
    for e in range(E):
        r = slice(at[e], at[e + 1])
        want[r] = times(x[tokens[r]], w[e])
    weight, out = ex.fp8_pack(w), torch.full((T * k, N), 77.0, dtype=dtype, device="cuda")
    ex.experts_linear(given.to(dtype), weight, plan, rows=rows, out=out)
    assert torch.equal(out, want.to(dtype))            # rows behind the last as they were
    out.fill_(77.0)
    ex.experts_linear(ex.fp8_quant(given), weight, plan, rows=rows, out=out)
    assert torch.equal(out, want.to(dtype))
    if dtype is F32:
        main = few(g, T * k, N)
        add = main.double()
        ex.experts_linear(given, weight, plan, rows=rows, add=main, out=main)
        assert torch.equal(main[:n].double(), (want + add)[:n]) and torch.equal(main[n:].double(), add[n:])


@pytest.mark.parametrize("shape", [s for s, _, _ in shapes.WGRAD])
@pytest.mark.parametrize("dtype,out", [(BF16, BF16), (F16, F16), (BF16, F32), (F16, F32), (F32, F32)])
def test_wgrad(shape, dtype, out):
    T, E, N, K, dead = shape
    g = gen(E + N)
    some = torch.tensor([e for e in range(E) if e not in dead])
    # experts of very different sizes: the first that has rows has half of them
    experts = torch.where(torch.rand(T, generator=g) < 0.5, some[0], some[torch.randint(0, len(some), (T,), generator=g)])
    plan = ex.plan(experts[:, None].to(torch.int32).contiguous().cuda(), E)
    at, tokens = plan.offsets.tolist(), plan.tokens.long()
    dy, x = few(g, T, N), few(g, T, K)
    want = torch.stack([times(dy[at[e]:at[e + 1]].t(), x[tokens[at[e]:at[e + 1]]].t()) if at[e] < at[e + 1]
                        else torch.zeros((N, K), dtype=torch.float64, device="cuda") for e in range(E)])
    dw = ex.experts_wgrad(dy.to(dtype), x.to(dtype), plan, dtype=out)
    assert dw.dtype is out and torch.equal(dw, want.to(out))
    assert torch.equal(ex.experts_wgrad(dy.to(dtype), x[tokens].to(dtype), plan, rows=True, dtype=out), dw)
    if out is F32:
        main = torch.full_like(dw, 5.0)
        ex.experts_wgrad(dy.to(dtype), x.to(dtype), plan, add=main, out=main)
        assert torch.equal(main.double(), want + 5)


@pytest.mark.parametrize("T,E,k,N,K,dead", [(16, 8, 2, 40, 256, (3,)), (150, 4, 2, 48, 256, ()), (500, 4, 2, 200, 200, (1,))])
def test_experts_in_f16(T, E, k, N, K, dead):
    """The forms of F16 that quantise on the way and that do not, both orders of rows, strided."""
    g = gen(T)
    plan = ex.plan(choices(g, T, E, k, dead).cuda(), E)
    at, tokens = plan.offsets.tolist(), plan.tokens.long()
    x, w = few(g, T, K), few(g, E, N, K)
    want = torch.cat([times(x[tokens[at[e]:at[e + 1]]], w[e]) for e in range(E)])
    weight = ex.fp8_pack(w.to(F16))
    for given, rows in ((x, False), (x[tokens], True)):
        y = ex.experts_linear(strided(given.to(F16).cpu()), weight, plan, rows=rows)
        assert y.dtype is F16 and torch.equal(y, want.to(F16))
        assert torch.equal(ex.experts_linear(given.to(F16), weight, plan, rows=rows, dtype=F32).double(), want)
