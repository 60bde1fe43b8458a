"""Host-side checks of how the experts' products run.  If one fails after a change of the choice, the sizes that reach each kernel
have moved, and with them what is tested."""
import ctypes

import pytest

import experts_shapes as shapes
from test_experts_host import fp8, wgrad

ex = pytest.importorskip("tensor_gemm_reduce_amd.experts")
gr = pytest.importorskip("tensor_gemm_reduce_amd.gemm_rs")

BF16, F16, F32 = 0, 1, 2


def plan(args, call="gemm_rs_fp8_plan"):
    info = ex.gemm_rs_fp8_info()
    assert getattr(ex.lib(), call)(ctypes.byref(args), ctypes.byref(info)) == gr.OK
    return {n: getattr(info, n) for n, _ in info._fields_}


def check(got, form):
    assert (got["tile"], got["stages"]) == form
    assert got["workgroups"] <= 256 if form[0] == 256 else got["workgroups"] >= got["tiles"]
    return got["tiles"] > got["workgroups"]   # several tiles for a workgroup


@pytest.mark.parametrize("shape,half,single", shapes.DENSE)
def test_dense_forms(shape, half, single):
    M, N, K = shape
    for x in (BF16, F16, ex.DTYPE_FP8):
        for out, form in ((BF16, half), (F16, half), (F32, single)):
            check(plan(fp8(x_dtype=x, out_dtype=out, M=M, N=N, K=K, x_rows=M)), form)


@pytest.mark.parametrize("shape,half,single", shapes.EXPERTS)
@pytest.mark.parametrize("rows", [False, True])
def test_experts_forms(shape, half, single, rows):
    T, E, k, N, K, _ = shape
    for out, form in ((BF16, half), (F16, half), (F32, single)):
        got = plan(fp8(x_dtype=ex.DTYPE_FP8, out_dtype=out, M=T * k, N=N, K=K, x_rows=T * k if rows else T, E=E, offsets=256,
                       tokens=0 if rows else 256))
        check(got, form)


@pytest.mark.parametrize("shape,half,single", shapes.WGRAD)
def test_wgrad_forms(shape, half, single):
    T, E, N, K, _ = shape
    for dtype, out, form in ((BF16, BF16, half), (F16, F16, half), (BF16, F32, single), (F32, F32, single)):
        got = plan(wgrad(dtype=dtype, out_dtype=out, M=T, N=N, K=K, E=E, x_rows=T), "gemm_rs_experts_wgrad_plan")
        check(got, form)


def test_all_forms_are_there():
    """Every (tile, stages) of each kind of product; tiles of 256 x 256 one and several to a workgroup, in odd and even steps."""
    for cases, few in ((shapes.DENSE, {(16, 0), (32, 0)}), (shapes.EXPERTS, {(16, 0)}), (shapes.WGRAD, set())):
        assert {h for _, h, _ in cases} == few | {(128, 2), (128, 4), (256, 2)}
        assert {s for _, _, s in cases} == few | {(128, 2), (256, 2)}
    for out in (BF16, F32):
        large = [(s, fp8(out_dtype=out, M=s[0], N=s[1], K=s[2], x_rows=s[0])) for s, _, f in shapes.DENSE if f == (256, 2)]
        assert {(check(plan(a), (256, 2)), -(-s[2] // 128) % 2) for s, a in large} == {(False, 1), (True, 0), (True, 1)}
        large = [(s, fp8(out_dtype=out, M=s[0] * s[2], N=s[3], K=s[4], x_rows=s[0], E=s[1], offsets=256, tokens=256))
                 for s, _, f in shapes.EXPERTS if f == (256, 2)]
        assert {(check(plan(a), (256, 2)), -(-s[4] // 128) % 2) for s, a in large} == {(False, 1), (True, 0), (True, 1)}
        large = [wgrad(out_dtype=out, M=s[0], N=s[2], K=s[3], E=s[1], x_rows=s[0]) for s, _, f in shapes.WGRAD if f == (256, 2)]
        assert {check(plan(a, "gemm_rs_experts_wgrad_plan"), (256, 2)) for a in large} == {False, True}


def test_quantising_on_the_way():
    few = dict(M=4, x_rows=4, N=16, K=130)
    assert plan(fp8(**few))["quantises"] == 1
    assert plan(fp8(x_dtype=ex.DTYPE_FP8, **few))["quantises"] == 0
    assert plan(fp8(**dict(few, K=5000), x_stride=5000))["quantises"] == 0
    assert plan(fp8(M=0, x_rows=0)) == dict(tile=0, stages=0, quantises=0, tiles=0, workgroups=0)


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), gr.ERR_INVALID_ARG),
    (dict(E=2), gr.ERR_INVALID_ARG),
    (dict(tokens=256), gr.ERR_INVALID_ARG),
    (dict(N=1 << 23), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(E=1025, offsets=256), gr.ERR_UNSUPPORTED_SHAPE),
    # more tiles than a launch has workgroups for: refused before anything is enqueued
    (dict(M=(1 << 31) - 1, x_rows=100, N=1, E=1, offsets=256, tokens=256), gr.ERR_UNSUPPORTED_SHAPE),
])
def test_plan_refuses(kw, code):
    info = ex.gemm_rs_fp8_info()
    assert ex.lib().gemm_rs_fp8_plan(ctypes.byref(fp8(**kw)), ctypes.byref(info)) == code
    assert ex.lib().gemm_rs_fp8_plan(None, ctypes.byref(info)) == gr.ERR_INVALID_ARG
    assert ex.lib().gemm_rs_fp8_plan(ctypes.byref(fp8()), None) == gr.ERR_INVALID_ARG
    assert ex.lib().gemm_rs_experts_wgrad_plan(ctypes.byref(wgrad(N=1 << 23)), ctypes.byref(info)) == gr.ERR_UNSUPPORTED_SHAPE
    assert ex.lib().gemm_rs_experts_wgrad_plan(ctypes.byref(wgrad()), None) == gr.ERR_INVALID_ARG
