"""Host-side checks of include/gemm_rs_experts.h's calls (no GPU calls): exports, constants, configuration checks, sizes."""
import ctypes
import os
import re

import pytest
import torch

from conftest import ROOT

ex = pytest.importorskip("tensor_gemm_reduce_amd.experts")
layer = pytest.importorskip("tensor_gemm_reduce_amd.layer")
gr = pytest.importorskip("tensor_gemm_reduce_amd.gemm_rs")


def header():
    with open(os.path.join(ROOT, "include", "gemm_rs_experts.h")) as f:
        return f.read()


def test_every_declared_function_is_bound_and_exported():
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(gemm_rs_\w+)\s*\(", header(), re.M))
    assert names == set(ex.EXPORTS)
    for n in names:
        assert hasattr(ex.lib(), n), n


def test_header_constants_match_binding():
    consts = dict(re.findall(r"#define GEMM_RS_(\w+)\s+(\d+)", header()))
    assert {"FP8_BLOCK", "DTYPE_FP8", "ROUTE_MAX_EXPERTS"} <= set(consts)
    for k, v in consts.items():
        assert getattr(ex, k) == int(v), k


def test_packed_arguments_have_the_structures_sizes():
    assert ex._FP8_ARGS.size == ctypes.sizeof(ex.gemm_rs_fp8_args)
    assert ex._WGRAD_ARGS.size == ctypes.sizeof(ex.gemm_rs_experts_wgrad_args)
    assert ex._ROUTE_CONFIG.size == ctypes.sizeof(ex.gemm_rs_route_config)
    assert ex._PLAN_ARGS.size == ctypes.sizeof(ex.gemm_rs_expert_plan_args)


def route(**kw):
    base = dict(dtype=0, E=8, k=2, score=0, renormalise=1, groups=1, keep_groups=1, scale=1.0)
    base.update(kw)
    return ex.gemm_rs_route_config(*base.values())


@pytest.mark.parametrize("kw,code", [
    (dict(), gr.OK),
    (dict(E=1, k=1), gr.OK),
    (dict(E=1024, k=64), gr.OK),
    (dict(E=1025), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(E=1024, k=65), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(k=9), gr.ERR_INVALID_ARG),
    (dict(k=0), gr.ERR_INVALID_ARG),
    (dict(E=0), gr.ERR_INVALID_ARG),
    (dict(groups=3), gr.ERR_INVALID_ARG),
    (dict(groups=4, keep_groups=2), gr.OK),
    (dict(groups=4, keep_groups=5), gr.ERR_INVALID_ARG),
    (dict(groups=4, keep_groups=0), gr.ERR_INVALID_ARG),
    (dict(E=1024, groups=128, keep_groups=2), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(score=2), gr.ERR_INVALID_ARG),
    (dict(dtype=3), gr.ERR_INVALID_ARG),
    (dict(renormalise=2), gr.ERR_INVALID_ARG),
    (dict(scale=float("nan")), gr.ERR_INVALID_ARG),
])
def test_route_validate(kw, code):
    assert ex.lib().gemm_rs_route_validate(ctypes.byref(route(**kw))) == code


def test_plan_workspace():
    size = ex.lib().gemm_rs_expert_plan_workspace
    assert size(0, 8, 2) == 0 and size(32, 8, 2) == 0    # one workgroup's choices
    assert size(33, 8, 2) == (3 + 1) * 8 * 4             # workgroups of 16 tokens: their counts, and the sums
    assert size(32768, 256, 8) == (512 + 1) * 256 * 4    # of 64 tokens
    assert size(1 << 20, 8, 2) == (8192 + 1) * 8 * 4     # of 128
    assert size(30, 64, 64) == (2 + 1) * 64 * 4          # of 16, whose threads have no room for more choices
    assert size(-1, 8, 2) == 0 and size(10, 1025, 2) == 0 and size(10, 8, 65) == 0
    assert size(1 << 40, 8, 2) == 0


def fp8(**kw):
    base = dict(x_dtype=0, out_dtype=0, M=4, N=16, K=130, x_rows=4, E=0, x=256, x_stride=130, x_scales=0, w=256, w_scales=256,
                offsets=0, tokens=0, add=0, add_stride=0, out=256, out_stride=16)
    base.update(kw)
    return ex.gemm_rs_fp8_args(*base.values())


def test_fp8_workspace():
    size = lambda **kw: ex.lib().gemm_rs_fp8_workspace(ctypes.byref(fp8(**kw)))  # noqa: E731
    assert size(M=17, x_rows=17) == 17 * 256 + 2 * 20 + 8      # q, and two blocks' scales of 17 + 3 rows, to 16 bytes
    assert size(x_dtype=ex.DTYPE_FP8) == 0
    assert size(x_rows=100, M=100) == 100 * 256 + 2 * 104
    assert size() == 0                                         # a few rows are quantised by the product's kernel
    assert size(out_dtype=1) > 0 and size(K=5000) > 0 and size(K=4096, N=1 << 20) > 0  # unless it has no such form
    assert size(M=0) == 0 and size(K=0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(N=0), gr.ERR_INVALID_ARG),
    (dict(x_dtype=4), gr.ERR_INVALID_ARG),
    (dict(out_dtype=3), gr.ERR_INVALID_ARG),
    (dict(E=2), gr.ERR_INVALID_ARG),                          # experts go to the other call
    (dict(tokens=256), gr.ERR_INVALID_ARG),
    (dict(x_rows=5), gr.ERR_INVALID_ARG),
    (dict(K=(1 << 22) + 1, x_stride=1 << 23), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(M=1 << 31, x_rows=1 << 31), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(M=0, x_rows=0), gr.OK),
    (dict(x=0), gr.ERR_INVALID_ARG),
    (dict(x=257), gr.ERR_MISALIGNED),
    (dict(w=264), gr.ERR_MISALIGNED),
    (dict(w_scales=0), gr.ERR_INVALID_ARG),
    (dict(x_stride=129), gr.ERR_INVALID_ARG),
    (dict(out_stride=15), gr.ERR_INVALID_ARG),
    (dict(add=512, add_stride=16), gr.ERR_INVALID_ARG),       # needs an FP32 result
    (dict(add=256, add_stride=17, out_dtype=2), gr.ERR_INVALID_ARG),  # in place, of another stride
    (dict(M=17, x_rows=17), gr.ERR_SCRATCH),
])
def test_fp8_linear_refuses(kw, code):
    assert ex.lib().gemm_rs_fp8_linear(ctypes.byref(fp8(**kw)), None, 0, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(E=0, offsets=256), gr.ERR_INVALID_ARG),
    (dict(E=2), gr.ERR_INVALID_ARG),                          # no offsets
    (dict(E=2, offsets=256, x_rows=3), gr.ERR_INVALID_ARG),   # rows without tokens are x's own
    (dict(E=2, offsets=256, tokens=256, x_rows=1 << 24), gr.ERR_UNSUPPORTED_SHAPE),  # gathered from 4 GiB
    (dict(E=2, offsets=258), gr.ERR_MISALIGNED),
    (dict(E=1025, offsets=256), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(E=2, offsets=256, M=0, x_rows=0), gr.OK),
    (dict(E=2, offsets=256, M=100, x_rows=100, N=16), gr.ERR_SCRATCH),
])
def test_experts_linear_refuses(kw, code):
    assert ex.lib().gemm_rs_experts_linear(ctypes.byref(fp8(**kw)), None, 0, None) == code


def wgrad(**kw):
    base = dict(dtype=0, out_dtype=2, M=300, N=16, K=40, E=3, x_rows=300, dy=256, dy_stride=16, x=256, x_stride=40, offsets=256,
                tokens=0, add=0, dw=256)
    base.update(kw)
    return ex.gemm_rs_experts_wgrad_args(*base.values())


def test_wgrad_workspace():
    size = lambda **kw: ex.lib().gemm_rs_experts_wgrad_workspace(ctypes.byref(wgrad(**kw)))  # noqa: E731
    blocks = 300 // 128 + 3                                    # at most one ragged block an expert
    assert size() == blocks * 128 * (16 + 40) + (blocks * 20 + 15) // 16 * 16 + (blocks * 44 + 15) // 16 * 16
    assert size(M=0, x_rows=0) == 0 and size(E=0) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(out_dtype=1), gr.ERR_INVALID_ARG),
    (dict(E=0), gr.ERR_INVALID_ARG),
    (dict(x_rows=299), gr.ERR_INVALID_ARG),
    (dict(dw=0), gr.ERR_INVALID_ARG),
    (dict(offsets=0), gr.ERR_INVALID_ARG),
    (dict(dy_stride=15), gr.ERR_INVALID_ARG),
    (dict(out_dtype=0, add=256), gr.ERR_INVALID_ARG),
    (dict(N=1 << 23), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(E=1025), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(M=1 << 26, x_rows=1 << 26), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(), gr.ERR_SCRATCH),
])
def test_experts_wgrad_refuses(kw, code):
    assert ex.lib().gemm_rs_experts_wgrad(ctypes.byref(wgrad(**kw)), None, 0, None) == code


def test_quant_and_combine_refuse():
    L = ex.lib()
    assert L.gemm_rs_fp8_quant(3, 1, 1, 256, 1, 256, 256, None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_fp8_quant(0, 1, 0, 256, 1, 256, 256, None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_fp8_quant(0, 1, 8, 256, 8, 264, 256, None) == gr.ERR_MISALIGNED
    assert L.gemm_rs_fp8_quant(0, 0, 8, 0, 8, 0, 0, None) == gr.OK
    assert L.gemm_rs_fp8_pack(0, 0, 1, 1, 0, 256, 256, 256, None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_fp8_pack(0, 1 << 16, 1, 1, 0, 256, 256, 256, None) == gr.ERR_UNSUPPORTED_SHAPE
    assert L.gemm_rs_combine(0, 1, 1, 1, 65, 256, 1, 256, None, 256, 1, None) == gr.ERR_UNSUPPORTED_SHAPE
    assert L.gemm_rs_combine(0, 1, 1, 8, 2, 256, 7, 256, None, 256, 8, None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_combine(0, 0, 0, 8, 2, 0, 8, 0, None, 0, 8, None) == gr.OK
    assert L.gemm_rs_combine_backward(0, 1, 1, 8, 2, 256, 8, None, 8, 256, None, 256, 8, 256, None) == gr.ERR_INVALID_ARG
    plan = ex.gemm_rs_expert_plan_args(256, 256, 256)
    assert L.gemm_rs_expert_plan(1 << 30, 8, 4, 256, ctypes.byref(plan), None, 0, None) == gr.ERR_UNSUPPORTED_SHAPE
    assert L.gemm_rs_expert_plan(2000, 8, 4, 256, ctypes.byref(plan), None, 0, None) == gr.ERR_SCRATCH
    assert L.gemm_rs_expert_plan(1, 8, 4, 256, None, None, 0, None) == gr.ERR_INVALID_ARG


def test_route_refuses_more_threads_than_a_launch_has():
    plan = ex.gemm_rs_expert_plan_args(256, 256, 256)
    call = lambda T: ex.lib().gemm_rs_route(ctypes.byref(route(k=1)), T, 256, 8, None, 256, 256, ctypes.byref(plan), None, 0, None)  # noqa: E731
    assert call(1 << 30) == gr.ERR_UNSUPPORTED_SHAPE and call(1 << 31) == gr.ERR_UNSUPPORTED_SHAPE
    assert call(1 << 20) == gr.ERR_SCRATCH
    assert call(-1) == gr.ERR_INVALID_ARG


def test_binding_refuses_before_a_device_is_needed():
    t = torch.ones(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="score"):
        ex.route(t, 2, score="top")
    with pytest.raises(ValueError, match="two dimensions"):
        ex.route(t[0], 2)
    with pytest.raises(TypeError, match="logits"):
        ex.route(t.double(), 2)
    with pytest.raises(layer.GemmRSLayerError):
        ex.route(t, 1 << 32)
    with pytest.raises(ValueError, match="device tensor"):
        ex.fp8_quant(t)
    with pytest.raises(ValueError, match="w: expected"):
        ex.fp8_pack(t[0])
    with pytest.raises(ValueError, match="device tensor"):
        ex.combine(t, None, None)
