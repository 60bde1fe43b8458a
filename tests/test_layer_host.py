"""Host-side checks of libgemm_rs_layer.so (no GPU calls): exports, constants,
configuration checks and sizes."""
import ctypes
import os
import re

import pytest
import torch

from conftest import ROOT

layer = pytest.importorskip("tensor_gemm_reduce_amd.layer")
gr = pytest.importorskip("tensor_gemm_reduce_amd.gemm_rs")


def header():
    with open(os.path.join(ROOT, "include", "gemm_rs_layer.h")) as f:
        return f.read()


def test_every_declared_function_is_bound_and_exported():
    names = set(re.findall(r"^\s*(?:int|size_t|const char \*)\s*\*?\s*(gemm_rs_\w+)\s*\(", header(), re.M))
    assert names == set(layer.EXPORTS)
    for n in names:
        assert hasattr(layer.lib(), n), n


def test_header_constants_match_binding():
    consts = dict(re.findall(r"#define GEMM_RS_(\w+)\s+(\d+)", header()))
    assert {"DTYPE_F32", "GATE_FULL", "NORM_MAX_WIDTH", "CKPT_NAN"} <= set(consts)
    for k, v in consts.items():
        assert getattr(layer, k) == int(v), k


def w4(**kw):
    base = dict(N=8192, K=1024, group=128, dtype=layer.DTYPE_BF16, zero_points=0)
    base.update(kw)
    return layer.gemm_rs_w4_config(*(base[k] for k in ("N", "K", "group", "dtype", "zero_points")))


@pytest.mark.parametrize("kw,code", [
    (dict(), gr.OK),
    (dict(N=1, K=2, group=32), gr.OK),
    (dict(K=1000, group=1000), gr.OK),          # one scale per row
    (dict(K=1000, group=96), gr.OK),
    (dict(group=48), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(group=0), gr.ERR_INVALID_ARG),
    (dict(K=1023), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(K=0), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(N=0), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(N=-1), gr.ERR_INVALID_ARG),
    (dict(dtype=layer.DTYPE_F32), gr.ERR_INVALID_ARG),
    (dict(zero_points=2), gr.ERR_INVALID_ARG),
    (dict(N=1 << 24, K=1 << 24), gr.ERR_UNSUPPORTED_SHAPE),
])
def test_w4_validate(kw, code):
    assert layer.lib().gemm_rs_w4_validate(ctypes.byref(w4(**kw))) == code


def test_w4_packed_bytes():
    size = lambda **kw: layer.lib().gemm_rs_w4_packed_bytes(ctypes.byref(w4(**kw)))  # noqa: E731
    assert size() == 8192 * 1024 // 2 + 8192 * 8 * 2                      # nibbles and scales, nothing padded
    assert size(group=32, zero_points=1) == 8192 * 1024 // 2 + 8192 * 32 * 3
    assert size(N=17, K=130, group=32) == 2 * 2 * 1024 + 2 * 2 * 16 * 4 * 2   # rows to 16, inputs to 128
    assert size(group=48) == 0


def norm(**kw):
    base = dict(width=8192, dtype=0, residual_dtype=0, parts=8, gate=0, post_norm=1, pre_norm=1, eps=1e-5, block_scale=1.0,
                residual_scale=1.0)
    base.update(kw)
    return layer.gemm_rs_norm_config(*base.values())


@pytest.mark.parametrize("kw,code", [
    (dict(), gr.OK),
    (dict(width=1), gr.OK),
    (dict(width=32768), gr.OK),
    (dict(width=32769), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(width=0), gr.ERR_UNSUPPORTED_SHAPE),
    (dict(residual_dtype=2), gr.OK),
    (dict(residual_dtype=1), gr.ERR_INVALID_ARG),
    (dict(dtype=2, residual_dtype=0), gr.ERR_INVALID_ARG),
    (dict(dtype=3, residual_dtype=2), gr.ERR_INVALID_ARG),
    (dict(parts=0), gr.ERR_INVALID_ARG),
    (dict(parts=9), gr.ERR_INVALID_ARG),
    (dict(gate=4), gr.ERR_INVALID_ARG),
    (dict(post_norm=2), gr.ERR_INVALID_ARG),
    (dict(eps=-1.0), gr.ERR_INVALID_ARG),
    (dict(eps=float("nan")), gr.ERR_INVALID_ARG),
    (dict(eps=0.0), gr.OK),
    (dict(block_scale=float("inf")), gr.ERR_INVALID_ARG),
    (dict(residual_scale=float("nan")), gr.ERR_INVALID_ARG),
])
def test_norm_validate(kw, code):
    assert layer.lib().gemm_rs_norm_validate(ctypes.byref(norm(**kw))) == code


def test_calls_without_rows_or_with_bad_arguments_touch_no_gpu():
    L = layer.lib()
    a = layer.gemm_rs_norm_args()
    assert L.gemm_rs_block_norm(ctypes.byref(norm()), 0, ctypes.byref(a), None) == gr.OK
    assert L.gemm_rs_block_norm(ctypes.byref(norm()), 4, ctypes.byref(a), None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_block_norm(ctypes.byref(norm()), -1, ctypes.byref(a), None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_w4_linear(ctypes.byref(w4()), None, 0, None, 0, None, 0, None) == gr.OK
    assert L.gemm_rs_w4_linear(ctypes.byref(w4()), None, 1, None, 1024, None, 8192, None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_w4_linear(ctypes.byref(w4()), 16, 1, 2, 1024, 3, 8192, None) == gr.ERR_MISALIGNED
    assert L.gemm_rs_w4_linear(ctypes.byref(w4()), 16, 1, 2, 1023, 2, 8192, None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_w4_linear(ctypes.byref(w4()), 8, 1, 2, 1024, 2, 8192, None) == gr.ERR_MISALIGNED
    assert L.gemm_rs_ckpt_pack(0, 0, 32, None, 32, None, None, None) == gr.OK
    assert L.gemm_rs_ckpt_pack(3, 1, 32, 16, 32, 16, 16, None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_ckpt_pack(0, 1, 32, 16, 31, 16, 16, None) == gr.ERR_INVALID_ARG
    assert L.gemm_rs_ckpt_pack(0, 1, 32, 16, 32, 8, 16, None) == gr.ERR_MISALIGNED
    assert L.gemm_rs_ckpt_unpack(0, 1, 0, 16, 16, 16, 32, None) == gr.ERR_INVALID_ARG
    g = layer.gemm_rs_norm_grad_args()
    assert L.gemm_rs_block_norm_backward(ctypes.byref(norm()), 4, ctypes.byref(g), None, 0, None) == gr.ERR_INVALID_ARG
    w = layer.gemm_rs_wgrad_args(0, 2, 8, 64, 64, 16, 64, 16, 16, None, 0, None, 64)
    assert L.gemm_rs_ckpt_wgrad(ctypes.byref(w), None, 0, None) == gr.ERR_INVALID_ARG     # no dw
    w.dw, w.out_dtype = 16, 1
    assert L.gemm_rs_ckpt_wgrad(ctypes.byref(w), None, 0, None) == gr.ERR_INVALID_ARG     # out f16 of bf16
    w.out_dtype, w.dtype = 2, 2
    assert L.gemm_rs_ckpt_wgrad(ctypes.byref(w), None, 0, None) == gr.ERR_INVALID_ARG     # f32 dy
    w.dtype, w.dw_stride = 0, 63
    assert L.gemm_rs_ckpt_wgrad(ctypes.byref(w), None, 0, None) == gr.ERR_INVALID_ARG
    w.dw_stride, w.dw = 64, 18
    assert L.gemm_rs_ckpt_wgrad(ctypes.byref(w), None, 0, None) == gr.ERR_MISALIGNED
    for code in (0, -1, -2, -3, -4, -5, -8, -99):
        assert L.gemm_rs_layer_strerror(code).decode()


def test_packed_argument_blocks_match_the_structures():
    for block, structure in ((layer._NORM_CONFIG, layer.gemm_rs_norm_config), (layer._NORM_ARGS, layer.gemm_rs_norm_args),
                             (layer._NORM_GRAD_ARGS, layer.gemm_rs_norm_grad_args),
                             (layer._WGRAD_ARGS, layer.gemm_rs_wgrad_args)):
        assert block.size == ctypes.sizeof(structure)
        n = len(block.unpack(bytes(block.size)))
        packed = structure.from_buffer_copy(block.pack(*range(1, n + 1)))
        values = []
        for name, _ in structure._fields_:
            v = getattr(packed, name)
            values += list(v) if isinstance(v, ctypes.Array) else [v]
        assert [int(v) for v in values] == list(range(1, n + 1))


def test_workspace_is_asked_for():
    size = layer.lib().gemm_rs_block_norm_workspace
    assert size(ctypes.byref(norm(post_norm=0)), 3) == 3 * 8192 * 4
    assert size(ctypes.byref(norm(gate=layer.GATE_CHANNEL)), 3) == 3 * 3 * 8192 * 4
    assert size(ctypes.byref(norm()), 0) == 0
    assert size(ctypes.byref(norm()), 1 << 20) <= 1 << 28


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        layer.ckpt_pack(x)
    with pytest.raises(TypeError):
        layer.ckpt_pack(x.to(torch.float64))
    with pytest.raises(ValueError):
        layer.block_norm(x)
    with pytest.raises(ValueError):
        layer.block_norm([x] * 9)
    with pytest.raises(TypeError):
        layer.w4_pack(torch.zeros(16, 32, dtype=torch.uint8), torch.ones(16, 1), group=64)
    with pytest.raises(layer.GemmRSLayerError) as e:
        layer.w4_pack(torch.zeros(16, 32, dtype=torch.uint8), torch.ones(16, 1, dtype=torch.float16), group=33)
    assert e.value.code == gr.ERR_UNSUPPORTED_SHAPE
