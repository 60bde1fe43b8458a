"""Host-side checks of how the weight gradient's work is cut, and of the workspace that takes."""
import ctypes

import pytest

layer = pytest.importorskip("tensor_gemm_reduce_amd.layer")


def wgrad_args(M, N, K, dtype=layer.DTYPE_BF16, out=layer.DTYPE_F32):
    """Arguments of contiguous buffers (never touched by the calls here)."""
    return layer.gemm_rs_wgrad_args(dtype, out, M, N, K, 16, N, 16, 16, None, 0, 16, K)


def workspace(M, N, K):
    return layer.lib().gemm_rs_ckpt_wgrad_workspace(ctypes.byref(wgrad_args(M, N, K)))


@pytest.mark.parametrize("M,N,K,edge,shares,cut", [
    (16384, 512, 256, 128, 256, 8), (4096, 8192, 1024, 256, 256, 128), (32768, 8192, 3584, 256, 256, 192),
    (4100, 300, 200, 128, 48, 6)])
def test_workspace_holds_a_piece_per_share_and_cut_tile(M, N, K, edge, shares, cut):
    """A share begins a piece, and so does a tile within it: no more pieces than shares and cut tiles."""
    assert workspace(M, N, K) % (edge * edge * 4) == 0
    assert shares < workspace(M, N, K) // (edge * edge * 4) <= shares + cut


# One product for every way the work is cut, by what the second kernel, the last round and the order of shares see:
# (M, N, K) and the plan it gets.
WGRAD_PLANS = [
    # by elements: odd N
    ((300, 777, 520), dict(words=0, tile=128, whole=35, workgroups=35)),
    # tiles of 128 x 128: fewer than workgroups; a last round left whole; cut, joined by one wave and by four; a whole
    # round and a cut rest
    ((300, 776, 520), dict(words=1, tile=128, whole=35, workgroups=35)),
    ((128, 4096, 2100), dict(words=1, tile=128, whole=544, workgroups=512)),
    ((1000, 300, 200), dict(words=1, tile=128, cut=6, shares=12, workgroups=12, join_waves=1)),
    ((4100, 300, 200), dict(words=1, tile=128, cut=6, shares=48, workgroups=48, join_waves=4)),
    ((1100, 8000, 1100), dict(words=1, tile=128, whole=512, cut=55, shares=123, workgroups=512, dealt=1, join_waves=1)),
    # tiles of 256 x 256: the same, and shares of their own dealt over the XCDs
    ((3000, 4096, 2100), dict(words=1, tile=256, whole=144, workgroups=144)),
    ((3000, 8192, 3584), dict(words=1, tile=256, whole=448, workgroups=256)),
    ((4100, 4040, 1030), dict(words=1, tile=256, cut=80, shares=256, workgroups=256, join_waves=1)),
    ((12300, 1030, 1000), dict(words=1, tile=256, cut=20, shares=256, workgroups=256, join_waves=4)),
    ((6300, 2050, 3500), dict(words=1, tile=256, cut=126, shares=256, workgroups=256, dealt=1, join_waves=1)),
    ((2840, 4104, 4130), dict(words=1, tile=256, whole=256, cut=33, shares=128, workgroups=256, dealt=1, join_waves=1)),
]


def plan(*shape, **kw):
    info = layer.gemm_rs_wgrad_info()
    assert layer.lib().gemm_rs_ckpt_wgrad_plan(ctypes.byref(wgrad_args(*shape, **kw)), ctypes.byref(info)) == 0
    return {n: getattr(info, n) for n, _ in info._fields_}


@pytest.mark.parametrize("shape,want", WGRAD_PLANS)
def test_plan_of_every_tested_product(shape, want):
    """If this fails after a change of the plan, the sizes that reach each path have moved, and with them what is tested."""
    full = dict(dict.fromkeys(("words", "tile", "whole", "cut", "shares", "workgroups", "dealt", "join_waves"), 0), **want)
    for dtype in (layer.DTYPE_BF16, layer.DTYPE_F16):
        assert plan(*shape, dtype=dtype, out=dtype) == full


def test_plan_covers_every_tile_once():
    for M in (1, 64, 700, 2816, 2817, 20000):
        for N in (2, 100, 2000, 9000):
            for K in (1, 300, 4000):
                p = plan(M, N, K)
                tiles = -(-N // p["tile"]) * -(-K // p["tile"])
                assert p["whole"] + p["cut"] == tiles and 1 <= p["workgroups"] <= 512
                assert (p["shares"] > p["cut"] > 0) == (p["join_waves"] > 0) == (workspace(M, N, K) > 0)


def test_plan_refuses_what_the_call_refuses():
    L = layer.lib()
    info = layer.gemm_rs_wgrad_info()
    bad = wgrad_args(8, 64, 64, dtype=layer.DTYPE_F32)
    assert L.gemm_rs_ckpt_wgrad_plan(ctypes.byref(bad), ctypes.byref(info)) == layer.ERR_INVALID_ARG
    assert L.gemm_rs_ckpt_wgrad_plan(ctypes.byref(wgrad_args(8, 1 << 23, 64)), ctypes.byref(info)) == layer.ERR_UNSUPPORTED_SHAPE
    assert L.gemm_rs_ckpt_wgrad_plan(ctypes.byref(wgrad_args(8, 64, 64)), None) == layer.ERR_INVALID_ARG
    assert L.gemm_rs_ckpt_wgrad_plan(None, ctypes.byref(info)) == layer.ERR_INVALID_ARG
