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
