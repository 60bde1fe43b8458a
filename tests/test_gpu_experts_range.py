"""GPU tests of the experts' operators at the ends of their ranges: buffers of exactly the stated sizes."""
import pytest
import torch

from tensor_gemm_reduce_amd import experts as ex
from test_gpu_experts import gen

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
