"""Host-side refusals of the experts' calls at the ends of their sizes (no GPU calls)."""
import ctypes

import pytest

from test_experts_host import fp8

ex = pytest.importorskip("tensor_gemm_reduce_amd.experts")
gr = pytest.importorskip("tensor_gemm_reduce_amd.gemm_rs")


def test_rows_without_any_input_are_refused():
    """Results of M rows from an x of none: there is nothing to take them from."""
    call = lambda **kw: ex.lib().gemm_rs_experts_linear(ctypes.byref(fp8(E=2, offsets=256, tokens=256, **kw)), None, 0, None)  # noqa: E731
    assert call(x_rows=0, M=4) == gr.ERR_INVALID_ARG
    assert call(x_rows=0, M=0) == gr.OK


def test_workspace_of_more_tokens_than_64_bits_count_choices_of():
    size = ex.lib().gemm_rs_expert_plan_workspace
    assert size((1 << 58) + 33, 8, 64) == 0   # T k wraps to 33 64
    assert size((1 << 62) + 1000, 8, 4) == 0
