"""CPU tests of what the layer operators' binding refuses before it touches a device."""
import pytest
import torch

layer = pytest.importorskip("tensor_gemm_reduce_amd.layer")
gr = pytest.importorskip("tensor_gemm_reduce_amd.gemm_rs")


@pytest.mark.parametrize("N,half,group", [(16, 64, (1 << 32) + 128), (16, 64, 128 - (1 << 32)), (1, (1 << 31) + 64, 128),
                                          ((1 << 32) + 16, 64, 128), (1, 1 << 30, 1 << 31)])
def test_w4_pack_refuses_sizes_past_31_bits(N, half, group):
    """Sizes whose low 32 bits alone would be a valid configuration."""
    q = torch.zeros((1, 1), dtype=torch.uint8).expand(N, half)
    scales = torch.ones((1, 1), dtype=torch.bfloat16).expand(N, 1)
    with pytest.raises(layer.GemmRSLayerError) as e:
        layer.w4_pack(q, scales, group=group)
    assert e.value.code in (gr.ERR_UNSUPPORTED_SHAPE, gr.ERR_INVALID_ARG)


def test_backward_refuses_a_gradient_of_no_output():
    """Without a pre weight the forward pass has no z, so a gradient of it has nowhere to go."""
    t = torch.ones(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="dz: needs a pre_weight"):
        layer.block_norm_backward(t, t, None, None, None)
