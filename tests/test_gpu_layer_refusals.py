"""GPU tests of what the layer operators' binding refuses so that no answer is silently wrong or lost."""
import pytest
import torch

from tensor_gemm_reduce_amd import layer

pytestmark = pytest.mark.gpu


def ones(*shape, dtype=torch.bfloat16):
    return torch.ones(shape, dtype=dtype, device="cuda")


def grad_calls():
    """name -> (call, its floating-point tensor arguments)"""
    weight = layer.w4_pack(ones(4, 16, dtype=torch.uint8), ones(4, 1), group=32)
    kept = layer.ckpt_pack(ones(2, 8))
    block = dict(pre_weight=ones(8), post_weight=ones(8))
    f32 = torch.float32
    return {
        "w4_pack": (lambda scales: layer.w4_pack(ones(4, 16, dtype=torch.uint8), scales, group=32), dict(scales=ones(4, 1))),
        "w4_linear": (lambda x, out: layer.w4_linear(x, weight, out), dict(x=ones(2, 32), out=ones(2, 4))),
        "block_norm": (lambda parts, residual, **kw: layer.block_norm(parts, residual, **kw),
                       dict(parts=ones(2, 8), residual=ones(2, 8), h=ones(2, 8), z=ones(2, 8), gate=ones(8), **block)),
        "block_norm of a list": (lambda part: layer.block_norm([ones(2, 8), part]), dict(part=ones(2, 8))),
        "block_norm of all parts": (lambda parts, gate: layer.block_norm(parts, gate=gate),
                                    dict(parts=ones(3, 2, 8), gate=ones(2, 1))),
        "block_norm_backward": (lambda **kw: layer.block_norm_backward(**kw),
                                dict(dz=ones(2, 8), dh=ones(2, 8), h=ones(2, 8), y=ones(2, 8), rstd=ones(2, 2, dtype=f32),
                                     gate=ones(2, 8), **block)),
        "ckpt_pack": (lambda x: layer.ckpt_pack(x), dict(x=ones(2, 8))),
        "ckpt_unpack": (lambda out: layer.ckpt_unpack(kept, out), dict(out=ones(2, 8))),
        "ckpt_wgrad": (lambda dy, add, out: layer.ckpt_wgrad(dy, kept, add=add, out=out),
                       dict(dy=ones(2, 4), add=ones(4, 8, dtype=f32), out=ones(4, 8, dtype=f32))),
    }


@pytest.mark.parametrize("name", ["w4_pack", "w4_linear", "block_norm", "block_norm of a list", "block_norm of all parts",
                                  "block_norm_backward", "ckpt_pack", "ckpt_unpack", "ckpt_wgrad"])
def test_gradients_are_not_lost_without_a_word(name):
    """The calls record no history for autograd: a tensor that asks for one is refused, unless gradients are off."""
    call, tensors = grad_calls()[name]
    call(**tensors)
    for which in tensors:
        asks = {k: v.clone().requires_grad_() if k == which else v for k, v in tensors.items()}
        with pytest.raises(RuntimeError, match="requires gradients"):
            call(**asks)
        for off in (torch.no_grad, torch.inference_mode):
            with off():
                call(**asks)


def test_inside_an_autograd_function():
    """Where gradients are off by themselves, and a linear layer's weight gradient comes from the checkpoint."""
    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            ctx.kept, ctx.w = layer.ckpt_pack(x), w
            return x @ w.t()

        @staticmethod
        def backward(ctx, dy):
            return dy @ ctx.w, layer.ckpt_wgrad(dy, ctx.kept, dtype=torch.bfloat16)

    x, w = ones(4, 64).requires_grad_(), ones(8, 64).requires_grad_()
    Linear.apply(x, w).backward(ones(4, 8))
    assert torch.equal(w.grad, torch.full_like(w, 4)) and torch.equal(x.grad, torch.full_like(x, 8))


@pytest.mark.parametrize("post", [False, True])
def test_backward_refuses_a_gradient_of_no_output(post):
    """Without a pre weight the forward pass has no z, so a gradient of it has nowhere to go."""
    t = ones(2, 8)
    kw = dict(post_weight=ones(8)) if post else {}
    rstd = ones(2, 2, dtype=torch.float32)
    with pytest.raises(ValueError, match="dz"):
        layer.block_norm_backward(t, t, None, t, rstd, **kw)
    assert torch.equal(layer.block_norm_backward(None, t, None, t, rstd, **kw).residual, t)
