"""One rank's share of a layer of experts behind a router, as a training step and as decode.

    python examples/experts_block.py [--workload tiny|mixtral] [--tokens T] [--decode D]

Every rank of a tensor-parallel group holds 1 / 8 of each expert's inner width F, all tokens and the router:

    r         = the router's choice of k of E experts, weights, plan        route
    gu        = z W1_e^T for the rows of every expert                       experts_linear (gathers the tokens)
    a         = silu(gate) * up
    y         = a W2_e^T                                                    experts_linear (rows in the experts' order)
    partial   = sum over a token's rows of weight * row                     combine
    h, z'     = sum of the ranks' partials, residual, next norm             block_norm

and backward, in 8 bits too:

    dy, dw    = the rows' gradients and the weights'                        combine_backward
    da, dz    = dy W2_e, dgu W1_e, added up over a token's rows             experts_linear, combine
    dW1, dW2  = the experts' weights' gradients                             experts_wgrad
    dlogits   = the router's                                                route_backward

Prints how far each result is from a plain FP32 computation with the unquantised operands and the same choices.
"""
from __future__ import annotations

import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from tensor_gemm_reduce_amd import experts as ex  # noqa: E402
from tensor_gemm_reduce_amd import layer  # noqa: E402


@dataclasses.dataclass(frozen=True)
class Shape:
    hidden: int
    inner: int   # this rank's share of an expert's inner width
    experts: int
    chosen: int
    tokens: int


SHAPES = {
    "tiny": Shape(hidden=512, inner=128, experts=8, chosen=2, tokens=200),
    "mixtral": Shape(hidden=6144, inner=2048, experts=8, chosen=2, tokens=4096),  # Mixtral-8x22B-shaped, one rank of TP=8
}


def far(got, want):
    """Relative distance in the 2-norm."""
    return float((got.float() - want).norm() / want.norm())


class Experts:
    def __init__(self, s: Shape, tokens, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(20280000 + seed)
        new = lambda *shape, scale=1.0: (scale * torch.randn(shape, generator=gen, device="cuda")).bfloat16()  # noqa: E731
        H, F, E = s.hidden, s.inner, s.experts
        self.s, self.tokens = s, tokens
        self.z, self.dout = new(tokens, H), new(tokens, H, scale=0.1)
        self.residual = new(tokens, H).float()
        self.pre = (1 + 0.1 * new(H)).bfloat16()
        self.router = new(E, H, scale=H ** -0.5)
        self.bias = 0.02 * new(E).float()
        self.w1, self.w2 = new(E, 2 * F, H, scale=H ** -0.5), new(E, H, F, scale=F ** -0.5)
        # once: both products' weights, and transposed for the gradients of their inputs
        self.q1, self.q2 = ex.fp8_pack(self.w1), ex.fp8_pack(self.w2)
        self.q1t, self.q2t = ex.fp8_pack(self.w1, transpose=True), ex.fp8_pack(self.w2, transpose=True)

    def forward(self):
        logits = self.z.float() @ self.router.float().t()
        r = ex.route(logits, self.s.chosen, score="sigmoid", bias=self.bias)
        gu = ex.experts_linear(self.z, self.q1, r)
        gate, up = gu.float().chunk(2, 1)
        a = (torch.nn.functional.silu(gate) * up).bfloat16()
        y = ex.experts_linear(a, self.q2, r, rows=True)
        partial = ex.combine(y, r, r.weights)
        norm = layer.block_norm([partial], self.residual, pre_weight=self.pre)  # the other ranks' partials join here
        return logits, r, gu, a, y, partial, norm

    def backward(self, logits, r, gu, a, y):
        dy, dweights = ex.combine_backward(self.dout, y, r, r.weights)
        dlogits = ex.route_backward(dweights, logits, r.experts, score="sigmoid")
        da = ex.experts_linear(dy, self.q2t, r, rows=True).float()
        gate, up = gu.float().chunk(2, 1)
        s = torch.sigmoid(gate)
        dgu = torch.cat((da * up * (s + gate * s * (1 - s)), da * gate * s), 1).bfloat16()
        dz = ex.combine(ex.experts_linear(dgu, self.q1t, r, rows=True), r, None).float() + dlogits @ self.router.float()
        return {"dz": dz, "dW1": ex.experts_wgrad(dgu, self.z, r), "dW2": ex.experts_wgrad(dy, a, r, rows=True),
                "d router": dlogits.t() @ self.z.float()}

    def plain(self, experts):
        """The same in FP32 by autograd, with unquantised operands and given choices: (partial, gradients)."""
        z, w1, w2, router = (t.float().requires_grad_() for t in (self.z, self.w1, self.w2, self.router))
        chosen = torch.sigmoid(z @ router.t()).gather(1, experts.long())
        weights = chosen / (chosen.sum(1, keepdim=True) + 1e-20)
        out = torch.zeros_like(z)
        for e in range(self.s.experts):
            t, j = (experts == e).nonzero(as_tuple=True)
            gate, up = (z[t] @ w1[e].t()).chunk(2, 1)
            y = (torch.nn.functional.silu(gate) * up) @ w2[e].t()
            out = out.index_add(0, t, weights[t, j].unsqueeze(1) * y)
        out.backward(self.dout.float())
        return out.detach(), {"dz": z.grad, "dW1": w1.grad, "dW2": w2.grad, "d router": router.grad}


def run(shape, tokens=None, decode=4, verbose=True):
    """A training step and a decode step; returns {what: relative distance from plain FP32}."""
    m = Experts(shape, tokens or shape.tokens)
    logits, r, gu, a, y, partial, norm = m.forward()
    grads = m.backward(logits, r, gu, a, y)
    want, want_grads = m.plain(r.experts)
    h = m.residual + want
    found = {"partial": far(partial, want), "h": far(norm.h, h),
             "z": far(norm.z, h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-5) * m.pre.float())}
    found |= {k: far(grads[k], want_grads[k]) for k in want_grads}
    d = Experts(shape, decode, seed=1)
    _, r, _, _, _, partial, _ = d.forward()
    found["decode partial"] = far(partial, d.plain(r.experts)[0])
    if verbose:
        print(f"{shape.experts} experts, {shape.chosen} for each of {m.tokens} tokens, hidden {shape.hidden}, inner {shape.inner}; "
              f"{decode} decoded token(s)")
        print(f"  weights {m.w1.numel() * 2 / (m.q1.q.numel() + m.q1.scales.numel()):.2f}x smaller than bf16")
        for k, v in found.items():
            print(f"  {k:16s} {v:.2e} from plain FP32")
    return found


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--workload", default="tiny", choices=list(SHAPES))
    p.add_argument("--tokens", type=int, default=None)
    p.add_argument("--decode", type=int, default=4)
    args = p.parse_args()
    run(SHAPES[args.workload], args.tokens, args.decode)
