"""One rank's row-parallel layer with everything around it, as a training step and as decode.

    python examples/layer_block.py [--workload tiny|o_proj|down_proj|mixtral_down] [--tokens T]

Training step on this rank's share of a TP=8 layer (the peers' partials are seeded stand-ins, as in the benchmark):

    kept        = the layer's input X_r in 8 bits                      ckpt_pack
    partials    = X_r W_r^T, routed to the ranks                       GemmRS (GEMM only: the sum is the next step's)
    y, h, z     = slice sum, post norm, gate, residual, pre norm       block_norm
    dY          = the gradient of the slice (all ranks' slices)        block_norm_backward
    main       += dY^T X_r                                             ckpt_wgrad

Decode: the same weights in 4 bits, a few tokens:

    partial     = x W4_r^T                                             w4_pack, w4_linear
    h, z        = sum with the peers' partials, norms, residual        block_norm

Prints how far each result is from a plain FP32 computation with the unquantised operands.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import synthetic  # noqa: E402
from tensor_gemm_reduce_amd import gemm_rs as gr  # noqa: E402
from tensor_gemm_reduce_amd import layer  # noqa: E402

GROUP = 128


def device_bf16(bits):
    return torch.from_numpy(bits.view("int16")).cuda().view(torch.bfloat16)


def quantise_4bit(w, group=GROUP):
    """Round-to-nearest 4-bit weights with a scale and zero point per `group` inputs: (q packed, scales, zeros)."""
    N, K = w.shape
    g = w.float().view(N, K // group, group)
    low, high = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    scale = ((high - low) / 15).clamp(min=1e-8).to(w.dtype)
    zero = torch.round(-low / scale.float()).clamp(0, 15)
    q = torch.round(g / scale.float().unsqueeze(-1) + zero.unsqueeze(-1)).clamp(0, 15).to(torch.uint8).view(N, K)
    return q[:, 0::2] | (q[:, 1::2] << 4), scale, zero.to(torch.uint8)


def far(got, want):
    """Relative distance in the 2-norm."""
    return float((got.float() - want).norm() / want.norm())


def rms(t):
    return torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-5)


class Block:
    """The layer's operands and the parameters around it on this rank."""

    def __init__(self, cfg, rank=0):
        self.cfg, self.rank = cfg, rank
        x, w, peers = synthetic.make_inputs(cfg, "balanced")
        self.x, self.w = device_bf16(x), device_bf16(w)
        self.peers = [device_bf16(p) for p in peers]
        gen = torch.Generator(device="cuda").manual_seed(synthetic.seed(cfg, 40))
        new = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        S, N = cfg.S, cfg.N
        self.post, self.pre = (1 + 0.1 * new(N)).bfloat16(), (1 + 0.1 * new(N)).bfloat16()
        self.gate = (0.5 + 0.1 * new(N)).bfloat16()
        self.residual = new(S, N)                       # the residual stream in 32 bits
        self.dz, self.dh = (0.1 * new(S, N)).bfloat16(), 0.1 * new(S, N)
        self.op = gr.GemmRS(cfg.M, N, cfg.K_local, rank=rank)
        self.send = [torch.empty((S, N), dtype=torch.bfloat16, device="cuda") for _ in range(7)]
        self.local = torch.empty((S, N), dtype=torch.bfloat16, device="cuda")
        self.out = torch.empty_like(self.local)

    def plain_norm(self, y, residual):
        u = y * rms(y) * self.post.float()
        h = residual + self.gate.float() * u
        return h, h * rms(h) * self.pre.float()

    def train(self, main):
        """One step; adds the weight gradient to `main` in place and returns the norm's outputs and the gradients."""
        kept = layer.ckpt_pack(self.x)
        self.op.run(gr.MODE_GEMM_ONLY, self.x, self.w, self.send, None, None, self.local)
        norm = layer.block_norm(self.peers + [self.local], self.residual, pre_weight=self.pre, post_weight=self.post,
                                gate=self.gate, save=True)
        grads = layer.block_norm_backward(self.dz, self.dh, norm.h, norm.y, norm.rstd, pre_weight=self.pre,
                                          post_weight=self.post, gate=self.gate)
        # the other ranks' slices of dY arrive by all-gather; here every slice is this rank's
        dy = grads.y.repeat(self.cfg.tp, 1)
        layer.ckpt_wgrad(dy, kept, add=main, out=main)
        return norm, grads, dy

    def decode(self, tokens, weight):
        """`tokens` rows through the 4-bit layer; every rank holds all rows, as after an all-reduce."""
        partial = layer.w4_linear(self.x[:tokens], weight)
        parts = [p[:tokens] for p in self.peers] + [partial]
        return partial, layer.block_norm(parts, self.residual[:tokens], pre_weight=self.pre, post_weight=self.post,
                                         gate=self.gate)


def run(cfg, tokens=4, verbose=True):
    """Runs both paths once; returns {what: relative distance from plain FP32}."""
    b = Block(cfg)
    tokens = min(tokens, cfg.S)
    main = torch.zeros((cfg.N, cfg.K_local), device="cuda")
    norm, grads, dy = b.train(main)
    # the fused layer's own slice sum is the same sum
    b.op.run(gr.MODE_FUSED, b.x, b.w, b.send, b.peers, b.out, b.local)
    torch.cuda.synchronize()
    if b.op.status() != gr.OK or not torch.equal(norm.y, b.out):
        raise RuntimeError("block_norm's slice sum differs from the fused layer's")
    y = sum(p.float() for p in b.peers) + b.local.float()
    h, z = b.plain_norm(y, b.residual)
    found = {"h": far(norm.h, h), "z": far(norm.z, z), "weight gradient (8-bit input)": far(main, dy.float().t() @ b.x.float())}

    group = GROUP if cfg.K_local % GROUP == 0 else cfg.K_local
    q, scales, zeros = quantise_4bit(b.w, group)
    weight = layer.w4_pack(q, scales, zeros, group=group)
    partial, dec = b.decode(tokens, weight)
    full = b.x[:tokens].float() @ b.w.float().t()
    h4, z4 = b.plain_norm(sum(p[:tokens].float() for p in b.peers) + partial.float(), b.residual[:tokens])
    found |= {"4-bit partial": far(partial, full), "decode h": far(dec.h, h4), "decode z": far(dec.z, z4)}
    b.op.close()
    if verbose:
        print(f"{cfg.name}: M={cfg.M} N={cfg.N} K_local={cfg.K_local}, {tokens} decoded token(s)")
        kept = layer.ckpt_pack(b.x)
        saved = b.x.numel() * 2 / (kept.q.numel() + kept.exps.numel())
        print(f"  checkpoint {saved:.2f}x smaller than bf16, 4-bit weights {b.w.numel() * 2 / weight.packed.numel():.2f}x")
        for k, v in found.items():
            print(f"  {k:32s} {v:.2e} from plain FP32")
    return found


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--workload", default="tiny", choices=[n for n in synthetic.CONFIGS if n != "large_prefill"])
    p.add_argument("--tokens", type=int, default=4)
    a = p.parse_args()
    run(synthetic.CONFIGS[a.workload], a.tokens)
