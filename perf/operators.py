"""The operators around the row-parallel layer: their cases, plain forms and 64-bit definitions.

Five calls, each one pass of a user's program (H: hidden width, K: this rank's share of the reduction
dimension, tokens: rows of the activations):

  w4       y = x w^T with 4-bit weights, w[n][k] = scale[n][k / group] (q[n][k] - zero[n][k / group])
  norm     u = rms(sum of the partials) post_weight, h = rscale residual + bscale gate u, z = rms(h) pre_weight
  normbwd  the gradients of norm
  ckpt     an activation kept in 8 bits (blocks of 32 with a power-of-two scale) and read back
  wgrad    dw = dy^T x^ (+ main) with x^ the activation kept in 8 bits

Sizes are those of the benchmark's configurations (synthetic.CONFIGS, AG_CONFIGS: hidden widths 8192 and 6144,
reduction shares 1024, 2048, 3584, slices of 64 to 4096 rows) and generic odd ones.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5
BLOCK = 32  # elements of a row that share one 8-bit checkpoint scale


def listed():
    return [
        # one decoded token through the o_proj shard of a 70B model: the smallest product, where latency counts
        {"name": "w4 o_proj 1 token", "op": "w4", "M": 1, "N": 8192, "K": 1024, "group": 128, "zeros": False, "type": "bf16"},
        # a decode batch through the gate/up shard (column-parallel, the whole hidden width as K), scales and zero points
        # every 64 weights
        {"name": "w4 gate_up 24 tokens", "op": "w4", "M": 24, "N": 7168, "K": 8192, "group": 64, "zeros": True, "type": "f16"},
        # one prompt chunk through a Mixtral-shaped expert's down projection: enough rows for the product to matter
        {"name": "w4 mixtral_down 500 tokens", "op": "w4", "M": 500, "N": 6144, "K": 2048, "group": 32, "zeros": False, "type": "bf16"},
        # after an all-reduce of one decoded token: eight partials, residual and the next norm
        {"name": "norm decode 1 row", "op": "norm", "S": 1, "N": 8192, "parts": 8, "post": False, "gate": "none", "type": "bf16", "residual": "bf16", "save": False},
        # a ragged batch behind a norm on both sides and a learned gate for each channel
        {"name": "norm sandwich 1021 rows", "op": "norm", "S": 1021, "N": 6144, "parts": 1, "post": True, "gate": "channel", "type": "f16", "residual": "f16", "save": False},
        # training on the large prefill's slice: eight partials, a residual stream in 32 bits, statistics kept
        {"name": "norm train 4096 rows", "op": "norm", "S": 4096, "N": 8192, "parts": 8, "post": True, "gate": "channel", "type": "bf16", "residual": "f32", "save": True},
        # the backward pass on o_proj's slice: few rows, so the sums over rows and the launches count
        {"name": "normbwd 64 rows", "op": "normbwd", "S": 64, "N": 8192, "post": False, "gate": "none", "type": "bf16", "residual": "bf16"},
        # the backward pass of the large prefill's slice with everything on
        {"name": "normbwd 4096 rows", "op": "normbwd", "S": 4096, "N": 8192, "post": True, "gate": "channel", "type": "bf16", "residual": "f32"},
        # an activation kept for the backward pass: a ragged one, and the large prefill's
        {"name": "ckpt 777x1000", "op": "ckpt", "M": 777, "K": 1000, "type": "f16"},
        {"name": "ckpt large_prefill", "op": "ckpt", "M": 32768, "K": 3584, "type": "bf16"},
        # the weight gradient of o_proj's shard, and of the large prefill's onto the running sum of the micro-batches
        {"name": "wgrad o_proj", "op": "wgrad", "M": 512, "N": 8192, "K": 1024, "main": False, "out": "bf16", "type": "bf16"},
        {"name": "wgrad large_prefill", "op": "wgrad", "M": 32768, "N": 8192, "K": 3584, "main": True, "out": "f32", "type": "bf16"},
    ]


def _size(rng, low, high, unit=1):
    """A size between low and high, even over the logarithm; half of them an odd multiple of `unit`, half any multiple of 8
    (or of `unit`, if larger)."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    if rng.random() < 0.5:
        v = unit * (2 * int(v / (2 * unit)) + 1)
    else:
        step = 8 * (unit // 8 or 1)
        v = step * (2 * int(v / (2 * step)) + 1)
    return max(unit, min(int(v), high - high % unit))


def draw(rng):
    op = rng.choice(("w4", "w4", "norm", "normbwd", "ckpt", "wgrad"))
    half = rng.choice(("bf16", "bf16", "f16"))
    if op == "w4":
        group = rng.choice((32, 64, 128))
        return {"op": op, "M": _size(rng, 1, 512), "N": _size(rng, 256, 16384), "K": _size(rng, 256, 8192, group),
                "group": group, "zeros": rng.random() < 0.5, "type": half}
    if op in ("norm", "normbwd"):
        c = {"op": op, "S": _size(rng, 1, 4096), "N": _size(rng, 256, 8192), "post": rng.random() < 0.5,
             "gate": rng.choice(("none", "channel", "token", "full")), "type": half, "residual": rng.choice((half, "f32"))}
        return c if op == "normbwd" else dict(c, parts=rng.choice((1, 2, 8)), save=rng.random() < 0.5)
    if op == "ckpt":
        return {"op": op, "M": _size(rng, 1, 32768), "K": _size(rng, 64, 3584), "type": rng.choice((half, "f32"))}
    return {"op": op, "M": _size(rng, 1, 16384), "N": _size(rng, 256, 8192, 8), "K": _size(rng, 128, 3584, 8),
            "main": rng.random() < 0.5, "out": rng.choice(("f32", half)), "type": half}


# ---- what a user's program has in hand before the call ----------------------------------------------------------

def _normal(gen, shape, kind, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(TYPES[kind])


def _activation(gen, rows, width, kind):
    """Activations as layers see them: every channel has its own spread, a few far above the rest."""
    spread = torch.exp(0.8 * torch.randn(width, generator=gen, device="cuda"))
    x = torch.randn((rows, width), generator=gen, device="cuda")
    return x.mul_(spread).to(TYPES[kind])


def _weight(gen, width, kind):
    return (1.0 + 0.1 * torch.randn(width, generator=gen, device="cuda")).to(TYPES[kind])


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(20260000 + seed)
    s = {"case": case}
    op = case["op"]
    if op == "w4":
        M, N, K, G = case["M"], case["N"], case["K"], case["group"]
        s["x"] = _normal(gen, (M, K), case["type"])
        q = torch.randn((N, K), generator=gen, device="cuda").mul_(2.6).add_(7.5).round_().clamp_(0, 15).to(torch.uint8)
        s["q"] = q[:, 0::2] | (q[:, 1::2] << 4)   # [N][K / 2], the even column in the low half of its byte
        s["scale"] = (torch.rand((N, K // G), generator=gen, device="cuda").add_(0.5) / (3 * math.sqrt(K))).to(TYPES[case["type"]])
        s["zero"] = torch.randint(6, 11, (N, K // G), generator=gen, device="cuda", dtype=torch.uint8) if case["zeros"] else None
    elif op in ("norm", "normbwd"):
        S, N, kind, rkind = case["S"], case["N"], case["type"], case["residual"]
        s["pre"] = _weight(gen, N, kind)
        s["post"] = _weight(gen, N, kind) if case["post"] else None
        shape = {"none": None, "channel": (N,), "token": (S, 1), "full": (S, N)}[case["gate"]]
        s["gate"] = _normal(gen, shape, kind, 0.5) if shape else None
        if op == "norm":
            s["parts"] = _normal(gen, (case["parts"], S, N), kind, 0.4)
            s["residual"] = _normal(gen, (S, N), rkind)
        else:
            y = _normal(gen, (S, N), kind, 0.4)
            h = _normal(gen, (S, N), rkind, 1.2)
            s["y"], s["h"] = y, h
            # what the forward pass kept of its statistics: 1 / rms of y and of h
            s["rstd"] = torch.stack([torch.rsqrt(t.float().square().mean(1) + EPS) for t in (y, h)])
            s["dz"] = _normal(gen, (S, N), kind, 0.1)
            s["dh"] = _normal(gen, (S, N), rkind, 0.1)
    elif op == "ckpt":
        s["x"] = _activation(gen, case["M"], case["K"], case["type"])
    else:
        M, N, K = case["M"], case["N"], case["K"]
        s["dy"] = _normal(gen, (M, N), case["type"], 1 / math.sqrt(M))
        s["q"], s["exp"] = _keep(_activation(gen, M, K, case["type"]))
        s["main"] = _normal(gen, (N, K), "f32") if case["main"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] == "w4":  # a serving program lays its weights out once, when it loads them
        from tensor_gemm_reduce_amd import layer

        s["weight"] = layer.w4_pack(s.pop("q"), s.pop("scale"), s.pop("zero"), group=case["group"])
    return s


# ---- one pass ------------------------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, c):
    from tensor_gemm_reduce_amd import layer

    op = c["op"]
    if op == "w4":
        return layer.w4_linear(s["x"], s["weight"])
    if op == "norm":
        out = layer.block_norm(s["parts"], s["residual"], pre_weight=s["pre"], post_weight=s["post"], gate=s["gate"],
                               block_scale=0.7, residual_scale=0.9, eps=EPS, save=c["save"])
        return {"h": out.h, "z": out.z, "y": out.y, "rstd": out.rstd} if c["save"] else {"h": out.h, "z": out.z}
    if op == "normbwd":
        g = layer.block_norm_backward(s["dz"], s["dh"], s["h"], s["y"], s["rstd"], pre_weight=s["pre"], post_weight=s["post"],
                                      gate=s["gate"], block_scale=0.7, residual_scale=0.9)
        return _named(g.residual, g.y, g.pre_weight, g.post_weight, g.gate)
    if op == "ckpt":
        return layer.ckpt_unpack(layer.ckpt_pack(s["x"]))
    kept = layer.Checkpoint(s["q"], s["exp"], c["K"], TYPES[c["type"]])
    return layer.ckpt_wgrad(s["dy"], kept, add=s["main"], dtype=TYPES[c["out"]])


def _run_plain(s, c):
    op = c["op"]
    if op == "w4":
        return _w4(s, c)
    if op == "norm":
        return _norm(s, c)
    if op == "normbwd":
        return _normbwd(s, c)
    if op == "ckpt":
        q, e = _keep(s["x"])
        return _value(q, e, c["K"]).to(TYPES[c["type"]])
    dw = s["dy"].float().t() @ _value(s["q"], s["exp"], c["K"])
    return (dw if s["main"] is None else s["main"] + dw).to(TYPES[c["out"]])


def _named(residual, y, pre, post, gate):
    g = {"residual": residual, "y": y, "pre_weight": pre, "post_weight": post, "gate": gate}
    return {k: v for k, v in g.items() if v is not None}


# ---- plain forms, in 32 bits, rounded once at the end --------------------------------------------------------------

def _w4(s, c):
    N, K, G = c["N"], c["K"], c["group"]
    q = torch.stack((s["q"] & 15, s["q"] >> 4), dim=-1).view(N, K // G, G).float()
    zero = 8.0 if s["zero"] is None else s["zero"].float().unsqueeze(-1)
    w = ((q - zero) * s["scale"].float().unsqueeze(-1)).view(N, K)
    return (s["x"].float() @ w.t()).to(s["x"].dtype)


def _norm(s, c):
    y = s["parts"].float().sum(0)
    ry = torch.rsqrt(y.square().mean(1, keepdim=True) + EPS)
    u = y * ry * s["post"].float() if c["post"] else y
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = 0.9 * s["residual"].float() + 0.7 * u
    rh = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    out = {"h": h.to(TYPES[c["residual"]]), "z": (h * rh * s["pre"].float()).to(TYPES[c["type"]])}
    if c["save"]:
        out["y"] = y.to(TYPES[c["type"]])
        out["rstd"] = torch.stack((ry.squeeze(1) if c["post"] else torch.ones_like(ry).squeeze(1), rh.squeeze(1)))
    return out


def _normbwd(s, c):
    kind = TYPES[c["type"]]
    ry, rh = s["rstd"][0].unsqueeze(1), s["rstd"][1].unsqueeze(1)
    hh = s["h"].float() * rh
    dz = s["dz"].float()
    wdz = dz * s["pre"].float()
    dh = s["dh"].float() + rh * (wdz - hh * (wdz * hh).mean(1, keepdim=True))
    dpre = (dz * hh).sum(0)
    y = s["y"].float()
    yy = y * ry if c["post"] else y
    u = yy * s["post"].float() if c["post"] else yy
    du = 0.7 * dh
    dgate = None
    if s["gate"] is not None:
        dgate = du * u
        dgate = dgate.sum(0) if c["gate"] == "channel" else dgate.sum(1, keepdim=True).to(kind) if c["gate"] == "token" else dgate.to(kind)
        du = du * s["gate"].float()
    dpost = None
    if c["post"]:
        dpost = (du * yy).sum(0)
        wdu = du * s["post"].float()
        du = ry * (wdu - yy * (wdu * yy).mean(1, keepdim=True))
    return _named((0.9 * dh).to(TYPES[c["residual"]]), du.to(kind), dpre, dpost, dgate)


def _keep(x):
    """An activation in 8 bits: blocks of 32 columns share the scale 2^e with e = floor(log2(max |x|)) - 6 (at least -126),
    and hold round(x 2^-e) limited to -127 .. 127.  Rows are padded with zeros to whole blocks."""
    M, K = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -K % BLOCK)).view(M, -1, BLOCK)
    e = (torch.frexp(v.abs().amax(-1))[1] - 7).clamp(min=-126)
    e = torch.where(v.abs().amax(-1) == 0, torch.full_like(e, -126), e)
    q = (v * _power(-e.unsqueeze(-1))).round().clamp(-127, 127)
    return q.to(torch.int8).view(M, -1), e.to(torch.int8)


def _value(q, e, K):
    M = q.shape[0]
    v = q.view(M, -1, BLOCK).float() * _power(e.unsqueeze(-1))
    return v.view(M, -1)[:, :K]


def _power(e):
    """2^e exactly, from its exponent bits (a library power may be an ulp off, which would turn ties)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    if work(case)["flops"] > 3e13:
        return None  # over 20 seconds in 64 bits
    s = _inputs(case, seed)
    op = case["op"]
    if op == "w4":
        rows = s["q"].to(torch.int64)
        w = torch.empty((case["N"], case["K"]), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (rows % 16).double(), (rows // 16).double()
        per_weight = lambda t: t.double().repeat_interleave(case["group"], dim=1)  # noqa: E731
        w = per_weight(s["scale"]) * (w - (8 if s["zero"] is None else per_weight(s["zero"])))
        return torch.matmul(s["x"].double(), w.transpose(0, 1).contiguous())
    if op == "norm":
        return _exact_norm(case, s)
    if op == "normbwd":
        return _exact_normbwd(case, s)
    if op == "ckpt":
        return _exact_ckpt(s["x"])
    scale = _exact_power(s["exp"].long())
    kept = (s["q"].double() * scale.repeat_interleave(BLOCK, dim=1))[:, :case["K"]]
    dw = torch.matmul(s["dy"].double().transpose(0, 1).contiguous(), kept)
    return dw if s["main"] is None else dw + s["main"].double()


def _double(s, *names):
    return [None if s.get(n) is None else s[n].double() for n in names]


def _exact_norm(c, s):
    parts, residual, pre, post, gate = _double(s, "parts", "residual", "pre", "post", "gate")
    y = parts.sum(dim=0)
    inv = lambda t: 1.0 / torch.sqrt((t * t).sum(dim=1) / c["N"] + EPS)  # noqa: E731
    block = y
    if post is not None:
        block = torch.einsum("sn,s,n->sn", y, inv(y), post)
    if gate is not None:
        block = block * gate
    h = residual * 0.9 + block * 0.7
    out = {"h": h, "z": torch.einsum("sn,s,n->sn", h, inv(h), pre)}
    if c["save"]:
        out["y"] = y
        out["rstd"] = torch.stack((inv(y) if post is not None else torch.ones_like(inv(y)), inv(h)))
    return out


def _exact_normbwd(c, s):
    """Each norm n = t w / rms(t): dt_i = r w_i d_i - r^3 t_i sum_j(w_j d_j t_j) / N, with r as the forward pass kept it."""
    dz, dh, h, y, rstd, pre, post, gate = _double(s, "dz", "dh", "h", "y", "rstd", "pre", "post", "gate")
    N = c["N"]

    def through(d, t, w, r):
        r = r[:, None]
        dot = (d * t) @ w
        return r * d * w - (r ** 3) * t * (dot / N)[:, None], (d * t * r).sum(dim=0)

    dt, dpre = through(dz, h, pre, rstd[1])
    total = dt + dh
    u = y if post is None else y * rstd[0][:, None] * post
    dblock = total * 0.7
    dgate = None
    if gate is not None:
        dgate = dblock * u
        if c["gate"] == "channel":
            dgate = dgate.sum(dim=0)
        elif c["gate"] == "token":
            dgate = dgate.sum(dim=1, keepdim=True)
        dblock = dblock * gate
    dpost = None
    if post is not None:
        dblock, dpost = through(dblock, y, post, rstd[0])
    return _named(total * 0.9, dblock, dpre, dpost, dgate)


def _exact_ckpt(x):
    M, K = x.shape
    out = torch.zeros((M, -(-K // BLOCK) * BLOCK), dtype=torch.float64, device=x.device)
    out[:, :K] = x
    blocks = out.view(M, -1, BLOCK)
    top = blocks.abs().max(dim=2, keepdim=True).values
    # the power of two at or below the largest value, from the exponent bits of its 64-bit form
    power = (top.view(torch.int64) >> 52) - 1023
    step = _exact_power(torch.clamp(power - 6, min=-126))
    return (torch.clamp(torch.round(blocks / step), -127, 127) * step).reshape(M, -1)[:, :K].contiguous()


def _exact_power(n):
    return torch.bitwise_left_shift(n + 1023, 52).view(torch.float64)


# ---- what a pass cannot do without ------------------------------------------------------------------------------------

def work(case):
    op = case["op"]
    b = BYTES[case["type"]]
    if op == "w4":
        M, N, K, G = case["M"], case["N"], case["K"], case["group"]
        weight = N * K // 2 + N * (K // G) * (b + (1 if case["zeros"] else 0))
        return {"bytes": weight + (M * K + M * N) * b, "flops": 2 * M * N * K}
    if op in ("norm", "normbwd"):
        S, N, r = case["S"], case["N"], BYTES[case["residual"]]
        gate = {"none": 0, "channel": N, "token": S, "full": S * N}[case["gate"]]
        weights = (2 if case["post"] else 1) * N
        if op == "norm":
            moved = case["parts"] * S * N * b + 2 * S * N * r + S * N * b + (weights + gate) * b
            if case["save"]:
                moved += S * N * b + 8 * S
            return {"bytes": moved, "flops": (case["parts"] + 9) * S * N}
        # y is read where a post norm or a gate needs it, else only its gradient is written
        needs_y = case["post"] or case["gate"] != "none"
        moved = S * N * (2 * b + 3 * r + (b if needs_y else 0)) + 8 * S + (weights + gate) * b
        moved += 4 * weights + gate * (4 if case["gate"] == "channel" else b)
        return {"bytes": moved, "flops": 20 * S * N}
    if op == "ckpt":
        M, K = case["M"], case["K"]
        blocks = -(-K // BLOCK)
        return {"bytes": 2 * M * K * b + 2 * M * blocks * (BLOCK + 1), "flops": 4 * M * K}
    M, N, K = case["M"], case["N"], case["K"]
    out = N * K * (BYTES[case["out"]] + (4 if case["main"] else 0))
    return {"bytes": M * N * b + M * -(-K // BLOCK) * (BLOCK + 1) + out, "flops": 2 * M * N * K}
