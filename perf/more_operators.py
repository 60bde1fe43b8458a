"""The router, the experts' products and the 8-bit floating-point product: their cases, plain forms and 64-bit definitions.

Four operators, each in its forward and its backward direction (T tokens, E experts, k of them for a token, R = T k rows
in the order of the experts; K inputs, N outputs):

  route     scores of the experts (softmax or sigmoid of the logits), the choice of k by score + bias inside the best
            groups, renormalised weights, and the plan: the rows of every expert in the order of the tokens;
            backward: the logits' gradient from the weights'
  fp8       y = x^ w^^T, x^ and w^ in e4m3 with a power-of-two scale for each block of 128 inputs (x: of a row; w: of 128
            rows); backward: dx = dy^ w^, and dw = dy^^T x^ with both in blocks of 128 tokens
  experts   the same for every row with its expert's weights; the rows come by token, or are in the experts' order;
            backward: the rows' gradients and dw of every expert
  combine   out[t] = sum_j weight[t][j] y[row of (t, j)]; backward: dy and the weights' gradient

Sizes are those of the benchmark's configurations (synthetic.CONFIGS, AG_CONFIGS: hidden widths 8192 and 6144, shares of
1024, 2048 and 3584 inputs, 8192 and 7168 outputs; a Mixtral-shaped expert: 8 of them, 2 for a token) and generic ones.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
BLOCK = 128   # inputs that share a scale; also a weight's rows that do
TOP = 448.0   # the largest e4m3 value


def listed():
    return [
        # one decoded token through a router of eight experts: the smallest call, where latency counts
        {"name": "route decode 1 token", "op": "route", "pass": "forward", "T": 1, "E": 8, "k": 2, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "renorm": True, "pad": 0, "type": "bf16"},
        # a prompt batch through many small experts: sigmoid scores, a bias for balance, 4 of 8 groups; the last rows are padding
        {"name": "route prefill 8192 tokens", "op": "route", "pass": "forward", "T": 8192, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "keep": 4, "renorm": True, "pad": 37, "type": "f32"},
        # training the router: a ragged batch, 6 of 64 experts, softmax scores
        {"name": "route backward 8191 tokens", "op": "route", "pass": "backward", "T": 8191, "E": 64, "k": 6, "score": "softmax",
         "bias": False, "groups": 1, "keep": 1, "renorm": True, "pad": 0, "type": "bf16"},
        # one decoded token through the o_proj shard of a 70B model
        {"name": "fp8 o_proj 1 token", "op": "fp8", "pass": "forward", "M": 1, "N": 8192, "K": 1024, "type": "bf16"},
        # a ragged prompt chunk through the gate/up shard (column-parallel, the whole hidden width as K)
        {"name": "fp8 gate_up 501 tokens", "op": "fp8", "pass": "forward", "M": 501, "N": 7168, "K": 8192, "type": "f16"},
        # the large prefill's down projection: the matrix instructions' rate
        {"name": "fp8 large_prefill", "op": "fp8", "pass": "forward", "M": 32768, "N": 8192, "K": 3584, "type": "bf16"},
        # the backward pass of the down projection: both gradients
        {"name": "fp8 backward down_proj", "op": "fp8", "pass": "backward", "M": 2048, "N": 8192, "K": 3584, "type": "bf16"},
        # a decode batch through the gate and up projections of eight experts: the weights' bytes count
        {"name": "experts decode 16 tokens", "op": "experts", "pass": "forward", "T": 16, "E": 8, "k": 2, "N": 4096, "K": 6144,
         "rows": False, "type": "bf16"},
        # a prompt through eight experts' down projection, rows already in the experts' order
        {"name": "experts mixtral_down 8192 tokens", "op": "experts", "pass": "forward", "T": 8192, "E": 8, "k": 2, "N": 6144,
         "K": 2048, "rows": True, "type": "bf16"},
        # training many small experts: ragged numbers of rows, gradients of the rows and of every expert's weights
        {"name": "experts backward 4095 tokens", "op": "experts", "pass": "backward", "T": 4095, "E": 64, "k": 6, "N": 1408,
         "K": 2048, "rows": False, "type": "bf16"},
        # a decode batch's rows back to its tokens
        {"name": "combine decode 24 tokens", "op": "combine", "pass": "forward", "T": 24, "k": 8, "N": 8192, "type": "bf16"},
        # the backward pass of a prompt's, two rows for a token
        {"name": "combine backward 8192 tokens", "op": "combine", "pass": "backward", "T": 8192, "k": 2, "N": 6144, "type": "bf16"},
    ]


def _size(rng, low, high):
    """A size between low and high, even over the logarithm; half of them odd, half a multiple of 8 where there is room."""
    v = int(math.exp(rng.uniform(math.log(low), math.log(high))))
    v = v | 1 if rng.random() < 0.5 or v < 16 else v // 8 * 8
    return max(low, min(v, high))


def draw(rng):
    op = rng.choice(("route", "fp8", "fp8", "experts", "experts", "combine"))
    half = rng.choice(("bf16", "bf16", "f16"))
    back = rng.random() < 0.35
    c = {"op": op, "pass": "backward" if back else "forward"}
    if op == "route":
        E = rng.choice((5, 8, 16, 60, 64, 100, 128, 160, 256))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0 and E // g >= 2])
        keep = rng.randint(1, groups)
        T = _size(rng, 1, 8192)
        score = rng.choice(("softmax", "sigmoid"))
        return dict(c, T=T, E=E, k=rng.randint(1, min(8, keep * (E // groups))), score=score, bias=rng.random() < 0.5, groups=groups,
                    keep=keep, renorm=rng.random() < 0.7, pad=rng.choice((0, T // 9)), type=rng.choice((half, "f32")))
    if op == "fp8":
        return dict(c, M=_size(rng, 1, 4096 if back else 8192), N=_size(rng, 256, 8192), K=_size(rng, 128, 8192), type=half)
    if op == "experts":
        E = rng.choice((4, 8, 16, 64))
        return dict(c, T=_size(rng, 1, 4096), E=E, k=rng.randint(1, min(6, E)), N=_size(rng, 256, 4096), K=_size(rng, 256, 4096),
                    rows=False if back else rng.random() < 0.5, type=half)
    return dict(c, T=_size(rng, 1, 8192), k=rng.randint(1, 8), N=_size(rng, 256, 8192), type=half)


# ---- what a user's program has in hand before the call ----------------------------------------------------------

def _normal(gen, shape, kind, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(TYPES[kind])


def _activation(gen, rows, width, kind):
    """Activations as layers see them: every channel has its own spread, a few far above the rest."""
    spread = torch.exp(0.8 * torch.randn(width, generator=gen, device="cuda"))
    return torch.randn((rows, width), generator=gen, device="cuda").mul_(spread).to(TYPES[kind])


def _choice(gen, T, E, k):
    """k different experts for each token, some of them more popular than others."""
    liked = 0.7 * torch.randn(E, generator=gen, device="cuda")
    s = torch.randn((T, E), generator=gen, device="cuda") + liked
    return s.argsort(dim=1, descending=True)[:, :k].to(torch.int32).contiguous()


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(20270000 + seed)
    s = {"case": case}
    op, back = case["op"], case["pass"] == "backward"
    if op == "route":
        T, E = case["T"], case["E"]
        logits = torch.randn((T, E), generator=gen, device="cuda").mul_(1.5)
        if case["pad"]:
            logits[T - case["pad"]:] = -math.inf  # padding: no expert is on
        s["logits"] = logits.to(TYPES[case["type"]])
        s["bias"] = 0.05 * torch.randn(E, generator=gen, device="cuda") if case["bias"] else None
        if back:
            s["experts"] = _choice_of(s["logits"], s["bias"], case)[0]
            s["dweights"] = torch.randn((T, case["k"]), generator=gen, device="cuda")
    elif op == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        s["x"] = _activation(gen, M, K, case["type"])
        s["w"] = _normal(gen, (N, K), case["type"], 1 / math.sqrt(3 * K))
        if back:
            s["dy"] = _normal(gen, (M, N), case["type"], 1 / math.sqrt(M))
    elif op == "experts":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        s["experts"] = _choice(gen, T, E, k)
        s["x"] = _activation(gen, T * k if case["rows"] else T, K, case["type"])
        s["w"] = _normal(gen, (E, N, K), case["type"], 1 / math.sqrt(3 * K))
        if back:
            s["dy"] = _normal(gen, (T * k, N), case["type"], 1 / math.sqrt(T))
    else:
        T, k, N = case["T"], case["k"], case["N"]
        s["experts"] = _choice(gen, T, 2 * k, k)
        s["weights"] = torch.rand((T, k), generator=gen, device="cuda").add_(0.05)
        s["y"] = _normal(gen, (T * k, N), case["type"])
        if back:
            s["dout"] = _normal(gen, (T, N), case["type"], 0.1)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, back = case["op"], case["pass"] == "backward"
    if own:  # a program lays its weights out once, and has the router's plan from the call before
        from tensor_gemm_reduce_amd import experts as ex

        if op in ("fp8", "experts"):
            w = s.pop("w")
            # the product's own order, or for the backward pass the transposed one
            s["weight"] = ex.fp8_pack(w, transpose=back)
        if op in ("experts", "combine"):
            s["plan"] = ex.plan(s["experts"], case["E"] if op == "experts" else 2 * case["k"])
        return s
    if op in ("fp8", "experts"):
        s["weight"] = _weight_values(s.pop("w").float())
    if op in ("experts", "combine"):
        s["offsets"], s["tokens"], s["slots"] = _plan(s["experts"], case["E"] if op == "experts" else 2 * case["k"])
        s["starts"] = s["offsets"].tolist()
    return s


# ---- one pass ------------------------------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, c):
    from tensor_gemm_reduce_amd import experts as ex

    op, back = c["op"], c["pass"] == "backward"
    if op == "route":
        kw = dict(score=c["score"], renormalise=c["renorm"], scale=2.5)
        if back:
            return ex.route_backward(s["dweights"], s["logits"], s["experts"], **kw)
        r = ex.route(s["logits"], c["k"], bias=s["bias"], groups=c["groups"], keep_groups=c["keep"], **kw)
        return {"weights": r.weights, "experts": r.experts, "offsets": r.offsets, "tokens": r.tokens, "slots": r.slots}
    if op == "fp8":
        if not back:
            return ex.fp8_linear(s["x"], s["weight"])
        dw = ex.fp8_linear(ex.fp8_quant(s["dy"], transpose=True), ex.fp8_quant(s["x"], transpose=True), dtype=torch.float32)
        return {"dx": ex.fp8_linear(s["dy"], s["weight"]), "dw": dw}
    if op == "experts":
        if not back:
            return ex.experts_linear(s["x"], s["weight"], s["plan"], rows=c["rows"])
        return {"dx": ex.experts_linear(s["dy"], s["weight"], s["plan"], rows=True),
                "dw": ex.experts_wgrad(s["dy"], s["x"], s["plan"], dtype=torch.float32)}
    if not back:
        return ex.combine(s["y"], s["plan"], s["weights"])
    dy, dweights = ex.combine_backward(s["dout"], s["y"], s["plan"], s["weights"])
    return {"dy": dy, "dweights": dweights}


def _run_plain(s, c):
    op, back = c["op"], c["pass"] == "backward"
    if op == "route":
        if back:
            return _route_backward(s, c)
        experts, weights = _choice_of(s["logits"], s["bias"], c)
        offsets, tokens, slots = _plan(experts, c["E"])
        return {"weights": weights, "experts": experts, "offsets": offsets, "tokens": tokens, "slots": slots}
    if op == "fp8":
        kind = s["x"].dtype
        if not back:
            return (_row_values(s["x"].float()) @ s["weight"].t()).to(kind)
        dx = _row_values(s["dy"].float()) @ s["weight"]
        dw = _row_values(s["dy"].float().t().contiguous()) @ _row_values(s["x"].float().t().contiguous()).t()
        return {"dx": dx.to(kind), "dw": dw}
    if op == "experts":
        return _experts(s, c)
    kind, weights = s["y"].dtype, s["weights"]
    slots = s["slots"].long()
    if not back:
        return (s["y"].float()[slots] * weights.unsqueeze(2)).sum(1).to(kind)
    dout, y = s["dout"].float(), s["y"].float()
    dweights = (y[slots] * dout.unsqueeze(1)).sum(2)
    dy = torch.empty_like(y)
    dy[slots] = weights.unsqueeze(2) * dout.unsqueeze(1)
    return {"dy": dy.to(kind), "dweights": dweights}


# ---- plain forms, in 32 bits (choices in 64), rounded once at the end ----------------------------------------------

def _scores(logits, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    return e / e.sum(1, keepdim=True).clamp(min=torch.finfo(e.dtype).tiny)


def _choice_of(logits, bias, c):
    """The chosen experts [T][k], best first, and their weights; -1 and 0 where fewer than k are on (their logit is not
    -inf).  Scores next to a border are compared in 64 bits; ties go to the lowest index."""
    T, E = logits.shape
    k, G = c["k"], c["groups"]
    on = logits > -math.inf
    key = _scores(logits.double(), c["score"])
    if bias is not None:
        key = key + bias.double()
    key = torch.where(on, key, torch.full_like(key, -math.inf))
    if G > 1:
        inside = key.view(T, G, E // G)
        best = inside.sort(dim=2, descending=True)[0][:, :, :2]  # a group counts by its two best
        total = torch.where(torch.isinf(best), torch.zeros_like(best), best).sum(2)
        total = torch.where(torch.isinf(best[:, :, 0]), torch.full_like(total, -math.inf), total)
        order = total.sort(dim=1, descending=True, stable=True)[1][:, :c["keep"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter_(1, order, True)
        key = torch.where(kept.unsqueeze(2), inside, torch.full_like(inside, -math.inf)).view(T, E)
    value, index = key.sort(dim=1, descending=True, stable=True)
    value, index = value[:, :k], index[:, :k]
    chosen = value > -math.inf
    s = torch.where(chosen, _scores(logits.float(), c["score"]).gather(1, index), torch.zeros((), device=key.device))
    if c["renorm"]:
        s = s / (s.sum(1, keepdim=True) + 1e-20)
    return torch.where(chosen, index, torch.full_like(index, -1)).to(torch.int32), 2.5 * s


def _plan(experts, E):
    """Where every (token, j) goes: rows in the order of the experts, and inside one of (token, j).  offsets [E + 1]: the
    experts' first rows; tokens [T k]: the rows' tokens, -1 behind the last row; slots [T][k]: the rows, -1 without one."""
    T, k = experts.shape
    flat = experts.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, E), flat)
    order = key.sort(stable=True)[1]
    counts = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    row = torch.arange(T * k, device=flat.device)
    tokens = torch.where(row < offsets[E], order // k, torch.full_like(row, -1))
    slots = torch.empty_like(row)
    slots[order] = row
    slots = torch.where(flat < 0, torch.full_like(row, -1), slots)
    return offsets.to(torch.int32), tokens.to(torch.int32), slots.view(T, k).to(torch.int32)


def _route_backward(s, c):
    experts = s["experts"].long()
    chosen = experts >= 0
    at = experts.clamp(min=0)
    p = _scores(s["logits"].float(), c["score"])
    sc = torch.where(chosen, p.gather(1, at), torch.zeros((), device=p.device))
    dw = 2.5 * torch.where(chosen, s["dweights"], torch.zeros((), device=p.device))
    if c["renorm"]:
        total = sc.sum(1, keepdim=True) + 1e-20
        dw = (dw - (dw * sc).sum(1, keepdim=True) / total) / total
    ds = torch.zeros_like(p).scatter_add_(1, at, dw)
    if c["score"] == "sigmoid":
        d = ds * p * (1 - p)
    else:
        d = p * (ds - (ds * p).sum(1, keepdim=True))
    return d.to(s["logits"].dtype)


def _power(e):
    """2^e exactly, from its exponent bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(top):
    """The smallest e >= -126 with top <= 448 2^e."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)
    return torch.where(top == 0, torch.full_like(e, -126), e)


def _row_values(x):
    """What a matrix in blocks of 128 columns of a row stands for."""
    M, K = x.shape
    v = torch.nn.functional.pad(x, (0, -K % BLOCK)).view(M, -1, BLOCK)
    e = _exponent(v.abs().amax(-1, keepdim=True))
    return ((v * _power(-e)).to(torch.float8_e4m3fn).float() * _power(e)).view(M, -1)[:, :K]


def _weight_values(w):
    """What weights (one matrix or one for each expert) in blocks of 128 x 128 stand for."""
    N, K = w.shape[-2:]
    v = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK))
    v = v.view(-1, v.shape[-2] // BLOCK, BLOCK, v.shape[-1] // BLOCK, BLOCK)
    e = _exponent(v.abs().amax((2, 4), keepdim=True))
    v = ((v * _power(-e)).to(torch.float8_e4m3fn).float() * _power(e)).flatten(3).flatten(1, 2)
    return v[:, :N, :K].reshape(w.shape)


def _experts(s, c):
    x, kind, starts, tokens = s["x"].float(), s["x"].dtype, s["starts"], s["tokens"].long()
    R = tokens.shape[0]
    if c["pass"] == "forward":
        x = _row_values(x)
        y = x.new_empty((R, c["N"]))
        for e in range(c["E"]):
            r = slice(starts[e], starts[e + 1])
            y[r] = (x[r] if c["rows"] else x[tokens[r]]) @ s["weight"][e].t()
        return y.to(kind)
    dy = s["dy"].float()
    dq = _row_values(dy)
    dx = x.new_empty((R, c["K"]))
    dw = x.new_zeros((c["E"], c["N"], c["K"]))
    for e in range(c["E"]):
        r = slice(starts[e], starts[e + 1])
        if starts[e] == starts[e + 1]:
            continue
        dx[r] = dq[r] @ s["weight"][e]
        dw[e] = _row_values(dy[r].t().contiguous()) @ _row_values(x[tokens[r]].t().contiguous()).t()
    return {"dx": dx.to(kind), "dw": dw}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------------

def exact(case, seed):
    if work(case)["flops"] > 3e13:
        return None  # over 20 seconds in 64 bits
    s = _inputs(case, seed)
    op, back = case["op"], case["pass"] == "backward"
    if op == "route":
        return _exact_route_backward(case, s) if back else _exact_route(case, s)
    if op == "fp8":
        x, w = s["x"].double(), _exact_e4m3(s["w"].double(), 128, 128)
        if not back:
            return torch.matmul(_exact_e4m3(x, 1, 128), w.transpose(0, 1).contiguous())
        dy = s["dy"].double()
        dw = torch.matmul(_exact_e4m3(dy, 128, 1).transpose(0, 1).contiguous(), _exact_e4m3(x, 128, 1))
        return {"dx": torch.matmul(_exact_e4m3(dy, 1, 128), w), "dw": dw}
    if op == "experts":
        return _exact_experts(case, s)
    row, _, _ = _exact_rows(s["experts"], 2 * case["k"])
    y, weights = s["y"].double(), s["weights"].double()
    if not back:
        out = torch.zeros((case["T"], case["N"]), dtype=torch.float64, device=y.device)
        for j in range(case["k"]):
            out += weights[:, j, None] * y[row[:, j]]
        return out
    dout = s["dout"].double()
    dy, dweights = torch.empty_like(y), torch.empty_like(weights)
    for j in range(case["k"]):
        dy[row[:, j]] = weights[:, j, None] * dout
        dweights[:, j] = torch.einsum("tn,tn->t", dout, y[row[:, j]])
    return {"dy": dy, "dweights": dweights}


def _exact_e4m3(x, rows, cols):
    """x with blocks of rows x cols scaled by the smallest power of two (from 2^-126 on) that brings them to at most 448,
    rounded to three bits behind the leading one (at least 2^-6), ties to even, and scaled back."""
    M, K = x.shape
    m, k = -(-M // rows), -(-K // cols)
    v = torch.zeros((m * rows, k * cols), dtype=torch.float64, device=x.device)
    v[:M, :K] = x
    v = v.view(m, rows, k, cols)
    top = v.abs().amax(dim=3, keepdim=True).amax(dim=1, keepdim=True)
    power = (top / TOP).view(torch.int64)
    # rounded up to a power of two (the quotient is one exactly where top is 448 times one)
    up = (power >> 52) - 1023 + ((power & ((1 << 52) - 1)) != 0).long()
    scale = _exact_power(torch.clamp(up, min=-126))
    u = v / scale
    lead = torch.clamp((u.view(torch.int64) >> 52 & 2047) - 1023, min=-6)
    step = _exact_power(lead - 3)
    return (torch.round(u / step) * step * scale).reshape(m * rows, k * cols)[:M, :K].contiguous()


def _exact_power(n):
    return torch.bitwise_left_shift(n + 1023, 52).view(torch.float64)


def _exact_scores(l, score):
    if score == "sigmoid":
        return torch.special.expit(l)
    p = torch.softmax(l, dim=1)
    return torch.where(torch.isnan(p), torch.zeros_like(p), p)  # a row of -inf


def _exact_rank(key):
    """How many keys of its row come before each: larger ones, and equal ones to the left."""
    n = key.shape[1]
    out = []
    for part in key.split(max(1, (1 << 26) // (n * n))):
        a, b = part[:, None, :], part[:, :, None]
        left = torch.ones((n, n), dtype=torch.bool, device=key.device).tril(-1)
        out.append(((a > b) | ((a == b) & left)).sum(dim=2))
    return torch.cat(out)


def _exact_route(c, s):
    l = s["logits"].double()
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    p = _exact_scores(l, c["score"])
    key = p if s["bias"] is None else p + s["bias"].double()
    off = torch.isneginf(l)
    key = key.masked_fill(off, -math.inf)
    if G > 1:
        parts = key.reshape(T * G, E // G)
        rank = _exact_rank(parts)
        total = torch.where((rank < 2) & ~torch.isneginf(parts), parts, torch.zeros_like(parts)).sum(dim=1)
        total = total.masked_fill(off.reshape(T * G, -1).all(dim=1), -math.inf)
        inside = _exact_rank(total.view(T, G)) < c["keep"]
        key = key.masked_fill(~inside.repeat_interleave(E // G, dim=1), -math.inf)
    rank = _exact_rank(key)
    experts = torch.full((T, k + 1), -1, dtype=torch.int32, device=l.device)
    weights = torch.zeros((T, k + 1), dtype=torch.float64, device=l.device)
    place = torch.where(torch.isneginf(key), torch.full_like(rank, k), rank.clamp(max=k))
    experts.scatter_(1, place, torch.arange(E, device=l.device, dtype=torch.int32).expand(T, E).contiguous())
    weights.scatter_(1, place, p)
    experts, weights = experts[:, :k].contiguous(), weights[:, :k]
    if c["renorm"]:
        weights = weights / (weights.sum(dim=1, keepdim=True) + 1e-20)
    row, tokens, offsets = _exact_rows(experts, E)
    return {"weights": 2.5 * weights, "experts": experts, "offsets": offsets, "tokens": tokens, "slots": row.to(torch.int32)}


def _exact_rows(experts, E):
    """Rows by counting, expert by expert: (row of each (token, j), the rows' tokens, the experts' first rows)."""
    T, k = experts.shape
    flat = experts.reshape(-1)
    row = torch.full((T * k,), -1, dtype=torch.int64, device=flat.device)
    tokens = torch.full((T * k,), -1, dtype=torch.int32, device=flat.device)
    starts, n = [0], 0
    for e in range(E):
        where = torch.nonzero(flat == e).reshape(-1)
        m = where.numel()
        row[where] = torch.arange(n, n + m, device=flat.device)
        tokens[n:n + m] = torch.div(where, k, rounding_mode="floor").to(torch.int32)
        n += m
        starts.append(n)
    return row.view(T, k), tokens, torch.tensor(starts, dtype=torch.int32, device=flat.device)


def _exact_route_backward(c, s):
    """Through the Jacobians: dl = J_score^T (mask) J_weights^T dw."""
    l, e = s["logits"].double(), s["experts"].long()
    p = _exact_scores(l, c["score"])
    hot = torch.zeros((e.shape[0], e.shape[1], c["E"]), dtype=torch.float64, device=l.device)
    hot.scatter_(2, e.clamp(min=0)[:, :, None], (e >= 0).double()[:, :, None])
    chosen = (hot * p[:, None, :]).sum(dim=2)
    dw = 2.5 * s["dweights"].double() * (e >= 0)
    if c["renorm"]:
        D = chosen.sum(dim=1, keepdim=True) + 1e-20
        dw = dw / D - (dw * chosen).sum(dim=1, keepdim=True) / (D * D)
    ds = (hot * dw[:, :, None]).sum(dim=1)
    if c["score"] == "sigmoid":
        return ds * p * torch.special.expit(-torch.where(torch.isneginf(l), torch.zeros_like(l), l))
    return ds * p - p * (ds * p).sum(dim=1, keepdim=True)


def _exact_experts(c, s):
    row, tokens, offsets = _exact_rows(s["experts"], c["E"])
    first = offsets.tolist()
    x = s["x"].double()
    if not c["rows"]:
        x = x[tokens.long()]
    y = torch.empty((tokens.numel(), c["N"]), dtype=torch.float64, device=x.device)
    dx = torch.empty((tokens.numel(), c["K"]), dtype=torch.float64, device=x.device)
    dw = torch.zeros((c["E"], c["N"], c["K"]), dtype=torch.float64, device=x.device) if "dy" in s else None
    for e in range(c["E"]):
        a, b = first[e], first[e + 1]
        if a == b:
            continue
        w = _exact_e4m3(s["w"][e].double(), 128, 128)
        if dw is None:
            y[a:b] = torch.matmul(_exact_e4m3(x[a:b], 1, 128), w.transpose(0, 1).contiguous())
            continue
        dy = s["dy"][a:b].double()
        dx[a:b] = torch.matmul(_exact_e4m3(dy, 1, 128), w)
        dw[e] = torch.matmul(_exact_e4m3(dy, 128, 1).transpose(0, 1).contiguous(), _exact_e4m3(x[a:b], 128, 1))
    return y if dw is None else {"dx": dx, "dw": dw}


# ---- what a pass cannot do without ------------------------------------------------------------------------------------

def _packed(n, k):
    """Bytes of n x k weights and their scales."""
    return n * k + -(-n // BLOCK) * -(-k // BLOCK)


def work(case):
    op, back = case["op"], case["pass"] == "backward"
    b = BYTES[case["type"]]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        if back:
            return {"bytes": 2 * T * E * b + 8 * T * k, "flops": 12 * T * E}
        return {"bytes": T * E * b + (4 * E if case["bias"] else 0) + 16 * T * k + 4 * (E + 1), "flops": (12 + k) * T * E}
    if op == "fp8":
        M, N, K = case["M"], case["N"], case["K"]
        if back:
            return {"bytes": M * N * b + 2 * M * K * b + _packed(N, K) + 4 * N * K, "flops": 4 * M * N * K}
        return {"bytes": M * K * b + M * N * b + _packed(N, K), "flops": 2 * M * N * K}
    if op == "experts":
        T, E, k, N, K = (case[n] for n in ("T", "E", "k", "N", "K"))
        R = T * k
        weights = min(E, R) * _packed(N, K)  # of the experts that can have a row
        x = (R if case["rows"] else T) * K * b
        if back:
            return {"bytes": R * N * b + x + R * K * b + weights + 4 * E * N * K, "flops": 4 * R * N * K}
        return {"bytes": x + R * N * b + weights + 8 * R, "flops": 2 * R * N * K}
    T, k, N = case["T"], case["k"], case["N"]
    if back:
        return {"bytes": (2 * T * k + T) * N * b + 12 * T * k, "flops": 3 * T * k * N}
    return {"bytes": (T * k + T) * N * b + 8 * T * k, "flops": 2 * T * k * N}
