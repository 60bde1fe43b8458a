"""ctypes binding of include/gemm_rs_experts.h (in libgemm_rs_layer.so): the router, the
experts' products and the 8-bit floating-point product beside the row-parallel layer.

  fp8_quant, fp8_pack, fp8_linear     matrices in e4m3 with a scale for each block of 128 inputs, and their product
  route, plan, route_backward         the choice of k experts for each token, and the rows of every expert
  experts_linear, experts_wgrad       the product of every row with its expert's weights, and the weights' gradients
  combine, combine_backward           a token's rows back into one

Argument checks and marshalling only, with the conventions of ``layer``: tensors live on
the current device, rows may be strided, work is enqueued on ``stream`` (default: torch's
current stream) and calls return at once; outputs and workspaces come from torch's
allocator on that stream; no history for autograd.  How many rows an expert has stays on
the device: no call waits for it.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import layer as _layer
from .gemm_rs import ERR_UNSUPPORTED_SHAPE
from .layer import (_CODES, GemmRSLayerError, _check, _device, _elsewhere, _flat, _on_stream, _ptr, _raw_stream,
                    _rows, _two)

# ---- constants mirrored from include/gemm_rs_experts.h -------------------------
FP8_BLOCK = 128
DTYPE_FP8 = 3
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
ROUTE_MAX_EXPERTS = 1024
ROUTE_MAX_CHOICES = 64

EXPORTS = ("gemm_rs_fp8_quant", "gemm_rs_fp8_quant_transposed", "gemm_rs_fp8_pack", "gemm_rs_fp8_plan", "gemm_rs_fp8_workspace",
           "gemm_rs_fp8_linear", "gemm_rs_experts_linear", "gemm_rs_experts_wgrad_plan", "gemm_rs_experts_wgrad_workspace",
           "gemm_rs_experts_wgrad",
           "gemm_rs_route_validate", "gemm_rs_expert_plan_workspace", "gemm_rs_route", "gemm_rs_expert_plan",
           "gemm_rs_route_backward", "gemm_rs_combine", "gemm_rs_combine_backward")

_vp, _i32, _i64, _f32, _size = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t)
_SCORES = {"softmax": SCORE_SOFTMAX, "sigmoid": SCORE_SIGMOID}


class gemm_rs_fp8_args(ctypes.Structure):
    _fields_ = [("x_dtype", _i32), ("out_dtype", _i32), ("M", _i64), ("N", _i64), ("K", _i64), ("x_rows", _i64), ("E", _i64),
                ("x", _vp), ("x_stride", _i64), ("x_scales", _vp), ("w", _vp), ("w_scales", _vp), ("offsets", _vp),
                ("tokens", _vp), ("add", _vp), ("add_stride", _i64), ("out", _vp), ("out_stride", _i64)]


class gemm_rs_experts_wgrad_args(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("out_dtype", _i32), ("M", _i64), ("N", _i64), ("K", _i64), ("E", _i64), ("x_rows", _i64),
                ("dy", _vp), ("dy_stride", _i64), ("x", _vp), ("x_stride", _i64), ("offsets", _vp), ("tokens", _vp),
                ("add", _vp), ("dw", _vp)]


class gemm_rs_route_config(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("dtype", "E", "k", "score", "renormalise", "groups", "keep_groups")] + [("scale", _f32)]


class gemm_rs_expert_plan_args(ctypes.Structure):
    _fields_ = [("offsets", _vp), ("tokens", _vp), ("slots", _vp)]


class gemm_rs_fp8_info(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("tile", "stages", "quantises", "tiles", "workgroups")]


# The argument blocks as calls pack them.
_FP8_ARGS = struct.Struct("2i5qQqQQQQQQqQq")
_WGRAD_ARGS = struct.Struct("2i5qQqQqQQQQ")
_ROUTE_CONFIG = struct.Struct("7if")
_PLAN_ARGS = struct.Struct("3Q")

_BOUND = None


def lib():
    global _BOUND
    if _BOUND is None:
        L = _layer.lib()
        a = _vp  # a structure's packed bytes
        L.gemm_rs_fp8_quant.argtypes = [_i32, _i64, _i64, _vp, _i64, _vp, _vp, _vp]
        L.gemm_rs_fp8_quant_transposed.argtypes = [_i32, _i64, _i64, _vp, _i64, _vp, _vp, _vp]
        L.gemm_rs_fp8_pack.argtypes = [_i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp]
        L.gemm_rs_fp8_plan.argtypes = [a, ctypes.POINTER(gemm_rs_fp8_info)]
        L.gemm_rs_fp8_workspace.argtypes = [a]
        L.gemm_rs_fp8_linear.argtypes = [a, _vp, _size, _vp]
        L.gemm_rs_experts_linear.argtypes = [a, _vp, _size, _vp]
        L.gemm_rs_experts_wgrad_plan.argtypes = [a, ctypes.POINTER(gemm_rs_fp8_info)]
        L.gemm_rs_experts_wgrad_workspace.argtypes = [a]
        L.gemm_rs_experts_wgrad.argtypes = [a, _vp, _size, _vp]
        L.gemm_rs_route_validate.argtypes = [a]
        L.gemm_rs_expert_plan_workspace.argtypes = [_i64, _i32, _i32]
        L.gemm_rs_route.argtypes = [a, _i64, _vp, _i64, _vp, _vp, _vp, a, _vp, _size, _vp]
        L.gemm_rs_expert_plan.argtypes = [_i64, _i32, _i32, _vp, a, _vp, _size, _vp]
        L.gemm_rs_route_backward.argtypes = [a, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp]
        L.gemm_rs_combine.argtypes = [_i32, _i64, _i64, _i64, _i32, _vp, _i64, _vp, _vp, _vp, _i64, _vp]
        L.gemm_rs_combine_backward.argtypes = [_i32, _i64, _i64, _i64, _i32, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i64, _vp, _vp]
        for name in EXPORTS:
            getattr(L, name).restype = _size if name.endswith("_workspace") else ctypes.c_int
        _BOUND = L
    return _BOUND


def _code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {t.dtype}")
    return code


def _ints(t, name, shape, dev):
    _flat(t, name, shape, torch.int32, dev)
    return t.data_ptr()


def _plan_rows(routing, rows, dev):
    """Addresses of a plan's first rows, and of its rows' tokens where x is gathered by them."""
    return (_ints(routing.offsets, "routing.offsets", (routing.E + 1,), dev),
            0 if rows else _ints(routing.tokens, "routing.tokens", (routing.rows,), dev))


def _workspace(like, size):
    return like.new_empty(size, dtype=torch.uint8) if size else None


# ---- matrices in 8 bits ---------------------------------------------------------------

def _up(n, unit):
    return -(-n // unit) * unit


class Fp8:
    """A matrix [rows][K], or E of them, in e4m3 with a power-of-two scale for each block of 128 columns of a row:
    q float8_e4m3fn [(E,) rows, K rounded up to 128], zeros past K; scales uint8 [(E,) blocks, rows + 3 rounded up to 4],
    e + 127 of the scale 2^e of a row's block (bytes past the rows are not used; 127 for a block of zeros).  A block with an
    infinity or a NaN stands for NaN."""

    __slots__ = ("q", "scales", "E", "rows", "K")

    def __init__(self, q, scales, rows, K):
        lead = q.shape[:-2]
        if q.dim() not in (2, 3) or rows < 0 or K < 1:
            raise ValueError(f"q: expected [rows][K] or [E][rows][K], got shape {tuple(q.shape)}")
        dev = q.get_device()
        _flat(q, "q", (*lead, rows, _up(K, FP8_BLOCK)), torch.float8_e4m3fn, dev)
        _flat(scales, "scales", (*lead, -(-K // FP8_BLOCK), _up(rows + 3, 4)), torch.uint8, dev)
        self.q, self.scales, self.rows, self.K = q, scales, rows, K
        self.E = lead[0] if lead else 0

    def values(self):
        """What the matrix stands for, in float32 (plain torch, for checks and exports)."""
        e = self.scales[..., :self.rows].transpose(-1, -2).to(torch.int32)
        scale = torch.ldexp(torch.ones((), device=self.q.device), e - 127)
        return (self.q.float() * scale.repeat_interleave(FP8_BLOCK, dim=-1))[..., :self.K]


def _new_fp8(like, lead, rows, K):
    m = Fp8.__new__(Fp8)
    m.q = like.new_empty((*lead, rows, _up(K, FP8_BLOCK)), dtype=torch.float8_e4m3fn)
    m.scales = like.new_empty((*lead, -(-K // FP8_BLOCK), _up(rows + 3, 4)), dtype=torch.uint8)
    m.E, m.rows, m.K = (lead[0] if lead else 0), rows, K
    return m


def _fp8(m, name, dev):
    if m.q.get_device() != dev:
        raise ValueError(f"{name}: on {m.q.device}, not on the current device")


def fp8_quant(x, *, transpose=False, stream=None) -> Fp8:
    """x [M][K] (bfloat16, float16 or float32) in 8 bits, in blocks of 128 columns of a row: each holds e4m3(x 2^-e) with
    the smallest e >= -126 that brings it to at most 448.

    transpose=True: x^T [K][M] in blocks of 128 rows of x, an operand of the weight gradient.
    """
    M, K = _two(x, "x")
    code = _code(x, "x")
    if K < 1 or (transpose and M < 1):
        raise ValueError(f"x: no blocks in shape {tuple(x.shape)}")
    dev = _device(x, "x")
    xs = _rows(x, "x", M, K, x.dtype, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(fp8_quant, other, (x,), x, transpose=transpose)
    m = _new_fp8(x, (), K, M) if transpose else _new_fp8(x, (), M, K)
    call = lib().gemm_rs_fp8_quant_transposed if transpose else lib().gemm_rs_fp8_quant
    _check(call(code, M, K, x.data_ptr(), xs, m.q.data_ptr(), m.scales.data_ptr(), _raw_stream(dev)), "gemm_rs_fp8_quant")
    return m


def fp8_pack(w, *, transpose=False, stream=None) -> Fp8:
    """Weights [N][K], or [E][N][K] for E experts, in 8 bits, in blocks of 128 x 128 that share a scale, once.

    transpose=True: w^T [K][N] with the same values, the operand of the input's gradient.
    """
    if w.dim() not in (2, 3):
        raise ValueError(f"w: expected [N][K] or [E][N][K], got shape {tuple(w.shape)}")
    lead, (N, K) = w.shape[:-2], w.shape[-2:]
    code = _code(w, "w")
    dev = _device(w, "w")
    _flat(w, "w", w.shape, w.dtype, dev)
    if min(w.shape) < 1:
        raise ValueError(f"w: empty shape {tuple(w.shape)}")
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(fp8_pack, other, (w,), w, transpose=transpose)
    m = _new_fp8(w, lead, K, N) if transpose else _new_fp8(w, lead, N, K)
    _check(lib().gemm_rs_fp8_pack(code, lead[0] if lead else 1, N, K, int(transpose), w.data_ptr(), m.q.data_ptr(),
                                  m.scales.data_ptr(), _raw_stream(dev)), "gemm_rs_fp8_pack")
    return m


# ---- the products -----------------------------------------------------------------------

def _product(name, x, weight, routing, rows, add, out, dtype, stream):
    K, N = weight.K, weight.rows
    raw = isinstance(x, torch.Tensor)
    if raw:
        x_rows, _ = _two(x, "x")
        code, x_scales = _code(x, "x"), 0
        dev = _device(x, "x")
        x_stride, like = _rows(x, "x", x_rows, K, x.dtype, dev), x
    else:
        if x.E or x.K != K:
            raise ValueError(f"x: {x.rows} rows of {x.K} inputs{' for each expert' if x.E else ''}, the weights have {K}")
        x_rows, x_stride, code, like = x.rows, 0, DTYPE_FP8, x.q
        dev = _device(x.q, "x")
        x_scales = x.scales.data_ptr()
    _fp8(weight, "weight", dev)
    M, E, offsets, tokens = x_rows, 0, 0, 0
    if routing is not None:
        M, E = routing.rows, routing.E
        if weight.E != E:
            raise ValueError(f"weight: of {weight.E} experts, the plan has {E}")
        want = M if rows else routing.T
        if x_rows != want:
            raise ValueError(f"x: {x_rows} rows, the plan has {want} {'rows' if rows else 'tokens'}")
        offsets, tokens = _plan_rows(routing, rows, dev)
    elif weight.E:
        raise ValueError("weight: of several experts; use experts_linear")
    if out is not None:
        dtype = out.dtype
    elif dtype is None:
        dtype = x.dtype if raw else torch.bfloat16
    if dtype not in _CODES:
        raise TypeError(f"dtype: expected bfloat16, float16 or float32, got {dtype}")
    if add is not None and dtype is not torch.float32:
        raise TypeError(f"add: needs a float32 out, not {dtype}")
    add_stride = 0 if add is None else _rows(add, "add", M, N, torch.float32, dev)
    out_stride = N if out is None else _rows(out, "out", M, N, dtype, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            used = [x] if raw else [x.q, x.scales]
            used += [weight.q, weight.scales, add, out] + ([routing.offsets, routing.tokens] if routing is not None else [])
            return _on_stream(_product, other, used, name, x, weight, routing, rows, add, out, dtype, None)
    if out is None:
        out = like.new_empty((M, N), dtype=dtype)
    args = _FP8_ARGS.pack(code, _CODES[dtype], M, N, K, x_rows, E, (x if raw else x.q).data_ptr(), x_stride, x_scales,
                          weight.q.data_ptr(), weight.scales.data_ptr(), offsets, tokens, _ptr(add), add_stride,
                          out.data_ptr(), out_stride)
    L = lib()
    size = L.gemm_rs_fp8_workspace(args)
    ws = _workspace(like, size)
    _check(getattr(L, name)(args, _ptr(ws), size, _raw_stream(dev)), name)
    return out


def fp8_linear(x, weight: Fp8, *, add=None, out=None, dtype=None, stream=None):
    """out [M][N] = x w^T (+ add), FP32 accumulation, rounded once.

    For bfloat16 and float16 results the products of eight neighbouring inputs lose what lies below 2^-13 of the largest of
    them, together less than 2^-10 of it: up to two half steps of float16, a quarter of bfloat16's.  dtype=torch.float32 keeps every
    product whole, at half the rate.
    x: [M][K] bfloat16, float16 or float32, quantised by the call as fp8_quant does, or an Fp8.  weight: an Fp8 [N][K].
    dtype: of out (default: x's; bfloat16 for an Fp8).  add: float32 [M][N] or None, with a float32 out, which may be it.
    The gradients of y = x w^T: fp8_linear(dy, fp8_pack(w, transpose=True)) and
    fp8_linear(fp8_quant(dy, transpose=True), fp8_quant(x, transpose=True), dtype=torch.float32).
    """
    return _product("gemm_rs_fp8_linear", x, weight, None, False, add, out, dtype, stream)


# ---- router --------------------------------------------------------------------------------

class Routing:
    """What route and plan return, for T tokens with k choices of E experts each and R = T k rows:
    weights float32 [T][k] and experts int32 [T][k] (-1: none); offsets int32 [E + 1], the experts' first rows and the
    number of rows; tokens int32 [R], the rows' tokens (-1 behind the last row); slots int32 [T][k], the choices' rows
    (-1: none).  plan leaves weights at None.  A program's own plan has to have these types and shapes, contiguous and on one
    device; what its numbers say is its own matter (rows and tokens out of range are not read)."""

    __slots__ = ("weights", "experts", "offsets", "tokens", "slots", "T", "k", "E", "rows")

    def __init__(self, weights, experts, offsets, tokens, slots, E):
        T, k = _two(experts, "experts")
        if E < 1:
            raise ValueError(f"E: {E}")
        dev = experts.get_device()
        for t, name, shape in ((experts, "experts", (T, k)), (offsets, "offsets", (E + 1,)), (tokens, "tokens", (T * k,)),
                               (slots, "slots", (T, k))):
            _flat(t, name, shape, torch.int32, dev)
        if weights is not None:
            _flat(weights, "weights", (T, k), torch.float32, dev)
        self._set(weights, experts, offsets, tokens, slots, E)

    def _set(self, weights, experts, offsets, tokens, slots, E):
        self.weights, self.experts, self.offsets, self.tokens, self.slots, self.E = weights, experts, offsets, tokens, slots, E
        self.T, self.k = experts.shape
        self.rows = self.T * self.k
        return self


def _new_plan(like, T, k, E):
    new = like.new_empty
    n = T * k
    ints = new(E + 1 + 2 * n, dtype=torch.int32)
    return ints[:E + 1], ints[E + 1:E + 1 + n], ints[E + 1 + n:].view(T, k)


def _route_config(logits, E, k, score, renormalise, scale, groups=1, keep_groups=1):
    if score not in _SCORES:
        raise ValueError(f"score: 'softmax' or 'sigmoid', got {score!r}")
    if not math.isfinite(scale):
        raise ValueError(f"scale: {scale}")
    if max(abs(E), abs(k), abs(groups), abs(keep_groups)) >= 1 << 31:
        raise GemmRSLayerError(ERR_UNSUPPORTED_SHAPE, "route")
    return _ROUTE_CONFIG.pack(_code(logits, "logits"), E, k, _SCORES[score], bool(renormalise), groups, keep_groups, scale)


def route(logits, k, *, score="softmax", bias=None, groups=1, keep_groups=None, renormalise=True, scale=1.0, stream=None) -> Routing:
    """The k experts of each token, their weights, and the plan of the experts' rows.

    logits: [T][E] bfloat16, float16 or float32; -inf turns an expert off for a token, and a token with fewer than k on has
    -1 and weight 0 for the rest, which take no row (a padded batch: rows of -inf).
    s = softmax or sigmoid of the logits; the largest s + bias are chosen (bias: float32 [E], for balance; ties to the
    lowest index), with groups > 1 from the keep_groups groups of neighbouring experts with the largest sums of their two
    best.  weights = scale s, or with renormalise scale s / (sum of the chosen s + 1e-20).
    """
    T, E = _two(logits, "logits")
    cfg = _route_config(logits, E, k, score, renormalise, scale, groups, groups if keep_groups is None else keep_groups)
    dev = _device(logits, "logits")
    ls = _rows(logits, "logits", T, E, logits.dtype, dev)
    if bias is not None:
        _flat(bias, "bias", (E,), torch.float32, dev)
    L = lib()
    _check(L.gemm_rs_route_validate(cfg), "gemm_rs_route")
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(route, other, (logits, bias), logits, k, score=score, bias=bias, groups=groups,
                              keep_groups=keep_groups, renormalise=renormalise, scale=scale)
    weights = logits.new_empty((T, k), dtype=torch.float32)
    experts = logits.new_empty((T, k), dtype=torch.int32)
    offsets, tokens, slots = _new_plan(logits, T, k, E)
    size = L.gemm_rs_expert_plan_workspace(T, E, k)
    ws = _workspace(logits, size)
    _check(L.gemm_rs_route(cfg, T, logits.data_ptr(), ls, _ptr(bias), weights.data_ptr(), experts.data_ptr(),
                           _PLAN_ARGS.pack(offsets.data_ptr(), tokens.data_ptr(), slots.data_ptr()), _ptr(ws), size,
                           _raw_stream(dev)), "gemm_rs_route")
    return Routing.__new__(Routing)._set(weights, experts, offsets, tokens, slots, E)


def plan(experts, num_experts, *, stream=None) -> Routing:
    """The plan of given choices: experts int32 [T][k], contiguous; an index outside 0 .. num_experts - 1 takes no row."""
    T, k = _two(experts, "experts")
    dev = _device(experts, "experts")
    _flat(experts, "experts", (T, k), torch.int32, dev)
    if max(abs(num_experts), k) >= 1 << 31:
        raise GemmRSLayerError(ERR_UNSUPPORTED_SHAPE, "plan")
    if num_experts < 1:
        raise ValueError(f"num_experts: {num_experts}")
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(plan, other, (experts,), experts, num_experts)
    L = lib()
    offsets, tokens, slots = _new_plan(experts, T, k, num_experts)
    size = L.gemm_rs_expert_plan_workspace(T, num_experts, k)
    ws = _workspace(experts, size)
    _check(L.gemm_rs_expert_plan(T, num_experts, k, experts.data_ptr(),
                                 _PLAN_ARGS.pack(offsets.data_ptr(), tokens.data_ptr(), slots.data_ptr()), _ptr(ws), size,
                                 _raw_stream(dev)), "gemm_rs_expert_plan")
    return Routing.__new__(Routing)._set(None, experts, offsets, tokens, slots, num_experts)


def route_backward(dweights, logits, experts, *, score="softmax", renormalise=True, scale=1.0, stream=None):
    """The logits' gradient [T][E] (of their type) from the weights' gradients float32 [T][k].

    logits, score, renormalise, scale: what route had; experts: what it chose (the choice itself has no gradient).
    """
    T, E = _two(logits, "logits")
    _, k = _two(experts, "experts")
    cfg = _route_config(logits, E, k, score, renormalise, scale)
    dev = _device(logits, "logits")
    ls = _rows(logits, "logits", T, E, logits.dtype, dev)
    ids = _ints(experts, "experts", (T, k), dev)
    _flat(dweights, "dweights", (T, k), torch.float32, dev)
    L = lib()
    _check(L.gemm_rs_route_validate(cfg), "gemm_rs_route_backward")
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(route_backward, other, (dweights, logits, experts), dweights, logits, experts, score=score,
                              renormalise=renormalise, scale=scale)
    out = logits.new_empty((T, E))
    _check(L.gemm_rs_route_backward(cfg, T, logits.data_ptr(), ls, ids, dweights.data_ptr(), out.data_ptr(), E,
                                    _raw_stream(dev)), "gemm_rs_route_backward")
    return out


# ---- experts ---------------------------------------------------------------------------------

def experts_linear(x, weight: Fp8, routing: Routing, *, rows=False, add=None, out=None, dtype=None, stream=None):
    """out [R][N]: every row times its expert's weights, in the order of the plan's rows; rows behind the last stay as they
    were (in a new output: unset).

    x: [T][K], a token's inputs (gathered by the product), or with rows=True [R][K], in the order of the rows: a tensor
    or an Fp8 as in fp8_linear.  weight: an Fp8 of E experts.
    Products are fp8_linear's, as are their roundings.
    The gradient of the rows' inputs: experts_linear(dy, fp8_pack(w, transpose=True), routing, rows=True), which
    combine(.., None) adds up over a token's rows.
    """
    return _product("gemm_rs_experts_linear", x, weight, routing, rows, add, out, dtype, stream)


def experts_wgrad(dy, x, routing: Routing, *, rows=False, add=None, out=None, dtype=torch.float32, stream=None):
    """The weights' gradients [E][N][K] = dy^T x (+ add) of every expert, both in 8 bits in blocks of 128 of its rows.

    dy: [R][N], x: [T][K] or with rows=True [R][K], of one type.  dtype: float32, every product whole, or dy's, with fp8_linear's
    roundings (out's, if given).
    add: float32 [E][N][K], contiguous, or None, with a float32 out, which may be it.
    """
    M, N = _two(dy, "dy")
    x_rows, K = _two(x, "x")
    code = _code(dy, "dy")
    dev = _device(dy, "dy")
    E = routing.E
    ys, xs = _rows(dy, "dy", routing.rows, N, dy.dtype, dev), _rows(x, "x", routing.rows if rows else routing.T, K, dy.dtype, dev)
    offsets, tokens = _plan_rows(routing, rows, dev)
    if out is not None:
        dtype = out.dtype
    if dtype is not torch.float32 and dtype is not dy.dtype:
        raise TypeError(f"dtype: expected float32 or {dy.dtype}, got {dtype}")
    if add is not None and dtype is not torch.float32:
        raise TypeError(f"add: needs a float32 out, not {dtype}")
    if min(N, K) < 1:
        raise ValueError(f"dy, x: no columns in shapes {tuple(dy.shape)}, {tuple(x.shape)}")
    for t, name, kind in ((add, "add", torch.float32), (out, "out", dtype)):
        if t is not None:
            _flat(t, name, (E, N, K), kind, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(experts_wgrad, other, (dy, x, routing.offsets, routing.tokens, add, out), dy, x, routing,
                              rows=rows, add=add, out=out, dtype=dtype)
    if out is None:
        out = dy.new_empty((E, N, K), dtype=dtype)
    args = _WGRAD_ARGS.pack(code, _CODES[dtype], M, N, K, E, x_rows, dy.data_ptr(), ys, x.data_ptr(), xs,
                            offsets, tokens, _ptr(add), out.data_ptr())
    L = lib()
    size = L.gemm_rs_experts_wgrad_workspace(args)
    ws = _workspace(dy, size)
    _check(L.gemm_rs_experts_wgrad(args, _ptr(ws), size, _raw_stream(dev)), "gemm_rs_experts_wgrad")
    return out


def _weights(weights, routing, dev):
    if weights is None:
        return 0
    _flat(weights, "weights", (routing.T, routing.k), torch.float32, dev)
    return weights.data_ptr()


def combine(y, routing: Routing, weights, *, out=None, stream=None):
    """out [T][N]: the sum over a token's choices of weight times row, FP32, rounded once.

    y: [R][N] in the order of the plan's rows.  weights: float32 [T][k] (route's), or None for ones.
    """
    R, N = _two(y, "y")
    code = _code(y, "y")
    dev = _device(y, "y")
    ys = _rows(y, "y", routing.rows, N, y.dtype, dev)
    slots = _ints(routing.slots, "routing.slots", (routing.T, routing.k), dev)
    w = _weights(weights, routing, dev)
    os = N if out is None else _rows(out, "out", routing.T, N, y.dtype, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(combine, other, (y, routing.slots, weights, out), y, routing, weights, out=out)
    if out is None:
        out = y.new_empty((routing.T, N))
    _check(lib().gemm_rs_combine(code, routing.T, R, N, routing.k, y.data_ptr(), ys, slots, w, out.data_ptr(), os,
                                 _raw_stream(dev)), "gemm_rs_combine")
    return out


def combine_backward(dout, y, routing: Routing, weights, *, dy=None, stream=None):
    """(dy [R][N], dweights float32 [T][k]) from dout [T][N]; rows of dy behind the last stay as they were (in a new one:
    unset).  y: combine's, or None for no weights' gradients (dweights is then None).  weights: combine's.
    """
    T, N = _two(dout, "dout")
    code = _code(dout, "dout")
    dev = _device(dout, "dout")
    ds = _rows(dout, "dout", routing.T, N, dout.dtype, dev)
    ys = N if y is None else _rows(y, "y", routing.rows, N, dout.dtype, dev)
    slots = _ints(routing.slots, "routing.slots", (routing.T, routing.k), dev)
    w = _weights(weights, routing, dev)
    dys = N if dy is None else _rows(dy, "dy", routing.rows, N, dout.dtype, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(combine_backward, other, (dout, y, routing.slots, weights, dy), dout, y, routing, weights, dy=dy)
    if dy is None:
        dy = dout.new_empty((routing.rows, N))
    dweights = None if y is None else dout.new_empty((routing.T, routing.k), dtype=torch.float32)
    _check(lib().gemm_rs_combine_backward(code, T, routing.rows, N, routing.k, dout.data_ptr(), ds, _ptr(y), ys, slots, w,
                                          dy.data_ptr(), dys, _ptr(dweights), _raw_stream(dev)), "gemm_rs_combine_backward")
    return dy, dweights
