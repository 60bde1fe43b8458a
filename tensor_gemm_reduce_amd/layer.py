"""ctypes binding of libgemm_rs_layer.so (include/gemm_rs_layer.h): the operators
around the row-parallel layer.

  w4_pack, w4_linear                  4-bit weights for a few tokens (decode)
  block_norm, block_norm_backward     slice sum, norms, gate and residual
  ckpt_pack, ckpt_unpack, ckpt_wgrad  activations kept in 8 bits, weight gradient

Argument checks and marshalling only: every step runs in the HIP kernels of the
library.  Tensors live on the current device; rows may be strided, elements of a
row are adjacent.  Work is enqueued on ``stream`` (a torch stream or a raw
handle; default: torch's current stream) and calls return at once; outputs
and workspaces come from torch's allocator on that stream.  The calls record no
history for autograd and refuse tensors that require gradients while gradients
are enabled; inside an autograd.Function they are not.

If the library is missing this module raises ImportError on first use: there is
no fallback path.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

from . import build as _build
from .gemm_rs import ERR_INVALID_ARG, ERR_UNSUPPORTED_SHAPE, OK  # noqa: F401

# ---- constants mirrored from include/gemm_rs_layer.h --------------------------
DTYPE_BF16 = 0
DTYPE_F16 = 1
DTYPE_F32 = 2
GATE_NONE = 0
GATE_CHANNEL = 1
GATE_TOKEN = 2
GATE_FULL = 3
NORM_MAX_PARTS = 8
NORM_MAX_WIDTH = 32768
CKPT_BLOCK = 32
CKPT_NAN = 127

EXPORTS = ("gemm_rs_layer_strerror", "gemm_rs_w4_validate", "gemm_rs_w4_packed_bytes", "gemm_rs_w4_pack",
           "gemm_rs_w4_linear", "gemm_rs_norm_validate", "gemm_rs_block_norm", "gemm_rs_block_norm_workspace",
           "gemm_rs_block_norm_backward", "gemm_rs_ckpt_pack", "gemm_rs_ckpt_unpack",
           "gemm_rs_ckpt_wgrad_plan", "gemm_rs_ckpt_wgrad_workspace", "gemm_rs_ckpt_wgrad")

_CODES = {torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16, torch.float32: DTYPE_F32}

_vp, _i32, _i64, _f32, _size = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t)


class gemm_rs_w4_config(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("N", "K", "group", "dtype", "zero_points")]


class gemm_rs_norm_config(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("width", "dtype", "residual_dtype", "parts", "gate", "post_norm", "pre_norm")] + [
        (n, _f32) for n in ("eps", "block_scale", "residual_scale")]


# The argument blocks as calls pack them (setting a ctypes field costs as much as packing a whole block).
_NORM_CONFIG = struct.Struct("7i3f")
_NORM_ARGS = struct.Struct(f"{NORM_MAX_PARTS}QqQqQQqQQqQqQqQ")
_NORM_GRAD_ARGS = struct.Struct("QqQqQqQqQQQQqQqQqQQQq")
_WGRAD_ARGS = struct.Struct("2i3qQqQQQqQq")


class gemm_rs_norm_args(ctypes.Structure):
    _fields_ = [("parts", _vp * NORM_MAX_PARTS), ("part_stride", _i64), ("residual", _vp), ("residual_stride", _i64),
                ("post_weight", _vp), ("gate", _vp), ("gate_stride", _i64), ("pre_weight", _vp), ("h", _vp),
                ("h_stride", _i64), ("z", _vp), ("z_stride", _i64), ("y", _vp), ("y_stride", _i64), ("rstd", _vp)]


class gemm_rs_norm_grad_args(ctypes.Structure):
    _fields_ = [("dz", _vp), ("dz_stride", _i64), ("dh", _vp), ("dh_stride", _i64), ("h", _vp), ("h_stride", _i64),
                ("y", _vp), ("y_stride", _i64), ("rstd", _vp), ("post_weight", _vp), ("gate", _vp),
                ("pre_weight", _vp), ("gate_stride", _i64), ("dresidual", _vp), ("dresidual_stride", _i64),
                ("dy", _vp), ("dy_stride", _i64), ("dpre_weight", _vp), ("dpost_weight", _vp), ("dgate", _vp),
                ("dgate_stride", _i64)]


class gemm_rs_wgrad_args(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("out_dtype", _i32), ("M", _i64), ("N", _i64), ("K", _i64), ("dy", _vp),
                ("dy_stride", _i64), ("q", _vp), ("exps", _vp), ("add", _vp), ("add_stride", _i64), ("dw", _vp),
                ("dw_stride", _i64)]


class gemm_rs_wgrad_info(ctypes.Structure):
    _fields_ = [(n, _i32) for n in ("words", "tile", "whole", "cut", "shares", "workgroups", "dealt", "join_waves")]


_LIB = None


def library_path() -> str:
    return _build.layer_library_path()


def lib():
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(
                f"{path} is missing: build it with `python -m tensor_gemm_reduce_amd.build` "
                "(there is no fallback implementation)")
        L = ctypes.CDLL(path)
        w4 = ctypes.POINTER(gemm_rs_w4_config)
        norm = wg = _vp  # a structure by reference, or its packed bytes
        L.gemm_rs_layer_strerror.argtypes = [ctypes.c_int]
        L.gemm_rs_layer_strerror.restype = ctypes.c_char_p
        L.gemm_rs_w4_validate.argtypes = [w4]
        L.gemm_rs_w4_packed_bytes.argtypes = [w4]
        L.gemm_rs_w4_pack.argtypes = [w4, _vp, _vp, _vp, _vp, _vp]
        L.gemm_rs_w4_linear.argtypes = [w4, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
        L.gemm_rs_norm_validate.argtypes = [norm]
        L.gemm_rs_block_norm.argtypes = [norm, _i64, _vp, _vp]
        L.gemm_rs_block_norm_workspace.argtypes = [norm, _i64]
        L.gemm_rs_block_norm_backward.argtypes = [norm, _i64, _vp, _vp, _size, _vp]
        L.gemm_rs_ckpt_pack.argtypes = [_i32, _i64, _i64, _vp, _i64, _vp, _vp, _vp]
        L.gemm_rs_ckpt_unpack.argtypes = [_i32, _i64, _i64, _vp, _vp, _vp, _i64, _vp]
        L.gemm_rs_ckpt_wgrad_plan.argtypes = [wg, ctypes.POINTER(gemm_rs_wgrad_info)]
        L.gemm_rs_ckpt_wgrad_workspace.argtypes = [wg]
        L.gemm_rs_ckpt_wgrad.argtypes = [wg, _vp, _size, _vp]
        for name in EXPORTS[1:]:
            getattr(L, name).restype = _size if name.endswith(("_bytes", "_workspace")) else ctypes.c_int
        _LIB = L
    return _LIB


class GemmRSLayerError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {lib().gemm_rs_layer_strerror(code).decode()} ({code})")


def _check(code: int, what: str) -> None:
    if code != OK:
        raise GemmRSLayerError(code, what)


# ---- argument checks ------------------------------------------------------------

_get_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)


_grad_mode = torch.is_grad_enabled  # looked up only where a tensor asks for gradients


def _lost_gradient(name):
    return RuntimeError(f"{name}: requires gradients, but the call records no history for autograd: pass it detached, or "
                        "call under torch.no_grad() (as inside an autograd.Function)")


def _device(t, name):
    """Index of the current device, which has to be t's."""
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name}: must be a device tensor")
    if d != _get_device():
        raise ValueError(f"{name}: on device {d}, but the current device is {_get_device()}")
    return d


def _rows(t, name, rows, width, dtype, dev):
    """Checks a [rows][width] tensor with adjacent row elements; returns its row stride."""
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != (rows, width):
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {(rows, width)}")
    s0, s1 = t.stride()
    if s1 != 1 and width != 1 or s0 < width and rows > 1:
        raise ValueError(f"{name}: rows must hold their elements side by side, strides are {(s0, s1)}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, not on the current device")
    if t.requires_grad and _grad_mode():
        raise _lost_gradient(name)
    return s0 if rows > 1 else max(s0, width)


def _flat(t, name, shape, dtype, dev):
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, not on the current device")
    if t.requires_grad and _grad_mode():
        raise _lost_gradient(name)


def _two(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected two dimensions, got shape {tuple(t.shape)}")
    return t.shape


def _elsewhere(stream, dev):
    """None, or the torch stream to switch to for a call whose `stream` is not the current one."""
    raw = stream if isinstance(stream, int) else stream.cuda_stream
    if raw == _raw_stream(dev):
        return None
    return torch.cuda.ExternalStream(raw, device=dev) if isinstance(stream, int) else stream


def _on_stream(call, stream, inputs, *args, **kw):
    """Runs call(...) with `stream` as torch's current stream, so that its outputs and
    workspace belong to that stream, and tells the allocator that the inputs are used there."""
    with torch.cuda.stream(stream):
        out = call(*args, **kw)
        for t in inputs:
            if t is not None:
                t.record_stream(stream)
    return out


# ---- 4-bit weights -----------------------------------------------------------------

class W4Weight:
    """Weights of w4_linear as w4_pack laid them out: w[n][k] = scale[n][k // group] (q[n][k] - zero[n][k // group])."""

    __slots__ = ("packed", "cfg", "ref", "N", "K", "group", "dtype")

    def __init__(self, packed, cfg, dtype):
        self.packed, self.cfg, self.dtype = packed, cfg, dtype
        self.ref = ctypes.byref(cfg)
        self.N, self.K, self.group = cfg.N, cfg.K, cfg.group


def w4_pack(q, scales, zeros=None, *, group, stream=None) -> W4Weight:
    """Lays 4-bit weights out for w4_linear, once.

    q: uint8 [N][K / 2], input k of a row in byte k // 2, even k in the low half;
    scales: bf16 or f16 [N][ceil(K / group)], also the type of x and y;
    zeros: uint8 of the scales' shape (0 .. 15), or None for 8 everywhere.
    group: a multiple of 32, or K.
    """
    N, half = _two(q, "q")
    if scales.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"scales: expected bfloat16 or float16, got {scales.dtype}")
    if max(N, 2 * half, abs(group)) >= 1 << 31:  # the structure would keep the low bits
        raise GemmRSLayerError(ERR_UNSUPPORTED_SHAPE, "w4_pack")
    cfg = gemm_rs_w4_config(N, 2 * half, group, _CODES[scales.dtype], int(zeros is not None))
    L = lib()
    _check(L.gemm_rs_w4_validate(ctypes.byref(cfg)), "gemm_rs_w4_validate")
    dev = _device(q, "q")
    shape = (N, -(-cfg.K // group))
    _flat(q, "q", (N, half), torch.uint8, dev)
    _flat(scales, "scales", shape, scales.dtype, dev)
    if zeros is not None:
        _flat(zeros, "zeros", shape, torch.uint8, dev)
    other = None if stream is None else _elsewhere(stream, dev)
    if other is not None:
        return _on_stream(w4_pack, other, (q, scales, zeros), q, scales, zeros, group=group)
    packed = q.new_empty(L.gemm_rs_w4_packed_bytes(ctypes.byref(cfg)))
    _check(L.gemm_rs_w4_pack(ctypes.byref(cfg), q.data_ptr(), scales.data_ptr(),
                             None if zeros is None else zeros.data_ptr(), packed.data_ptr(), _raw_stream(dev)),
           "gemm_rs_w4_pack")
    return W4Weight(packed, cfg, scales.dtype)


def w4_linear(x, weight: W4Weight, out=None, *, stream=None):
    """y = x w^T for x [M][K] (any M; made for few rows), FP32 accumulation, rounded once to x's type.

    An infinity or a NaN in a row of x makes that row of y NaN.
    """
    M, _ = _two(x, "x")
    N, dtype = weight.N, weight.dtype
    dev = _device(x, "x")
    xs = _rows(x, "x", M, weight.K, dtype, dev)
    if weight.packed.get_device() != dev:
        raise ValueError(f"weight: on {weight.packed.device}, not on the current device")
    ys = N if out is None else _rows(out, "out", M, N, dtype, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(w4_linear, other, (x, weight.packed, out), x, weight, out)
    if out is None:
        out = x.new_empty((M, N))
    _check(lib().gemm_rs_w4_linear(weight.ref, weight.packed.data_ptr(), M, x.data_ptr(), xs, out.data_ptr(), ys,
                                   _raw_stream(dev)), "gemm_rs_w4_linear")
    return out


# ---- block norm -----------------------------------------------------------------------

def _ptr(t):
    return 0 if t is None else t.data_ptr()


class BlockNorm:
    """Outputs of block_norm: h, z (None without a pre weight), and with save=True y and rstd."""

    __slots__ = ("h", "z", "y", "rstd")

    def __init__(self, h, z, y, rstd):
        self.h, self.z, self.y, self.rstd = h, z, y, rstd


class BlockNormGrads:
    """Gradients from block_norm_backward; None for what the forward pass did not have."""

    __slots__ = ("residual", "y", "pre_weight", "post_weight", "gate")

    def __init__(self, residual, y, pre_weight, post_weight, gate):
        self.residual, self.y, self.pre_weight, self.post_weight, self.gate = residual, y, pre_weight, post_weight, gate


def _gate(gate, S, N, dtype, dev):
    """(kind, row stride) of a gate: [N] for every row, [S][1] per row or [S][N]."""
    if gate.dim() == 1:
        _flat(gate, "gate", (N,), dtype, dev)
        return GATE_CHANNEL, 0
    if gate.shape == (S, 1) and N != 1:
        _flat(gate, "gate", (S, 1), dtype, dev)
        return GATE_TOKEN, 0
    return GATE_FULL, _rows(gate, "gate", S, N, dtype, dev)


def _weight(t, name, N, dtype, dev):
    if t is None:
        return 0
    _flat(t, name, (N,), dtype, dev)
    return t.data_ptr()


def _parts(parts, dev):
    """(a tensor of them, S, N, pointers, row stride) of a [S][N] tensor, a list of them or a [P][S][N] tensor."""
    if isinstance(parts, torch.Tensor):
        if parts.dim() == 2:
            S, N = parts.shape
            return parts, S, N, (parts.data_ptr(),), _rows(parts, "parts", S, N, parts.dtype, dev)
        if parts.dim() != 3 or not 1 <= parts.shape[0] <= NORM_MAX_PARTS:
            raise ValueError(f"parts: [S][N], or 1 to {NORM_MAX_PARTS} of them, got shape {tuple(parts.shape)}")
        P, S, N = parts.shape
        s0, s1, s2 = parts.stride()
        if s2 != 1 and N != 1 or s1 < N and S > 1:
            raise ValueError(f"parts: rows must hold their elements side by side, strides are {(s0, s1, s2)}")
        if parts.requires_grad and _grad_mode():
            raise _lost_gradient("parts")
        step, base = s0 * parts.element_size(), parts.data_ptr()
        return parts, S, N, range(base, base + P * step, step) if step > 0 else [base] * P, s1 if S > 1 else max(s1, N)
    if not 1 <= len(parts) <= NORM_MAX_PARTS:
        raise ValueError(f"parts: 1 to {NORM_MAX_PARTS}, got {len(parts)}")
    first = parts[0]
    S, N = _two(first, "parts[0]")
    strides = [_rows(p, f"parts[{i}]", S, N, first.dtype, dev) for i, p in enumerate(parts)]
    if strides != strides[:1] * len(parts):
        raise ValueError(f"parts: row strides differ: {strides}")
    return first, S, N, [p.data_ptr() for p in parts], strides[0]


_NO_PARTS = tuple((0,) * (NORM_MAX_PARTS - n) for n in range(NORM_MAX_PARTS + 1))


def block_norm(parts, residual=None, *, pre_weight=None, post_weight=None, gate=None, block_scale=1.0,
               residual_scale=1.0, eps=1e-5, save=False, h=None, z=None, stream=None) -> BlockNorm:
    """What follows the row-parallel layer, in one pass over each row (FP32, one rounding per output):

      y = sum of the parts;  u = y / rms(y) * post_weight (y itself without a post weight)
      h = residual_scale * residual + block_scale * gate * u
      z = h / rms(h) * pre_weight (no z without a pre weight),  rms(t) = sqrt(mean(t^2) + eps)

    parts: a [S][N] tensor, a list of 1 .. 8 of them, or a [P][S][N] tensor: the ranks' partials in the order they
    are added.  residual and h: parts' type or float32 (h has the residual's type; parts' without one).
    gate: [N], [S][1] or [S][N].  h may be the residual itself, to update it in place.
    save=True also returns y and rstd ([2][S] float32: 1 / rms(y), 1 / rms(h)) for block_norm_backward.
    """
    if not isinstance(parts, torch.Tensor) and not parts:
        raise ValueError(f"parts: 1 to {NORM_MAX_PARTS}, got none")
    dev = _device(parts if isinstance(parts, torch.Tensor) else parts[0], "parts")
    first, S, N, pointers, part_stride = _parts(parts, dev)
    dtype = first.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"parts: expected bfloat16, float16 or float32, got {dtype}")
    rdtype, residual_ptr, residual_stride = dtype, 0, 0
    if residual is not None:
        rdtype = residual.dtype
        if rdtype is not dtype and rdtype is not torch.float32:
            raise TypeError(f"residual: expected {dtype} or float32, got {rdtype}")
        residual_ptr, residual_stride = residual.data_ptr(), _rows(residual, "residual", S, N, rdtype, dev)
    elif h is not None and h.dtype is torch.float32:
        rdtype = torch.float32
    kind = gate_ptr = gate_stride = 0
    if gate is not None:
        kind, gate_stride = _gate(gate, S, N, dtype, dev)
        gate_ptr = gate.data_ptr()
    pre, post = _weight(pre_weight, "pre_weight", N, dtype, dev), _weight(post_weight, "post_weight", N, dtype, dev)
    h_stride = N if h is None else _rows(h, "h", S, N, rdtype, dev)
    z_stride = N if z is None else _rows(z, "z", S, N, dtype, dev)
    if z is not None and pre_weight is None:
        raise ValueError("z: needs a pre_weight")
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            used = [parts] if isinstance(parts, torch.Tensor) else list(parts)
            return _on_stream(block_norm, other, used + [residual, gate, pre_weight, post_weight, h, z], parts, residual,
                              pre_weight=pre_weight, post_weight=post_weight, gate=gate, block_scale=block_scale,
                              residual_scale=residual_scale, eps=eps, save=save, h=h, z=z)
    if h is None:
        h = first.new_empty((S, N)) if rdtype is dtype else first.new_empty((S, N), dtype=rdtype)
    z_ptr = y_ptr = rstd_ptr = 0
    y = rstd = None
    if pre_weight is not None:
        if z is None:
            z = first.new_empty((S, N))
        z_ptr = z.data_ptr()
    if save:
        y, rstd = first.new_empty((S, N)), first.new_empty((2, S), dtype=torch.float32)
        y_ptr, rstd_ptr = y.data_ptr(), rstd.data_ptr()
    n = len(pointers)
    cfg = _NORM_CONFIG.pack(N, code, _CODES[rdtype], n, kind, post_weight is not None, pre_weight is not None, eps,
                            block_scale, residual_scale)
    args = _NORM_ARGS.pack(*pointers, *_NO_PARTS[n], part_stride, residual_ptr, residual_stride, post, gate_ptr,
                           gate_stride, pre, h.data_ptr(), h_stride, z_ptr, z_stride, y_ptr, N, rstd_ptr)
    _check(lib().gemm_rs_block_norm(cfg, S, args, _raw_stream(dev)), "gemm_rs_block_norm")
    return BlockNorm(h, z, y, rstd)


def block_norm_backward(dz, dh, h, y, rstd, *, pre_weight=None, post_weight=None, gate=None, block_scale=1.0,
                        residual_scale=1.0, stream=None) -> BlockNormGrads:
    """Gradients of block_norm's inputs from dz (None without a pre weight) and dh (None: zero).

    h, y, rstd: what block_norm(save=True) returned; h is only read with a pre weight, y only with a post weight or a
    gate (either may then be None, but dz or y is needed for the parts' type).  Every part's gradient is .y.  Weight and [N]-gate gradients are float32, sums over
    rows in a fixed order; .residual has the residual's type.
    """
    like = dz if dz is not None else y
    if like is None:
        raise ValueError("dz or y is needed")
    if dz is not None and pre_weight is None:
        raise ValueError("dz: needs a pre_weight")
    name = "dz" if dz is not None else "y"
    S, N = _two(like, name)
    dev = _device(like, name)
    dtype = like.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name}: expected bfloat16, float16 or float32, got {dtype}")
    stream_of = dh if dh is not None else h
    rdtype = dtype if stream_of is None else stream_of.dtype
    if rdtype is not dtype and rdtype is not torch.float32:
        raise TypeError(f"dh, h: expected {dtype} or float32, got {rdtype}")
    kind = gate_ptr = gate_stride = 0
    if gate is not None:
        kind, gate_stride = _gate(gate, S, N, dtype, dev)
        gate_ptr = gate.data_ptr()
    pre, post = _weight(pre_weight, "pre_weight", N, dtype, dev), _weight(post_weight, "post_weight", N, dtype, dev)
    dz_ptr = dz_stride = h_ptr = h_stride = y_ptr = y_stride = dh_ptr = dh_stride = rstd_ptr = 0
    if pre_weight is not None:
        if dz is None or h is None:
            raise ValueError("a pre_weight needs dz and h")
        dz_ptr, dz_stride = dz.data_ptr(), _rows(dz, "dz", S, N, dtype, dev)
        h_ptr, h_stride = h.data_ptr(), _rows(h, "h", S, N, rdtype, dev)
    if post_weight is not None or gate is not None:
        if y is None:
            raise ValueError("a post_weight or a gate needs y")
        y_ptr, y_stride = y.data_ptr(), _rows(y, "y", S, N, dtype, dev)
    if pre_weight is not None or post_weight is not None:
        if rstd is None:
            raise ValueError("a pre_weight or post_weight needs rstd")
        _flat(rstd, "rstd", (2, S), torch.float32, dev)
        rstd_ptr = rstd.data_ptr()
    if dh is not None:
        dh_ptr, dh_stride = dh.data_ptr(), _rows(dh, "dh", S, N, rdtype, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(block_norm_backward, other, (dz, dh, h, y, rstd, pre_weight, post_weight, gate), dz, dh, h,
                              y, rstd, pre_weight=pre_weight, post_weight=post_weight, gate=gate,
                              block_scale=block_scale, residual_scale=residual_scale)
    new = like.new_empty
    dy = new((S, N))
    dres = new((S, N)) if rdtype is dtype else new((S, N), dtype=rdtype)
    dpre = new(N, dtype=torch.float32) if pre else None
    dpost = new(N, dtype=torch.float32) if post else None
    dgate = None
    if kind == GATE_CHANNEL:
        dgate = new(N, dtype=torch.float32)
    elif kind != GATE_NONE:
        dgate = new(gate.shape)
    cfg = _NORM_CONFIG.pack(N, code, _CODES[rdtype], 1, kind, post_weight is not None, pre_weight is not None, 0.0,
                            block_scale, residual_scale)
    args = _NORM_GRAD_ARGS.pack(dz_ptr, dz_stride, dh_ptr, dh_stride, h_ptr, h_stride, y_ptr, y_stride, rstd_ptr, post,
                                gate_ptr, pre, gate_stride, dres.data_ptr(), N, dy.data_ptr(), N, _ptr(dpre),
                                _ptr(dpost), _ptr(dgate), N)
    L = lib()
    size = L.gemm_rs_block_norm_workspace(cfg, S)
    ws = new(size // 4, dtype=torch.float32) if size else None
    _check(L.gemm_rs_block_norm_backward(cfg, S, args, _ptr(ws), size, _raw_stream(dev)), "gemm_rs_block_norm_backward")
    return BlockNormGrads(dres, dy, dpre, dpost, dgate)


# ---- 8-bit checkpoints -----------------------------------------------------------------

class Checkpoint:
    """An activation [M][K] kept in 8 bits: q int8 [M][K rounded up to 32], exps int8 [M][that / 32], and the type it
    had.  A block of 32 columns stands for q 2^exp (exp 127: the block held an infinity or a NaN, and stands for NaN)."""

    __slots__ = ("q", "exps", "K", "dtype")

    def __init__(self, q, exps, K, dtype):
        blocks = -(-K // CKPT_BLOCK)
        M, _ = _two(q, "q")
        if dtype not in _CODES:
            raise TypeError(f"dtype: expected bfloat16, float16 or float32, got {dtype}")
        dev = q.get_device()
        _flat(q, "q", (M, blocks * CKPT_BLOCK), torch.int8, dev)
        _flat(exps, "exps", (M, blocks), torch.int8, dev)
        self.q, self.exps, self.K, self.dtype = q, exps, K, dtype


def ckpt_pack(x, *, stream=None) -> Checkpoint:
    """Keeps x [M][K] (bfloat16, float16 or float32) in 8 bits: round(x 2^-e) with e = floor(log2(max |x|)) - 6 for
    every 32 columns of a row."""
    M, K = _two(x, "x")
    dtype = x.dtype
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"x: expected bfloat16, float16 or float32, got {dtype}")
    if K < 1:
        raise ValueError("x: needs at least one column")
    dev = _device(x, "x")
    xs = _rows(x, "x", M, K, dtype, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(ckpt_pack, other, (x,), x)
    blocks = -(-K // CKPT_BLOCK)
    q = x.new_empty((M, blocks * CKPT_BLOCK), dtype=torch.int8)
    exps = q.new_empty((M, blocks))
    _check(lib().gemm_rs_ckpt_pack(code, M, K, x.data_ptr(), xs, q.data_ptr(), exps.data_ptr(), _raw_stream(dev)),
           "gemm_rs_ckpt_pack")
    kept = Checkpoint.__new__(Checkpoint)
    kept.q, kept.exps, kept.K, kept.dtype = q, exps, K, dtype
    return kept


def ckpt_unpack(kept: Checkpoint, out=None, *, stream=None):
    """The values a checkpoint stands for, in the type it was made from."""
    q, K = kept.q, kept.K
    M = q.shape[0]
    dev = _device(q, "checkpoint")
    xs = K if out is None else _rows(out, "out", M, K, kept.dtype, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(ckpt_unpack, other, (q, kept.exps, out), kept, out)
    if out is None:
        out = q.new_empty((M, K), dtype=kept.dtype)
    _check(lib().gemm_rs_ckpt_unpack(_CODES[kept.dtype], M, K, q.data_ptr(), kept.exps.data_ptr(), out.data_ptr(), xs,
                                     _raw_stream(dev)), "gemm_rs_ckpt_unpack")
    return out


def ckpt_wgrad(dy, kept: Checkpoint, *, add=None, out=None, dtype=torch.float32, stream=None):
    """The weight gradient dw [N][K] = dy^T x^ (+ add) of a linear layer whose input was kept as `kept`.

    dy: [M][N] bfloat16 or float16 (float16 needs a checkpoint of a float16 activation).  add: float32 [N][K] or None.
    dtype: float32 or dy's (out's, if given).  out may be `add` (float32): gradients accumulated in place.
    """
    M, N = _two(dy, "dy")
    dev = _device(dy, "dy")
    ydtype, q, K = dy.dtype, kept.q, kept.K
    if ydtype is not torch.bfloat16 and ydtype is not torch.float16:
        raise TypeError(f"dy: expected bfloat16 or float16, got {ydtype}")
    if ydtype is torch.float16 and kept.dtype is not torch.float16:
        raise TypeError(f"dy: float16 with a checkpoint of {kept.dtype}")
    if q.shape[0] != M:
        raise ValueError(f"dy has {M} rows, the checkpoint {q.shape[0]}")
    if q.get_device() != dev:
        raise ValueError(f"checkpoint: on {q.device}, not on the current device")
    if out is not None:
        dtype = out.dtype
    if dtype is not torch.float32 and dtype is not ydtype:
        raise TypeError(f"dtype: expected float32 or {ydtype}, got {dtype}")
    ys = _rows(dy, "dy", M, N, ydtype, dev)
    add_stride = 0 if add is None else _rows(add, "add", N, K, torch.float32, dev)
    out_stride = K if out is None else _rows(out, "out", N, K, dtype, dev)
    if stream is not None:
        other = _elsewhere(stream, dev)
        if other is not None:
            return _on_stream(ckpt_wgrad, other, (dy, q, kept.exps, add, out), dy, kept, add=add, out=out, dtype=dtype)
    if out is None:
        out = dy.new_empty((N, K)) if dtype is ydtype else dy.new_empty((N, K), dtype=dtype)
    args = _WGRAD_ARGS.pack(_CODES[ydtype], _CODES[dtype], M, N, K, dy.data_ptr(), ys, q.data_ptr(),
                            kept.exps.data_ptr(), _ptr(add), add_stride, out.data_ptr(), out_stride)
    L = lib()
    size = L.gemm_rs_ckpt_wgrad_workspace(args)
    ws = q.new_empty(size) if size else None
    _check(L.gemm_rs_ckpt_wgrad(args, _ptr(ws), size, _raw_stream(dev)), "gemm_rs_ckpt_wgrad")
    return out
