"""ctypes binding of the operators between a prompt and its next token (argument
marshalling only).

q8_rows and q8_matmul over a Q8Matrix (projections in 8-bit integers), route_experts
with a RoutingRule (also taken by MoECache.forward), and sample_tokens.  The formulas
and layouts are set out in include/moe_cache.h.  Tensors are torch tensors on one GPU;
devices and streams are as in `decoder`.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from .binding import RouteRule, _check, load_library
from .decoder import _I32, _TYPES, _At, _cuda, _elsewhere, _raw_stream, _rows, _weight

_PAD = 128  # zero codes up to a multiple of this end a row in 8 bits
_SCORES = {"softmax": 0, "sigmoid": 1}


class _SampleOpts(ctypes.Structure):
    _fields_ = [(n, ctypes.c_double) for n in ("temperature", "top_p", "min_p")] + [("top_k", ctypes.c_int32)] + \
               [(n, ctypes.c_void_p) for n in ("temperatures", "top_ps", "min_ps", "top_ks")]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        P, I32, I64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        sig = {
            "moe_q8_rows": (I32, [P, I32, I64, I32, I32, P, I64, P, P]),
            "moe_q8_matmul": (I32, [P, I64, P, I32, P, I64, P, I32, I32, P, I32, I64, P]),
            "moe_q8_linear_workspace": (I64, [I32, I32, I32]),
            "moe_q8_linear": (I32, [P, I32, I64, I32, P, I64, P, I32, I32, P, I32, I64, P, I64, P]),
            "moe_route": (I32, [P, I32, I64, P, I32, I32, ctypes.POINTER(RouteRule), P, P, P]),
            "moe_sample_workspace": (I64, [I32, I32]),
            "moe_sample": (I32, [P, I32, I64, I32, I32, P, ctypes.POINTER(_SampleOpts), P, P, P, I64, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


class Q8Rows:
    """Rows in 8-bit integers: codes int8 [n, cols rounded up to 128] (zeros past cols) and
    scales float32 [n], as q8_rows makes them.  values() gives what they stand for."""

    def __init__(self, codes, scales, cols: int):
        dev = _cuda(codes, "codes")
        if codes.dtype != torch.int8 or codes.dim() != 2 or not codes.is_contiguous() or cols < 1 or \
                codes.shape[1] != -(-cols // _PAD) * _PAD:
            raise ValueError("codes must be contiguous int8 [n, cols rounded up to 128]")
        if scales.get_device() != dev or scales.dtype != torch.float32 or scales.shape != (codes.shape[0],) or \
                not scales.is_contiguous():
            raise ValueError("scales must be contiguous float32 [n] beside the codes")
        self.codes, self.scales, self.cols = codes, scales, cols
        self._index = dev

    def values(self):
        """float32 [n, cols]."""
        return self.codes[:, :self.cols].float() * self.scales.unsqueeze(1)


def q8_rows(x, stream=None) -> Q8Rows:
    """The rows of x [n, cols] (float32, bfloat16 or float16) in 8-bit integers with a scale
    each: max|x| / 127 and rint(x / scale).  Worth its own call where several matrices take
    the same x."""
    dev = _cuda(x, "x")
    if _elsewhere(dev, stream):
        with _At(dev, stream, x):
            return q8_rows(x)
    ldx = _rows(x, "x", dev)
    n, cols = x.shape
    padded = -(-cols // _PAD) * _PAD
    codes = torch.empty((n, padded), dtype=torch.int8, device=x.device)
    scales = torch.empty(n, dtype=torch.float32, device=x.device)
    rc = _library().moe_q8_rows(x.data_ptr(), _TYPES[x.dtype], ldx, n, cols, codes.data_ptr(), padded,
                                scales.data_ptr(), _raw_stream(dev))
    if rc:
        _check(rc)
    return Q8Rows(codes, scales, cols)


class Q8Matrix:
    """A matrix [rows, cols] in 8-bit integers on the GPU: codes int8 [rows, cols] with
    contiguous rows, scales float32 [rows] (contiguous).  Both are kept, not copied, where
    a row of codes starts every multiple of 16 bytes; else the codes are copied once into
    rows that do."""

    def __init__(self, codes, scales):
        dev = _cuda(codes, "codes")
        if codes.dtype != torch.int8 or codes.dim() != 2 or codes.shape[0] < 1 or codes.shape[1] < 1 or \
                (codes.shape[1] > 1 and codes.stride(1) != 1):
            raise ValueError("codes must be int8 [rows, cols] with contiguous rows")
        self.rows, self.cols = codes.shape
        if self.rows >= 1 << 24 or self.cols > 131072:
            raise ValueError("a matrix holds fewer than 2^24 rows, of at most 131072 columns")
        if scales.get_device() != dev or scales.dtype != torch.float32 or scales.shape != (self.rows,) or \
                not scales.is_contiguous():
            raise ValueError("scales must be contiguous float32 [rows] beside the codes")
        if codes.data_ptr() % 16 or self.cols % 16 or (
                self.rows > 1 and (codes.stride(0) % 16 or not self.cols <= codes.stride(0) <= 1 << 22)):
            with torch.cuda.device(dev):
                laid = torch.zeros((self.rows, -(-self.cols // 16) * 16), dtype=torch.int8, device=codes.device)
                laid[:, :self.cols] = codes
            codes = laid
        self.codes, self.scales, self.device = codes, scales, codes.device
        self._index = dev
        self._head = (codes.data_ptr(), codes.stride(0), scales.data_ptr(), self.rows, self.cols)

    @classmethod
    def from_weights(cls, w, stream=None):
        """From w [rows, cols] (float32, bfloat16 or float16): a scale per row, its output
        channel, as q8_rows gives it."""
        q = q8_rows(w, stream)
        m = cls(q.codes, q.scales)
        m.cols = q.cols
        m._head = m._head[:4] + (q.cols,)
        return m


def q8_matmul(x, w: Q8Matrix, out=None, dtype: Optional[torch.dtype] = None, stream=None):
    """out [T, rows] = x times w transposed.  x is [T, cols] (float32, bfloat16 or float16),
    rounded to 8 bits with a scale per row on the way, or Q8Rows of cols columns.  The sums
    of products are exact; out is of `dtype` (default: x's, float32 for Q8Rows)."""
    dev = w._index
    rows8 = isinstance(x, Q8Rows)
    if _elsewhere(dev, stream):
        with _At(dev, stream, *((x.codes, x.scales) if rows8 else (x,)), w.codes, w.scales, out):
            return q8_matmul(x, w, out, dtype)
    if rows8:
        if x._index != dev or x.cols != w.cols:
            raise ValueError(f"x must hold rows of {w.cols} columns on cuda:{dev}")
        T, dt = x.codes.shape[0], torch.float32
    else:
        ldx = _rows(x, "x", dev, None, w.cols)
        T, dt = x.shape[0], x.dtype
    if T > 1 << 20:
        raise ValueError("x holds more than 2^20 rows")
    if out is None:
        dt = dtype or dt
        if dt not in _TYPES:
            raise ValueError("dtype must be float32, bfloat16 or float16")
        out = w.scales.new_empty((T, w.rows), dtype=dt)
        ldo = w.rows
    else:
        ldo = _rows(out, "out", dev, T, w.rows, dtype)
        dt = out.dtype
    lib = _library()
    wp, ldw, sp, rows, cols = w._head
    if rows8:
        rc = lib.moe_q8_matmul(x.codes.data_ptr(), x.codes.shape[1], x.scales.data_ptr(), T, wp, ldw, sp, rows, cols,
                               out.data_ptr(), _TYPES[dt], ldo, _raw_stream(dev))
    else:
        need = T * (-(-cols // _PAD) * _PAD + 4)  # as moe_q8_linear_workspace says
        ws = w.codes.new_empty(need) if need else None
        rc = lib.moe_q8_linear(x.data_ptr(), _TYPES[x.dtype], ldx, T, wp, ldw, sp, rows, cols, out.data_ptr(),
                               _TYPES[dt], ldo, ws.data_ptr() if need else None, need, _raw_stream(dev))
    if rc:
        _check(rc)
    return out


class RoutingRule:
    """How experts are selected from a router's logits: scores ("softmax" or "sigmoid"), a
    bias given with the call that takes part in the selection alone, `groups` of
    consecutive experts of which the `keep_groups` best are kept (by their best expert, or
    by the sum of their best two), the top_k best experts of those, weights renormalised
    over them (renorm) and multiplied by `scale`."""

    def __init__(self, top_k: int, score: str = "softmax", groups: int = 1, keep_groups: Optional[int] = None,
                 group_best: int = 1, renorm: bool = True, scale: float = 1.0):
        if score not in _SCORES:
            raise ValueError("score must be 'softmax' or 'sigmoid'")
        if not 1 <= top_k <= 64:
            raise ValueError("top_k must be in [1, 64]")
        keep = groups if keep_groups is None else keep_groups
        for name, v in (("keep_groups", keep), ("groups", groups), ("group_best", group_best)):
            if not -_I32 <= v <= _I32:  # (their ranges are checked with the experts they are for)
                raise ValueError(f"{name} must be a 32-bit number")
        self._c = RouteRule(top_k, _SCORES[score], groups, keep, group_best, 1 if renorm else 0, scale)
        self._cp = ctypes.pointer(self._c)

    @property
    def top_k(self) -> int:
        return self._c.top_k


def route_experts(logits, rule: RoutingRule, bias=None, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(idx int32 [T, top_k], weights float32 [T, top_k]) of logits [T, n_experts]; bias
    float32 [n_experts] or None."""
    dev = _cuda(logits, "logits")
    if _elsewhere(dev, stream):
        with _At(dev, stream, logits, bias):
            return route_experts(logits, rule, bias)
    ld = _rows(logits, "logits", dev)
    T, E = logits.shape
    bp = None if bias is None else _weight(bias, "bias", dev, E)
    k = rule._c.top_k
    idx, w = logits.new_empty((T, k), dtype=torch.int32), logits.new_empty((T, k), dtype=torch.float32)
    rc = _library().moe_route(logits.data_ptr(), _TYPES[logits.dtype], ld, bp, T, E, rule._cp, idx.data_ptr(),
                              w.data_ptr(), _raw_stream(dev))
    if rc:
        _check(rc)
    return idx, w


def _setting(v, name, dev, rows, dtype, keep):
    """(the call's value, the rows' pointer)."""
    if not torch.is_tensor(v):
        return v, None
    if v.get_device() != dev or v.dtype != dtype or v.shape != (rows,) or not v.is_contiguous():
        raise ValueError(f"{name} must be a number or contiguous {dtype} [{rows}] on cuda:{dev}")
    return keep, v.data_ptr()


def sample_tokens(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None) \
        -> Tuple[torch.Tensor, torch.Tensor]:
    """(tokens int32 [T], probabilities float32 [T]) drawn from logits [T, vocab] with the
    random numbers u float32 [T] in [0, 1).  Each setting is a number, or a tensor with one
    per row (float32; top_k int32).  temperature 0 takes the likeliest token, top_k 0,
    top_p 1 and min_p 0 keep all.  A row whose logits are all minus infinity (or NaN) gives
    token -1 with probability 0."""
    dev = _cuda(logits, "logits")
    if _elsewhere(dev, stream):
        with _At(dev, stream, logits, u, *(v for v in (temperature, top_k, top_p, min_p) if torch.is_tensor(v))):
            return sample_tokens(logits, u, temperature, top_k, top_p, min_p)
    ld = _rows(logits, "logits", dev)
    T, V = logits.shape
    up = _weight(u, "u", dev, T)
    f32 = torch.float32
    t0, tp = _setting(temperature, "temperature", dev, T, f32, 1.0)
    k0, kp = _setting(top_k, "top_k", dev, T, torch.int32, 0)
    p0, pp = _setting(top_p, "top_p", dev, T, f32, 1.0)
    m0, mp = _setting(min_p, "min_p", dev, T, f32, 0.0)
    if not 0 <= k0 <= _I32:
        raise ValueError("top_k must be in [0, 2^31)")
    opts = _SampleOpts(t0, p0, m0, k0, tp, pp, mp, kp)
    token, prob = u.new_empty(T, dtype=torch.int32), u.new_empty(T)
    lib = _library()
    need = lib.moe_sample_workspace(T, V)
    if need < 0:
        _check(need)
    ws = u.new_empty(need, dtype=torch.uint8) if need else None
    rc = lib.moe_sample(logits.data_ptr(), _TYPES[logits.dtype], ld, T, V, up, opts, token.data_ptr(), prob.data_ptr(),
                        ws.data_ptr() if need else None, need, _raw_stream(dev))
    if rc:
        _check(rc)
    return token, prob
