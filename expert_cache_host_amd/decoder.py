"""ctypes binding of the decoder-layer operators (argument marshalling only).

block_norm, q4_matvec over a Q4Matrix, and KVCache.append / attend / read: what a
decoder layer needs around the routed MoE layer.  The formulas and layouts are
set out in include/moe_cache.h.  Tensors are torch tensors on one GPU; calls go
to the given stream, or to the current stream of that GPU; they record no gradients.
A given stream is not made to wait for the current one: the caller orders it behind
the work that fills the inputs.  Tensors given to such a call may be dropped at once;
what it allocates belongs to the given stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import numpy as np
import torch

from .binding import _check, load_library

_I32 = 0x7fffffff  # sizes and counts are 32-bit integers at the C interface
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


class _KvCache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_codes", "k_scales", "v_codes", "v_scales")] + \
               [(n, ctypes.c_int32) for n in ("n_pages", "page_tokens", "kv_heads", "head_dim")]


class _KvBatch(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("pages", "start", "past")] + \
               [(n, ctypes.c_int32) for n in ("n_seqs", "max_pages", "n_rows")]


_lib = None


def _library():
    global _lib
    if _lib is None:
        lib = load_library()
        P, I32, I64, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
        C, B = ctypes.POINTER(_KvCache), ctypes.POINTER(_KvBatch)
        sig = {
            "moe_block_norm": (I32, [P, I32, I64, P, I32, I64, P, P, I32, I64, P, I32, I32, F, F, F,
                                     P, I64, P, I32, I64, P]),
            "moe_q4_matvec": (I32, [P, P, I32, I32, I32, P, I32, I64, I32, P, I64, P]),
            "moe_kv_append": (I32, [C, B, I32, P, I64, P, I64, P, I32, I32, P, I64, I32, P, I64, P]),
            "moe_kv_read": (I32, [C, B, P, P, P]),
            "moe_kv_attend_workspace": (I64, [C, B, I32, I32, I32]),
            "moe_kv_attend": (I32, [C, B, I32, P, I64, I32, F, I32, P, I64, P, I64, P]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


# the current stream's handle by device index (a Stream object costs a microsecond)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


class _At:
    """Makes a device and a stream current, so that the launch and what the call allocates
    belong to them; the stream's use of `tensors` is recorded, so that their memory is not
    given out again before the call has run."""

    def __init__(self, index, stream, *tensors):
        self.guards = [torch.cuda.device(index)]
        self.stream, self.tensors = stream, tensors
        if stream is not None:
            if stream.device.index != index:
                raise ValueError(f"the stream is on {stream.device}, the tensors on cuda:{index}")
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        if self.stream is not None and exc[0] is None:
            for t in self.tensors:
                if t is not None:
                    t.record_stream(self.stream)
        for g in reversed(self.guards):
            g.__exit__(*exc)
        return False


def _elsewhere(index, stream):
    """Whether the call must make its device or stream current first."""
    return stream is not None or torch.cuda.current_device() != index


def _fault(t, name, index, rows, d, dtype):
    if t.get_device() != index:
        return f"{name} is on {t.device}, not on cuda:{index}"
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (d is not None and t.shape[1] != d):
        return f"{name} must be [{'rows' if rows is None else rows}, {'d' if d is None else d}], not {list(t.shape)}"
    if t.shape[1] > 1 and t.stride(1) != 1:
        return f"{name}'s rows must be contiguous"
    if max(t.shape) > _I32:
        return f"{name} has more than 2^31 - 1 rows or columns"
    if dtype is None:
        return f"{name} must be float32, bfloat16 or float16"
    return f"{name} must be {dtype}"


def _rows(t, name, index, rows=None, d=None, dtype=None):
    """Checks a [rows, d] tensor with contiguous rows; returns its row stride."""
    shape = t.shape
    if t.get_device() == index and len(shape) == 2 and (rows is None or shape[0] == rows) and \
            (d is None or shape[1] == d) and (t.dtype in _TYPES if dtype is None else t.dtype == dtype):
        st = t.stride()
        if (st[1] == 1 or shape[1] <= 1) and shape[0] <= _I32 and shape[1] <= _I32:
            return st[0]
    raise ValueError(_fault(t, name, index, rows, d, dtype))


def _cuda(t, name):
    i = t.get_device()
    if i < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    return i


def _weight(w, name, index, d):
    if w.get_device() != index or w.dtype != torch.float32 or w.shape != (d,) or not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32 [{d}] on cuda:{index}")
    return w.data_ptr()


def block_norm(h, y=None, post_w=None, gate=None, pre_w=None, *, res_scale: float = 1.0,
               block_scale: float = 1.0, eps: float = 1e-6, h_out=None, x_out=None,
               x_dtype: Optional[torch.dtype] = None, stream=None):
    """(h', x): a block's residual update and the norm before the next block.

        n  = y / sqrt(mean(y^2) + eps) * post_w        (post_w None: n = y)
        h' = res_scale * h + block_scale * gate * n    (y None: res_scale * h)
        x  = h' / sqrt(mean(h'^2) + eps) * pre_w       (pre_w None: x is None)

    h [T, d], y [T, d], gate [d] or [T, d], post_w and pre_w float32 [d].  h' has h's
    type, x `x_dtype` (default: y's type, else h's).  h_out may be h, x_out may be y.
    With y None and res_scale 1, h' is h itself, returned without a copy unless
    h_out is given.
    """
    dev = _cuda(h, "h")
    if _elsewhere(dev, stream):
        with _At(dev, stream, h, y, post_w, gate, pre_w, h_out, x_out):
            return block_norm(h, y, post_w, gate, pre_w, res_scale=res_scale, block_scale=block_scale, eps=eps,
                              h_out=h_out, x_out=x_out, x_dtype=x_dtype)
    ldh = _rows(h, "h", dev)
    T, d = h.shape
    hd = xd = h.dtype
    yp = gp = wp = vp = hp = xp = None
    ldy = yt = ldg = gt = ldho = ldx = xt = 0
    if y is not None:
        ldy = _rows(y, "y", dev, T, d)
        xd = y.dtype
        yt = _TYPES[xd]
        yp = y.data_ptr()
        if gate is not None:
            gt = _TYPES.get(gate.dtype)
            if gate.dim() != 1:
                ldg = _rows(gate, "gate", dev, T, d)
            elif gate.get_device() != dev or gt is None or gate.shape != (d,) or not gate.is_contiguous():
                raise ValueError("gate must be [d] or have h's rows, beside h, float32, bfloat16 or float16")
            gp = gate.data_ptr()
        if post_w is not None:
            wp = _weight(post_w, "post_w", dev, d)
    elif post_w is not None or gate is not None:
        raise ValueError("post_w and gate need y")
    if pre_w is not None:
        vp = _weight(pre_w, "pre_w", dev, d)
    elif x_out is not None:
        raise ValueError("x_out needs pre_w")
    keep = y is None and res_scale == 1.0 and h_out is None
    if keep and pre_w is None:
        raise ValueError("nothing to compute: y and pre_w are None")
    if h_out is not None:
        ldho = _rows(h_out, "h_out", dev, T, d, hd)
        hp = h_out.data_ptr()
    elif not keep:
        h_out = h.new_empty((T, d))
        ldho, hp = d, h_out.data_ptr()
    if x_out is not None:
        ldx = _rows(x_out, "x_out", dev, T, d, x_dtype)
        xt, xp = _TYPES[x_out.dtype], x_out.data_ptr()
    elif pre_w is not None:
        xd = x_dtype or xd
        if xd not in _TYPES:
            raise ValueError("x_dtype must be float32, bfloat16 or float16")
        x_out = h.new_empty((T, d), dtype=xd)
        ldx, xt, xp = d, _TYPES[xd], x_out.data_ptr()
    rc = _library().moe_block_norm(h.data_ptr(), _TYPES[hd], ldh, yp, yt, ldy, wp, gp, gt, ldg, vp, T, d, res_scale,
                                   block_scale, eps, hp, ldho, xp, xt, ldx, _raw_stream(dev))
    if rc:
        _check(rc)
    return (h if keep else h_out), x_out


class Q4Matrix:
    """A matrix [rows, cols] in 4 bits on the GPU: codes uint8 [rows, cols / 32, 16] and
    scales float16 [rows, cols / group] (both contiguous, kept, not copied)."""

    def __init__(self, codes, scales):
        dev = _cuda(codes, "codes")
        if codes.dtype != torch.uint8 or codes.dim() != 3 or codes.shape[2] != 16 or \
                not codes.is_contiguous():
            raise ValueError("codes must be contiguous uint8 [rows, cols / 32, 16]")
        self.rows, self.cols = codes.shape[0], codes.shape[1] * 32
        if scales.get_device() != dev or scales.dtype != torch.float16 or scales.dim() != 2 or \
                scales.shape[0] != self.rows or not scales.is_contiguous():
            raise ValueError("scales must be contiguous float16 [rows, cols / group] beside the codes")
        if not 1 <= self.rows <= 1 << 30 or self.cols > _I32 or scales.shape[1] < 1 or \
                scales.shape[1] * (g := self.cols // scales.shape[1]) != self.cols or g not in (32, 64, 128):
            raise ValueError("scales must hold one scale per 32, 64 or 128 weights")
        self.group = g
        self.codes, self.scales, self.device = codes, scales, codes.device
        self._index = dev
        self._head = (codes.data_ptr(), scales.data_ptr(), self.rows, self.cols, g)

    @classmethod
    def from_blocks(cls, blocks, rows: int, cols: int, group: int = 32, device="cuda"):
        """From host bytes in the interchange layout: per group of a row a binary16 scale,
        then the nibble bytes of its blocks of 32 (group 32 is Q4_0)."""
        if group not in (32, 64, 128) or rows < 1 or cols < group or cols % group:
            raise ValueError("cols must be a multiple of group (32, 64 or 128)")
        b = np.ascontiguousarray(blocks, dtype=np.uint8).reshape(-1)
        n = 2 + group // 2
        if b.size != rows * (cols // group) * n:
            raise ValueError(f"blocks holds {b.size} bytes, {rows * (cols // group) * n} needed")
        b = b.reshape(rows, cols // group, n)
        scales = np.ascontiguousarray(b[:, :, :2]).view(np.float16).reshape(rows, cols // group)
        codes = np.ascontiguousarray(b[:, :, 2:]).reshape(rows, cols // 32, 16)
        return cls(torch.from_numpy(codes).to(device), torch.from_numpy(scales.copy()).to(device))


def q4_matvec(x, w: Q4Matrix, out=None, stream=None):
    """out [T, rows] = x [T, cols] times w transposed, in x's type (float32 sums)."""
    dev = w._index
    if _elsewhere(dev, stream):
        with _At(dev, stream, x, w.codes, w.scales, out):
            return q4_matvec(x, w, out)
    ldx = _rows(x, "x", dev, None, w.cols)
    T, dt = x.shape[0], x.dtype
    if out is None:
        out = x.new_empty((T, w.rows))
        ldo = w.rows
    else:
        ldo = _rows(out, "out", dev, T, w.rows, dt)
    rc = _library().moe_q4_matvec(*w._head, x.data_ptr(), _TYPES[dt], ldx, T, out.data_ptr(), ldo, _raw_stream(dev))
    if rc:
        _check(rc)
    return out


class KVCache:
    """A paged cache of keys and values in 4 bits over the caller's four tensors:

        k_codes  uint8   [n_pages, kv_heads, page_tokens, head_dim / 32, 16]
        k_scales float16 [n_pages, kv_heads, page_tokens, head_dim / 32]
        v_codes  uint8   [n_pages, kv_heads, page_tokens, 16, head_dim / 32]
        v_scales float16 [n_pages, kv_heads, page_tokens, head_dim / 32]

    A batch is given by pages int32 [n_seqs, max_pages], start int32 [n_seqs + 1] and
    past int32 [n_seqs]: rows start[s] .. start[s+1]-1 of the tensors are sequence s's
    new tokens, at positions past[s], past[s] + 1, ...
    """

    def __init__(self, k_codes, k_scales, v_codes, v_scales):
        dev = _cuda(k_codes, "k_codes")
        if k_codes.dim() != 5 or k_codes.shape[4] != 16:
            raise ValueError("k_codes must be [n_pages, kv_heads, page_tokens, head_dim / 32, 16]")
        n, h, p, nb = (int(v) for v in k_codes.shape[:4])
        want = {"k_codes": (k_codes, torch.uint8, (n, h, p, nb, 16)),
                "k_scales": (k_scales, torch.float16, (n, h, p, nb)),
                "v_codes": (v_codes, torch.uint8, (n, h, p, 16, nb)),
                "v_scales": (v_scales, torch.float16, (n, h, p, nb))}
        for name, (t, dtype, shape) in want.items():
            if t.get_device() != dev or t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on cuda:{dev}")
        if n < 1 or n > _I32 or h < 1 or h > 1024 or p < 16 or p % 16 or p > 65536 or nb not in (2, 4, 8):
            raise ValueError("head_dim must be 64, 128 or 256, page_tokens a multiple of 16 up to 65536, "
                             "kv_heads at most 1024")
        self.device, self.tensors = k_codes.device, (k_codes, k_scales, v_codes, v_scales)
        self._index = dev
        self.n_pages, self.kv_heads, self.page_tokens, self.head_dim = n, h, p, nb * 32
        self._c = _KvCache(k_codes.data_ptr(), k_scales.data_ptr(), v_codes.data_ptr(),
                           v_scales.data_ptr(), n, p, h, nb * 32)
        self._cp = ctypes.pointer(self._c)

    @classmethod
    def create(cls, n_pages: int, page_tokens: int, kv_heads: int, head_dim: int, device="cuda"):
        """A cache over new tensors (zeroed)."""
        shape, nb = (n_pages, kv_heads, page_tokens), head_dim // 32
        if head_dim not in (64, 128, 256):
            raise ValueError("head_dim must be 64, 128 or 256")
        z = lambda s, t: torch.zeros(shape + s, dtype=t, device=device)  # noqa: E731
        return cls(z((nb, 16), torch.uint8), z((nb,), torch.float16), z((16, nb), torch.uint8),
                   z((nb,), torch.float16))

    def _batch(self, pages, start, past, rows):
        dev, i32 = self._index, torch.int32
        n, m = pages.shape if pages.dim() == 2 else (0, 0)
        if pages.get_device() != dev or start.get_device() != dev or past.get_device() != dev or \
                pages.dtype != i32 or start.dtype != i32 or past.dtype != i32 or \
                not 1 <= n <= _I32 or not 1 <= m <= _I32 or start.shape != (n + 1,) or past.shape != (n,) or \
                not (pages.is_contiguous() and start.is_contiguous() and past.is_contiguous()):
            raise ValueError("pages must be [n_seqs, max_pages], start [n_seqs + 1] and past [n_seqs], "
                             f"contiguous int32 on cuda:{dev}")
        return _KvBatch(pages.data_ptr(), start.data_ptr(), past.data_ptr(), n, m, rows)

    def append(self, k, v, pages, start, past, q=None, inv_freq=None, interleaved: bool = False,
               q_out=None, stream=None):
        """Writes k, v [T, kv_heads * head_dim] into the cache, the keys rotated by their
        positions (inv_freq float32 [rot_dim / 2] or None); returns q [T, q_heads * head_dim]
        rotated likewise, or None.  Rows of no sequence, or of a negative past, are left as
        they are in `q_out` (undefined in a new one)."""
        dev, D, dt = self._index, self.head_dim, k.dtype
        if _elsewhere(dev, stream):
            with _At(dev, stream, k, v, pages, start, past, q, inv_freq, q_out, *self.tensors):
                return self.append(k, v, pages, start, past, q, inv_freq, interleaved, q_out)
        ldk = _rows(k, "k", dev, None, self.kv_heads * D)
        T = k.shape[0]
        ldv = _rows(v, "v", dev, T, self.kv_heads * D, dt)
        rot, fp = 0, None
        if inv_freq is not None:
            rot = 2 * inv_freq.shape[0] if inv_freq.dim() == 1 else -1
            if rot < 0 or rot > D or inv_freq.dtype != torch.float32 or inv_freq.get_device() != dev or \
                    not inv_freq.is_contiguous():
                raise ValueError("inv_freq must be contiguous float32 [rot_dim / 2] beside the cache, "
                                 "rot_dim <= head_dim")
            fp = inv_freq.data_ptr() if rot else None
        b = self._batch(pages, start, past, T)
        qp = op = None
        ldq = ldqo = heads = 0
        if q is not None:
            ldq = _rows(q, "q", dev, T, None, dt)
            heads, qp = self._heads(q), q.data_ptr()
        elif q_out is not None:
            raise ValueError("q_out needs q")
        if q is not None:
            if q_out is None:
                q_out = q.new_empty((T, heads * D))
                ldqo = heads * D
            else:
                ldqo = _rows(q_out, "q_out", dev, T, heads * D, dt)
            op = q_out.data_ptr()
        rc = _library().moe_kv_append(self._cp, b, _TYPES[dt], k.data_ptr(), ldk, v.data_ptr(), ldv, fp, rot,
                                      1 if interleaved else 0, qp, ldq, heads, op, ldqo, _raw_stream(dev))
        if rc:
            _check(rc)
        return q_out

    def _heads(self, q) -> int:
        n = q.shape[1]
        if n < 1 or n % (self.kv_heads * self.head_dim):
            raise ValueError("q must be [T, q_heads * head_dim], q_heads a multiple of kv_heads")
        return n // self.head_dim

    def read(self, pages, start, past, rows: int, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """(k, v) float32 [rows, kv_heads, head_dim]: the values the cache holds for the
        batch's rows (0 in a hole; undefined for rows of no sequence)."""
        if not 0 <= rows <= _I32:
            raise ValueError("rows must be in [0, 2^31)")
        if _elsewhere(self._index, stream):
            with _At(self._index, stream, pages, start, past, *self.tensors):
                return self.read(pages, start, past, rows)
        b = self._batch(pages, start, past, rows)
        k = torch.empty((rows, self.kv_heads, self.head_dim), dtype=torch.float32, device=self.device)
        v = torch.empty_like(k)
        rc = _library().moe_kv_read(self._cp, b, k.data_ptr(), v.data_ptr(), _raw_stream(self._index))
        if rc:
            _check(rc)
        return k, v

    def attend(self, q, pages, start, past, scale: float, window: int = 0, out=None, stream=None):
        """out [T, q_heads * head_dim] = softmax(scale * q K^T) V over the keys each row
        sees: positions up to its own, within `window` when window > 0.  Rows of no sequence
        are left as they are in `out` (undefined in a new one)."""
        dev, dt = self._index, q.dtype
        if _elsewhere(dev, stream):
            with _At(dev, stream, q, pages, start, past, out, *self.tensors):
                return self.attend(q, pages, start, past, scale, window, out)
        ldq = _rows(q, "q", dev)
        T, n = q.shape
        heads = self._heads(q)
        b = self._batch(pages, start, past, T)
        lib, ty = _library(), _TYPES[dt]
        if not 0 <= window <= _I32:
            raise ValueError("window must be in [0, 2^31)")
        if out is None:
            out = q.new_empty((T, n))
            ldo = n
        else:
            ldo = _rows(out, "out", dev, T, n, dt)
        need = lib.moe_kv_attend_workspace(self._cp, b, ty, heads, window)
        if need < 0:
            _check(need)
        ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
        rc = lib.moe_kv_attend(self._cp, b, ty, q.data_ptr(), ldq, heads, scale, window, out.data_ptr(), ldo,
                               ws.data_ptr() if need else None, need, _raw_stream(dev))
        if rc:
            _check(rc)
        return out
