"""The decoder-layer operators around the MoE layer, plainly, in binary64 (numpy).

block_norm, Q4 matrices, the rotation, the cache's 4-bit code and attention, as
include/moe_cache.h defines them.
"""
import numpy as np


def block_norm(h, y=None, post_w=None, gate=None, pre_w=None, res_scale=1.0, block_scale=1.0, eps=1e-6):
    """(h', x) in binary64; x is None without pre_w."""
    h = np.asarray(h, np.float64) * float(np.float32(res_scale))
    if y is not None:
        n = np.asarray(y, np.float64)
        if post_w is not None:
            n = n / np.sqrt((n * n).mean(1, keepdims=True) + float(np.float32(eps))) * np.asarray(post_w, np.float64)
        if gate is not None:
            n = n * np.asarray(gate, np.float64)
        h = h + float(np.float32(block_scale)) * n
    if pre_w is None:
        return h, None
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + float(np.float32(eps))) * np.asarray(pre_w, np.float64)


def q4_values(codes, scales):
    """[rows, cols] of codes uint8 [rows, cols/32, 16] and scales float16 [rows, cols/group]."""
    q = np.concatenate([codes & 15, codes >> 4], -1).astype(np.float64) - 8
    rows = codes.shape[0]
    w = q.reshape(rows, -1)
    group = w.shape[1] // scales.shape[1]
    return w * np.repeat(scales.astype(np.float64), group, 1)


def rotate(x, pos, inv_freq, interleaved):
    """x [T, H, D] turned by position pos [T], rounded to float32."""
    x = np.array(x, np.float64)
    if inv_freq is None or len(inv_freq) == 0:
        return x.astype(np.float32)
    n = len(inv_freq)
    a = np.asarray(pos, np.float64)[:, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(a)[:, None], np.sin(a)[:, None]
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    p, q = x[..., i].copy(), x[..., j].copy()
    x[..., i], x[..., j] = p * c - q * s, q * c + p * s
    return x.astype(np.float32)


def q4_encode(x):
    """codes [.., D/32, 32] uint8 and scales [.., D/32] float16 of x [.., D] float32."""
    big = float(np.finfo(np.float32).max)
    b = np.nan_to_num(np.asarray(x, np.float32).astype(np.float64), nan=0.0, posinf=big, neginf=-big)
    b = b.reshape(*b.shape[:-1], -1, 32)
    at = np.abs(b).argmax(-1, keepdims=True)
    m = np.take_along_axis(b, at, -1)[..., 0]
    d = np.clip(m / -8, -65504.0, 65504.0).astype(np.float32).astype(np.float16) + np.float16(0)
    dd = d.astype(np.float64)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(dd == 0, 8, np.clip(np.floor(b / dd + 8.5), 0, 15))
    return code.astype(np.uint8), np.where(d == 0, np.float16(0), d)


def q4_decode(codes, scales):
    """[.., D] binary64 of codes [.., D/32, 32] and scales [.., D/32]."""
    v = (codes.astype(np.float64) - 8) * scales.astype(np.float64)[..., None]
    return v.reshape(*v.shape[:-2], v.shape[-2] * 32)


def attend(q, k, v, seen, scale):
    """out [H, D] of one row q [H, D] over keys k, v [n, Hkv, D] (binary64) where seen [n]."""
    H, D = q.shape
    out = np.zeros((H, D))
    idx = np.nonzero(seen)[0]
    if len(idx) == 0:
        return out
    G = H // k.shape[1]
    for h in range(H):
        z = (k[idx, h // G] @ np.asarray(q[h], np.float64)) * scale
        p = np.exp(z - z.max())
        out[h] = (p / p.sum()) @ v[idx, h // G]
    return out
