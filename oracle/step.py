"""The operators between a prompt and its next token, plainly (numpy): rows and
products in 8-bit integers, routing by a rule, sampling, as include/moe_cache.h
defines them.
"""
import numpy as np

F32 = np.float32


def q8_rows(x):
    """(codes int64 [n, cols], scales float32 [n]) of x [n, cols] float64 holding float32 values."""
    x = np.asarray(x, np.float64)
    top = np.abs(x).max(1)
    ok = np.isfinite(top)
    with np.errstate(invalid="ignore", under="ignore"):
        s = np.where(ok, (np.where(ok, top, 0).astype(F32) / F32(127)).astype(F32), F32(np.nan)).astype(F32)
        live = ok & (s > 0)
        # the quotient of two float32 numbers lies no closer to a half integer than 2^-33 of itself unless it is one:
        # binary64 decides it
        q = np.where(live[:, None], x / np.where(live, s, 1).astype(np.float64)[:, None], 0.0)
    return np.clip(np.rint(q), -127, 127).astype(np.int64), s


def q8_matmul(codes, scales, w, w_scales):
    """float32 [T, rows], every rounding as documented (codes and w whole numbers)."""
    z = (np.asarray(codes, np.float64) @ np.asarray(w, np.float64).T)  # exact: below 2^53
    with np.errstate(over="ignore", invalid="ignore"):
        return (z.astype(F32) * scales[:, None]).astype(F32) * w_scales[None, :]


def route(z, bias, k, score="softmax", groups=1, keep=None, best=1, renorm=True, scale=1.0):
    """(idx int64 [T, k], weights float64 [T, k])."""
    z = np.asarray(z, np.float64).copy()
    z[np.isnan(z)] = -np.inf
    z = np.minimum(z, float(np.finfo(F32).max))
    T, E = z.shape
    keep = groups if keep is None else keep
    idx, wts = np.zeros((T, k), np.int64), np.zeros((T, k))
    for t in range(T):
        out = np.isneginf(z[t])
        with np.errstate(over="ignore", invalid="ignore"):
            if score == "softmax":
                s = np.where(out, 0.0, np.exp(z[t] - z[t].max()))
                s = s / s.sum() if s.sum() > 0 else s
            else:
                s = 1 / (1 + np.exp(-z[t]))
        c = z[t].copy()
        pair = np.where(out, -np.inf, s)
        if bias is not None:
            b = np.where(np.isnan(bias), -np.inf, np.asarray(bias, np.float64))
            c = np.where(out, -np.inf, s + b)
            pair = c
        ids = np.arange(E)
        if keep < groups:
            n = E // groups
            val = []
            for g in range(groups):
                v = np.sort((pair if best == 2 else c)[g * n:(g + 1) * n])[::-1]
                val.append(v[0] if best == 1 else -np.inf if np.isneginf(v[1]) else v[0] + v[1])
            kept = sorted(range(groups), key=lambda g: (-val[g], g))[:keep]
            ids = np.array([e for e in ids if e // n in kept])
        top = sorted(ids, key=lambda e: (-c[e], e))[:k]
        idx[t] = top
        w = np.where(np.isneginf(c[top]), 0.0, s[top])
        if renorm:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        wts[t] = float(F32(scale)) * w
    return idx, wts


def sample(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(tokens, probabilities) of rows z [T, V]; the settings are numbers or [T]."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    at = lambda v, t: float(v[t]) if np.ndim(v) else float(v)  # noqa: E731
    tok, prob = np.zeros(T, np.int64), np.zeros(T)
    for t in range(T):
        temp, k, share, least = at(temperature, t), int(at(top_k, t)), at(top_p, t), at(min_p, t)
        r = np.where(np.isnan(z[t]), -np.inf, np.minimum(z[t], float(np.finfo(F32).max)))
        order = np.lexsort((np.arange(V), -r))
        if np.isneginf(r[order[0]]):
            tok[t] = -1
            continue
        if not temp > 0:
            tok[t], prob[t] = order[0], 1.0
            continue
        with np.errstate(under="ignore"):
            p = np.where(np.isneginf(r[order]), 0.0, np.exp((r[order] - r[order[0]]) / temp))
        w = np.rint(p * 2.0 ** 42).astype(np.uint64)
        n = k if 0 < k < V else V
        run = np.cumsum(w)
        total = int(run[n - 1])
        if share < 1:
            goal = max(int(np.ceil(max(share, 0.0) * float(total))), 1)
            n = min(n, int(np.searchsorted(run, np.uint64(goal))) + 1)
        if least > 0:
            n = min(n, int((p >= min(least, 1.0)).sum()))
        kept = int(run[n - 1])
        x = float(u[t])
        x = min(x, 1.0) if x >= 0 else 0.0
        goal = min(int(x * float(kept)), kept - 1)
        i = int(np.searchsorted(run, np.uint64(goal), side="right"))
        tok[t], prob[t] = order[i], p[i] * 2.0 ** 42 / kept
    return tok, prob
