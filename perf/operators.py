"""The operators of a decoder layer around the routed MoE layer: what is measured of them.

Four operators, each in a plain form of elementary torch operations (float32, float64 where angles and the borders of
4-bit codes need it) and through the library:

* norm    -- the norms before and after a block, with the block's gate, the residual scale and the residual sum:
             h' = a h + b gate * norm(y) w_post,  x = norm(h') w_pre;
* matvec  -- a few tokens times a matrix held in 4 bits with a binary16 scale per group of weights;
* append  -- the new tokens' keys (rotated by their positions) and values into a paged cache held in 4 bits, the queries
             rotated on the way, and the rows as the cache holds them read back;
* attend  -- attention of the new tokens over that cache, grouped heads, causal, optionally within a window.

The cache is four tensors: codes of keys [pages, kv_heads, page_tokens, D/32, 16], codes of values [pages, kv_heads,
page_tokens, 16, D/32] (byte j of a block: element j in the low nibble, element j + 16 in the high one), and the
binary16 scales of both [pages, kv_heads, page_tokens, D/32]; an element is scale * (code - 8).
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the Gemma-like layer at decode: one token, residual in float32, a learned gate per channel
        dict(name="norm token 2816", op="norm", T=1, d=2816, h="f32", y="f32", gate="channel", parts="both"),
        # a prompt's ubatch at the large shape: bfloat16 residual, the MoE layer's float32 output
        dict(name="norm ubatch 512x6144", op="norm", T=512, d=6144, h="bf16", y="f32", gate="none", parts="both"),
        # a long prompt in binary16 with a row length no vector width divides, gates computed per element
        dict(name="norm odd 4093x2045", op="norm", T=4093, d=2045, h="f16", y="f16", gate="full", parts="both"),
        # one stream's query, key and value projections of the Gemma-like layer
        dict(name="matvec 1x2816x8192 f32", op="matvec", T=1, rows=8192, cols=2816, group=32, x="f32"),
        # four streams (the largest decode call of the MoE layer) through the large shape's projections
        dict(name="matvec 4x6144x10240 bf16", op="matvec", T=4, rows=10240, cols=6144, group=64, x="bf16"),
        # a burst of speculated tokens, rows and columns that end inside a tile
        dict(name="matvec 45x2144x5003 f16", op="matvec", T=45, rows=5003, cols=2144, group=32, x="f16"),
        # the vocabulary's projection for one token
        dict(name="matvec 1x2048x131072 f32", op="matvec", T=1, rows=131072, cols=2048, group=32, x="f32"),
        # decode: four streams append one token each
        dict(name="append 4 tokens bf16", op="append", S=4, new_lo=1, new_hi=1, past_lo=100, past_hi=9000, Hq=32,
             Hkv=8, D=128, P=64, x="bf16", rot=128, inter=False),
        # prompts of several sequences packed in one call, ragged, partial rotation in interleaved pairs
        dict(name="append ragged 6x~900 f32", op="append", S=6, new_lo=700, new_hi=1100, past_lo=1, past_hi=200000,
             Hq=16, Hkv=8, D=256, P=16, x="f32", rot=64, inter=True),
        # decode of four streams at short contexts, where latency counts
        dict(name="attend 4x~300 f32", op="attend", S=4, new_lo=1, new_hi=1, past_lo=1, past_hi=500, Hq=32, Hkv=8,
             D=128, P=64, x="f32", window=0),
        # decode of a full batch at long ragged contexts
        dict(name="attend 32x~12000 bf16", op="attend", S=32, new_lo=1, new_hi=1, past_lo=6000, past_hi=16000, Hq=64,
             Hkv=8, D=128, P=64, x="bf16", window=0),
        # prompt chunks of 512 over what is cached, local layers with a window
        dict(name="attend chunk 3x512 f16", op="attend", S=3, new_lo=470, new_hi=512, past_lo=2, past_hi=6000, Hq=16,
             Hkv=8, D=256, P=32, x="f16", window=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "matvec", "append", "attend"])
    if op == "norm":
        d = _log(rng, 24, 8192)
        return dict(op=op, T=_log(rng, 1, min(4096, (4093 * 2045) // d)), d=d, h=rng.choice(list(TYPES)),
                    y=rng.choice(list(TYPES)), gate=rng.choice(["none", "channel", "full"]),
                    parts=rng.choice(["both", "both", "pre", "post"]))
    if op == "matvec":
        group = rng.choice([32, 64, 128])
        cols = group * _log(rng, 1, 12288 // group)
        return dict(op=op, T=_log(rng, 1, 64), rows=_log(rng, 16, min(32768, (1 << 27) // cols)), cols=cols,
                    group=group, x=rng.choice(list(TYPES)))
    D = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 8])
    P = rng.choice([16, 32, 48, 64, 128])
    many = rng.random() < 0.5
    if op == "append":
        S = _log(rng, 1, 8 if many else 64)
        n = _log(rng, 2, 1000) if many else 1
        return dict(op=op, S=S, new_lo=max(1, n // 2), new_hi=n, past_lo=1, past_hi=_log(rng, 2, 200000), Hq=Hkv * G,
                    Hkv=Hkv, D=D, P=P, x=rng.choice(list(TYPES)), rot=rng.choice([0, 32, D // 2, D]),
                    inter=rng.random() < 0.5)
    S = _log(rng, 1, 4 if many else 32)
    n = _log(rng, 2, 512) if many else 1
    return dict(op=op, S=S, new_lo=max(1, n // 2), new_hi=n, past_lo=1,
                past_hi=_log(rng, 2, min(32768, (1 << 29) // (S * n * Hkv * G), (1 << 29) // (S * Hkv * D))),
                Hq=Hkv * G, Hkv=Hkv, D=D, P=P, x=rng.choice(list(TYPES)),
                window=rng.choice([0, 0, _log(rng, 1, 4096)]))


# ------------------------------------------------------------------------------------------------ inputs

def _counts(c):
    """New tokens and cached tokens of each sequence: spread over the case's ranges, the same for every seed."""
    i = torch.arange(c["S"], dtype=torch.float64) + 1
    u, v = (i * 0.6180339887498949) % 1, (i * 0.7548776662466927) % 1
    new = (c["new_lo"] + torch.floor(u * (c["new_hi"] - c["new_lo"] + 1))).long()
    lo, hi = c["past_lo"], c["past_hi"]
    past = (lo * (hi / lo) ** v if hi > 16 * lo else lo + (hi - lo) * v).round().long().clamp(lo, hi)
    return new, past


def _codes(shape, g):
    """Two codes a byte, as quantised normal values have them."""
    lo = (torch.randn(shape, generator=g, device=DEV, dtype=torch.float16) * 3.5 + 8.5).clamp_(0, 15.9).to(torch.uint8)
    hi = (torch.randn(shape, generator=g, device=DEV, dtype=torch.float16) * 3.5 + 8.5).clamp_(0, 15.9).to(torch.uint8)
    return lo | (hi << 4)


def _scales(shape, g, size):
    s = (torch.rand(shape, generator=g, device=DEV) * 0.5 + 0.75) * size
    return torch.where(torch.rand(shape, generator=g, device=DEV) < 0.5, -s, s).half()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    st = {"case": dict(c)}
    if c["op"] == "norm":
        T, d = c["T"], c["d"]
        st["h"] = (rn(T, d) * 3).to(TYPES[c["h"]])
        st["y"] = None if c["parts"] == "pre" else (rn(T, d) * (0.2 + rn(T, 1).abs())).to(TYPES[c["y"]])
        st["post_w"] = None if c["parts"] == "pre" else 1 + 0.1 * rn(d)
        st["pre_w"] = None if c["parts"] == "post" else 1 + 0.1 * rn(d)
        st["gate"] = None
        if c["parts"] != "pre" and c["gate"] != "none":
            st["gate"] = torch.sigmoid(rn(d)) if c["gate"] == "channel" else torch.sigmoid(rn(T, d)).to(TYPES[c["y"]])
        return st
    if c["op"] == "matvec":
        st["x"] = (rn(c["T"], c["cols"]) * 2).to(TYPES[c["x"]])
        st["q"] = _codes((c["rows"], c["cols"] // 32, 16), g)
        st["s"] = _scales((c["rows"], c["cols"] // c["group"]), g, 0.006)
        if own:  # the handle a program keeps with its weights (the same two tensors)
            import expert_cache_host_amd as m
            st["w"] = m.Q4Matrix(st["q"], st["s"])
        return st
    S, Hkv, D, P = c["S"], c["Hkv"], c["D"], c["P"]
    new, past = _counts(c)
    total = new + past
    if c["op"] == "append":
        # only the pages that take new tokens are resident; earlier ones are out of reach of the call
        first = past // P
        need = (total + P - 1) // P - first
    else:
        first = torch.zeros_like(past)
        need = (total + P - 1) // P
    n_pages = int(need.sum()) + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32).cpu()
    pages = torch.full((S, int(((total + P - 1) // P).max())), -1, dtype=torch.int32)
    at = 0
    for s in range(S):
        k = int(need[s])
        pages[s, int(first[s]):int(first[s]) + k] = order[at:at + k]
        at += k
    st["pages"] = pages.to(DEV)
    st["past"] = past.to(torch.int32).to(DEV)
    start = torch.zeros(S + 1, dtype=torch.int64)
    start[1:] = torch.cumsum(new, 0)
    st["start"] = start.to(torch.int32).to(DEV)
    T = int(start[-1])
    st["T"], st["n_max"], st["len_max"] = T, int(new.max()), int(total.max())
    shape = (n_pages, Hkv, P)
    if c["op"] == "append":
        st["k_q"] = torch.zeros(shape + (D // 32, 16), dtype=torch.uint8, device=DEV)
        st["v_q"] = torch.zeros(shape + (16, D // 32), dtype=torch.uint8, device=DEV)
        st["k_s"] = torch.zeros(shape + (D // 32,), dtype=torch.float16, device=DEV)
        st["v_s"] = torch.zeros(shape + (D // 32,), dtype=torch.float16, device=DEV)
        # one row of all projections a token, as the projection's matrix yields it
        qkv = (rn(T, (c["Hq"] + 2 * Hkv) * D) * 1.5).to(TYPES[c["x"]])
        a, b = c["Hq"] * D, (c["Hq"] + Hkv) * D
        st["xq"], st["xk"], st["xv"] = qkv[:, :a], qkv[:, a:b], qkv[:, b:]
        st["inv_freq"] = None
        if c["rot"]:
            i = torch.arange(c["rot"] // 2, dtype=torch.float64)
            st["inv_freq"] = (10000.0 ** (-2 * i / c["rot"])).float().to(DEV)
    else:
        st["k_q"] = _codes(shape + (D // 32, 16), g)
        st["v_q"] = _codes(shape + (16, D // 32), g)
        st["k_s"] = _scales(shape + (D // 32,), g, 0.3)
        st["v_s"] = _scales(shape + (D // 32,), g, 0.3)
        st["xq"] = (rn(T, c["Hq"] * D) * 1.5).to(TYPES[c["x"]])
    if own:  # the handle a program keeps with its cache (the same four tensors)
        import expert_cache_host_amd as m
        st["cache"] = m.KVCache(st["k_q"], st["k_s"], st["v_q"], st["v_s"])
    return st


# ------------------------------------------------------------------------------------------------ one pass

A, B, EPS = 0.9, 1.1, 1e-6


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def _own(st):
    import expert_cache_host_amd as m
    c = st["case"]
    if c["op"] == "norm":
        h, x = m.block_norm(st["h"], st["y"], st["post_w"], st["gate"], st["pre_w"], res_scale=A, block_scale=B,
                            eps=EPS, x_dtype=TYPES[c["y"]])
        return [h] if x is None else [h, x]
    if c["op"] == "matvec":
        return [m.q4_matvec(st["x"], st["w"])]
    if c["op"] == "append":
        q = st["cache"].append(st["xk"], st["xv"], st["pages"], st["start"], st["past"], q=st["xq"],
                               inv_freq=st["inv_freq"], interleaved=c["inter"])
        k, v = st["cache"].read(st["pages"], st["start"], st["past"], st["T"])
        return [q, k, v]
    return [st["cache"].attend(st["xq"], st["pages"], st["start"], st["past"], scale=c["D"] ** -0.5,
                               window=c["window"])]


def _norm(st):
    c = st["case"]
    h = st["h"].float() * A
    if st["y"] is not None:
        y = st["y"].float()
        n = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * st["post_w"]
        if st["gate"] is not None:
            n = n * st["gate"].float()
        h = h + B * n
    out = [h.to(TYPES[c["h"]])]
    if st["pre_w"] is not None:
        out.append((h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * st["pre_w"]).to(TYPES[c["y"]]))
    return out


def _matvec(st):
    c = st["case"]
    w = torch.cat([st["q"] & 15, st["q"] >> 4], 2).float() - 8
    w = w.view(c["rows"], -1, c["group"]) * st["s"].float().unsqueeze(2)
    return [(st["x"].float() @ w.view(c["rows"], c["cols"]).t()).to(TYPES[c["x"]])]


def _rows_of(st):
    """Sequence and position of every new token."""
    t = torch.arange(st["T"], device=DEV)
    s = torch.searchsorted(st["start"].long(), t, right=True) - 1
    return s, st["past"].long()[s] + t - st["start"].long()[s]


def _turn(x, ang, inter):
    """Rotates the first pairs of x [T, H, D] in 64 bits; the result rounded to 32."""
    n = ang.shape[1]
    x = x.double()
    if n == 0:
        return x.float()
    cs, sn = torch.cos(ang).unsqueeze(1), torch.sin(ang).unsqueeze(1)
    if inter:
        p, q = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        r = torch.stack([p * cs - q * sn, q * cs + p * sn], -1).flatten(2)
    else:
        p, q = x[..., :n], x[..., n:2 * n]
        r = torch.cat([p * cs - q * sn, q * cs + p * sn], 2)
    return torch.cat([r, x[..., 2 * n:]], 2).float()


def _quantise(x):
    """Codes [.., D/32, 32] and scales [.., D/32] of x [.., D] in float32: the scale maps the block's first largest
    value to code 0; borders are compared in 64 bits."""
    b = x.unflatten(-1, (-1, 32)).double()
    at = b.abs().argmax(-1, keepdim=True)
    d = (b.gather(-1, at) / -8).float().half()
    codes = torch.where(d == 0, 8.0, torch.floor(b / torch.where(d == 0, 1, d).double() + 8.5).clamp(0, 15))
    return codes.to(torch.uint8), d.squeeze(-1)


def _append(st):
    c = st["case"]
    T, D, P = st["T"], c["D"], c["P"]
    s, pos = _rows_of(st)
    n = c["rot"] // 2
    ang = pos.double().unsqueeze(1) * (st["inv_freq"].double() if n else torch.empty(0, device=DEV).double())
    q = _turn(st["xq"].reshape(T, c["Hq"], D), ang, c["inter"]).to(TYPES[c["x"]]).flatten(1)
    page = st["pages"][s, pos // P].long()
    at = pos % P
    kq, ks = _quantise(_turn(st["xk"].reshape(T, c["Hkv"], D), ang, c["inter"]))
    vq, vs = _quantise(st["xv"].reshape(T, c["Hkv"], D).float())
    st["k_q"][page, :, at] = kq[..., :16] | (kq[..., 16:] << 4)
    st["v_q"][page, :, at] = (vq[..., :16] | (vq[..., 16:] << 4)).transpose(2, 3)
    st["k_s"][page, :, at] = ks
    st["v_s"][page, :, at] = vs
    return [q, _values(st["k_q"][page, :, at], st["k_s"][page, :, at]),
            _values(st["v_q"][page, :, at].transpose(-1, -2), st["v_s"][page, :, at])]


def _values(q, s):
    """[.., D] float32 of codes [.., D/32, 16] and scales [.., D/32]."""
    return ((torch.cat([q & 15, q >> 4], -1).float() - 8) * s.float().unsqueeze(-1)).flatten(-2)


def _attend(st):
    c = st["case"]
    S, Hkv, D, P = c["S"], c["Hkv"], c["D"], c["P"]
    G, N, L = c["Hq"] // Hkv, st["n_max"], st["len_max"]
    n_pages = (L + P - 1) // P
    page = st["pages"][:, :n_pages].long().clamp(min=0)
    seq = lambda a: a[page].transpose(1, 2).flatten(2, 3)  # noqa: E731  [S, Hkv, n_pages * P, ...]
    k = _values(seq(st["k_q"]), seq(st["k_s"]))
    s, pos = _rows_of(st)
    i = pos - st["past"].long()[s]
    q = torch.zeros((S, N, Hkv, G, D), device=DEV)
    q[s, i] = st["xq"].reshape(-1, Hkv, G, D).float()
    q = q.permute(0, 2, 3, 1, 4).reshape(S * Hkv, G * N, D)
    z = torch.bmm(q, k.reshape(S * Hkv, -1, D).transpose(1, 2).contiguous()) * D ** -0.5
    del k
    last = st["past"].long().view(S, 1, 1, 1, 1) + torch.arange(N, device=DEV).view(1, 1, 1, N, 1)
    key = torch.arange(n_pages * P, device=DEV)
    seen = key <= last
    if c["window"]:
        seen = seen & (key > last - c["window"])
    z = z.view(S, Hkv, G, N, -1).masked_fill_(~seen, -math.inf)
    z -= z.amax(-1, keepdim=True)
    z.exp_()
    z /= z.sum(-1, keepdim=True)
    v = _values(seq(st["v_q"].transpose(-1, -2)), seq(st["v_s"]))
    o = torch.bmm(z.view(S * Hkv, G * N, -1), v.view(S * Hkv, -1, D))
    o = o.view(S, Hkv, G, N, D)[s, :, :, i]
    return [o.reshape(-1, c["Hq"] * D).to(TYPES[c["x"]])]


_PLAIN = {"norm": _norm, "matvec": _matvec, "append": _append, "attend": _attend}


# ------------------------------------------------------------------------------------------------ what it needs

def work(case):
    c = case
    if c["op"] == "norm":
        n = c["T"] * c["d"]
        b, f = 2 * n * BYTES[c["h"]], 2 * n
        if c["parts"] != "pre":
            b, f = b + n * BYTES[c["y"]] + 4 * c["d"], f + 7 * n
            b += n * BYTES[c["y"]] if c["gate"] == "full" else 4 * c["d"] if c["gate"] == "channel" else 0
        if c["parts"] != "post":
            b, f = b + n * BYTES[c["y"]] + 4 * c["d"], f + 5 * n
        return {"bytes": b, "flops": f}
    if c["op"] == "matvec":
        n = c["rows"] * c["cols"]
        return {"bytes": n // 2 + 2 * n // c["group"] + c["T"] * (c["rows"] + c["cols"]) * BYTES[c["x"]],
                "flops": 2 * c["T"] * n}
    new, past = _counts(c)
    T, D = int(new.sum()), c["D"]
    row = c["Hkv"] * 2 * (D // 2 + D // 16)  # a token's keys and values in 4 bits, with their scales
    table = 4 * (2 * c["S"] + 1)
    if c["op"] == "append":
        return {"bytes": T * ((2 * c["Hq"] + 2 * c["Hkv"]) * D * BYTES[c["x"]] + 2 * row + 2 * c["Hkv"] * D * 4) + table,
                "flops": T * D * (6 * c["Hq"] + 16 * c["Hkv"])}
    pairs = keys = 0
    for n, p in zip(new.tolist(), past.tolist()):
        w = c["window"] or n + p
        pairs += sum(min(w, p + i + 1) for i in range(n))
        keys += min(n + p, w + n - 1)
    return {"bytes": keys * row + 2 * T * c["Hq"] * D * BYTES[c["x"]] + table + 4 * (keys // c["P"]),
            "flops": 4 * pairs * c["Hq"] * D}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """From the definitions, one row, head or sequence at a time, in float64."""
    c, st = case, prepare(case, seed)
    if c["op"] == "norm":
        h = st["h"].double() * A
        if st["y"] is not None:
            y = st["y"].double()
            r = 1 / torch.sqrt(y.square().sum(1) / c["d"] + EPS)
            g = torch.ones(c["d"], device=DEV).double() if st["gate"] is None else st["gate"].double()
            h += B * g * (r[:, None] * y * st["post_w"].double())
        if st["pre_w"] is None:
            return [h]
        return [h, h / torch.sqrt(h.square().sum(1) / c["d"] + EPS)[:, None] * st["pre_w"].double()]
    if c["op"] == "matvec":
        out = torch.zeros(c["T"], c["rows"], dtype=torch.float64, device=DEV)
        x = st["x"].double().view(c["T"], -1, 2, 16)
        per = c["group"] // 32
        for r in range(0, c["rows"], 4096):
            q, s = st["q"][r:r + 4096].double(), st["s"][r:r + 4096].double().repeat_interleave(per, 1)
            hi = torch.floor(q / 16)
            w = torch.stack([(q - 16 * hi - 8), hi - 8], 2) * s[:, :, None, None]
            out[:, r:r + 4096] = x.flatten(1) @ w.flatten(1).T
        return [out]
    new, past = _counts(c)
    H, Hkv, D, P = c["Hq"], c["Hkv"], c["D"], c["P"]
    if c["op"] == "append":
        parts = [[], [], []]
        row = 0
        for n, p in zip(new.tolist(), past.tolist()):
            pos = torch.arange(p, p + n, device=DEV, dtype=torch.float64)
            q, k, v = (st[a][row:row + n].double().view(n, -1, D) for a in ("xq", "xk", "xv"))
            q, k = q.clone(), k.clone()
            for j in range(c["rot"] // 2):
                a, b = (2 * j, 2 * j + 1) if c["inter"] else (j, j + c["rot"] // 2)
                w = torch.polar(torch.ones_like(pos), pos * st["inv_freq"][j].double())[:, None]
                for x in (q, k):
                    z = torch.complex(x[:, :, a], x[:, :, b]) * w
                    x[:, :, a], x[:, :, b] = z.real, z.imag
            parts[0].append(q.flatten(1))
            for out, x in ((parts[1], k), (parts[2], v)):
                x = x.float().double().view(n, Hkv, D // 32, 32)  # keys are rounded to 32 bits before their codes
                big = x.abs().max(-1, keepdim=True).values
                first = (x.abs() == big).to(torch.int8).argmax(-1, keepdim=True)
                d = (torch.gather(x, -1, first) / -8).float().half().double()
                ratio = torch.where(d == 0, 0.0, x / torch.where(d == 0, 1.0, d))
                out.append((d * (torch.floor(ratio + 8.5).clamp(0, 15) - 8)).view(n, Hkv, D))
            row += n
        return [torch.cat(a) for a in parts]
    out = torch.zeros(st["T"], H, D, dtype=torch.float64, device=DEV)
    row = 0
    for s, (n, p) in enumerate(zip(new.tolist(), past.tolist())):
        L = n + p
        lo = max(0, p + 1 - c["window"]) if c["window"] else 0
        at = torch.arange(lo, L, device=DEV)
        pg, off = st["pages"][s].long()[at // P], at % P
        pos = torch.arange(p, L, device=DEV)[:, None]
        hidden = (at > pos) | ((at <= pos - c["window"]) if c["window"] else False)
        q = st["xq"][row:row + n].double().view(n, H, D)
        for h in range(Hkv):
            kb, vb = st["k_q"][pg, h, off].long(), st["v_q"][pg, h, off].long().transpose(1, 2)
            k, v = (torch.stack([b % 16, torch.div(b, 16, rounding_mode="floor")], 2).double() - 8 for b in (kb, vb))
            k = (k * st["k_s"][pg, h, off].double()[:, :, None, None]).flatten(1)
            v = (v * st["v_s"][pg, h, off].double()[:, :, None, None]).flatten(1)
            for j in range(h * H // Hkv, (h + 1) * H // Hkv):
                z = (q[:, j] @ k.T) / math.sqrt(D)
                out[row:row + n, j] = torch.softmax(z.masked_fill(hidden, -math.inf), 1) @ v
        row += n
    return [out.flatten(1)]
