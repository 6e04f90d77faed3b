"""Operators between a prompt and its next token, around the routed MoE layer: what is measured of them.

Three operators, each in a plain form of elementary torch operations and through the library:

* q8     -- tokens times a matrix held in 8-bit integers with a scale per channel; the tokens are rounded to 8 bits with
            a scale each on the way:
              s_t = max_c |x_tc| / 127,  a_tc = rint(x_tc / s_t),  out_tr = s_t w_r sum_c a_tc b_rc;
* route  -- the selection of experts from the router's logits: softmax or sigmoid scores, a bias that takes part in the
            selection alone, groups of experts, the k best, weights renormalised over them;
* sample -- the next token of each row of logits with temperature, top-k, top-p and min-p from a given random number:
              tokens in falling order (equal ones by their ids), p_i = exp((z_i - z_0) / temperature), kept are the
              first min(k, least n whose sum reaches top_p of the first k's, number with p_i >= min_p); the token is
              the first whose running sum passes u times the kept sum.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # one stream's query, key and value projections of the Gemma-like layer
        dict(name="q8 token 1x2816x8192 f32", op="q8", T=1, cols=2816, rows=8192, x="f32"),
        # a batch of streams through the large shape's projections
        dict(name="q8 streams 24x6144x10240 bf16", op="q8", T=24, cols=6144, rows=10240, x="bf16"),
        # a prompt's last piece, sizes that end inside every tile
        dict(name="q8 odd 509x2045x5003 f16", op="q8", T=509, cols=2045, rows=5003, x="f16"),
        # a prompt's ubatch at the large shape
        dict(name="q8 ubatch 512x6144x10240 bf16", op="q8", T=512, cols=6144, rows=10240, x="bf16"),
        # several prompts' chunks packed in one call
        dict(name="q8 prompts 4096x6144x16384 bf16", op="q8", T=4096, cols=6144, rows=16384, x="bf16"),
        # one token of a layer of 128 experts, softmax scores with a bias, where latency counts
        dict(name="route token 1x128 f32", op="route", T=1, E=128, k=8, x="f32", score="softmax", bias=True, groups=1,
             keep=1, best=1, renorm=True),
        # a prompt's ubatch over 256 experts in 8 groups, of which the 4 with the largest pair count
        dict(name="route ubatch 512x256 f32", op="route", T=512, E=256, k=8, x="f32", score="sigmoid", bias=True,
             groups=8, keep=4, best=2, renorm=True),
        # a long prompt over the most experts a layer may have, no groups
        dict(name="route prompt 12288x512 bf16", op="route", T=12288, E=512, k=10, x="bf16", score="sigmoid", bias=True,
             groups=1, keep=1, best=1, renorm=True),
        # one stream's next token, one setting for the call
        dict(name="sample 1x131072 f32", op="sample", T=1, V=131072, x="f32", per_row=False, temp=0.8, top_k=50,
             top_p=0.95, min_p=0.0),
        # four streams, temperature alone: the whole vocabulary stays
        dict(name="sample 4x65003 f16 unfiltered", op="sample", T=4, V=65003, x="f16", per_row=False, temp=1.0, top_k=0,
             top_p=1.0, min_p=0.0),
        # a batch of streams of one server, each with settings of its own (greedy ones among them)
        dict(name="sample 32x131072 bf16 mixed", op="sample", T=32, V=131072, x="bf16", per_row=True, temp=0.9,
             top_k=200, top_p=0.9, min_p=0.02),
        # the largest batch and vocabulary
        dict(name="sample 64x262144 f32 top-p", op="sample", T=64, V=262144, x="f32", per_row=True, temp=1.1, top_k=0,
             top_p=0.92, min_p=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["q8", "route", "sample"])
    x = rng.choice(list(TYPES))
    if op == "q8":
        cols, rows = _log(rng, 16, 12288), _log(rng, 16, 32768)
        rows = min(rows, (1 << 27) // cols)
        return dict(op=op, T=_log(rng, 1, min(4096, (4096 * 6144 * 16384) // (cols * rows))), cols=cols, rows=rows, x=x)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        keep = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, (12288 * 512) // max(E, 384)), E=E, k=rng.randint(1, min(16, keep * E // groups)),
                    x=x, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.7, groups=groups, keep=keep,
                    best=rng.choice([1, 2]), renorm=rng.random() < 0.8)
    V = _log(rng, 200, 262144)
    return dict(op=op, T=_log(rng, 1, 64), V=V, x=x, per_row=rng.random() < 0.5, temp=round(rng.uniform(0.3, 1.5), 3),
                top_k=rng.choice([0, _log(rng, 1, 1000)]), top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.005, 0.2), 3)]))


# ------------------------------------------------------------------------------------------------ inputs

SCALE = 2.5  # the factor on a layer's routed weights


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    rand = lambda *s: torch.rand(s, generator=g, device=DEV)  # noqa: E731
    st = {"case": dict(c)}
    if c["op"] == "q8":
        # a few channels stand out, as they do in a model's residual stream
        channel = 1 + 12 * (rand(c["cols"]) < 0.01).float()
        st["x"] = (rn(c["T"], c["cols"]) * channel * (0.3 + rand(c["T"], 1))).to(TYPES[c["x"]])
        st["q"] = (rn(c["rows"], c["cols"]) * 36).round_().clamp_(-127, 127).to(torch.int8)
        st["s"] = (0.5 + rand(c["rows"])) * 4e-4
        if own:  # the handle a program keeps with its weights
            import expert_cache_host_amd as m
            st["w"] = m.Q8Matrix(st["q"], st["s"])
        return st
    if c["op"] == "route":
        st["z"] = (rn(c["T"], c["E"]) * 1.5 + 0.7 * rn(c["E"])).to(TYPES[c["x"]])
        st["b"] = None
        if c["bias"]:
            st["b"] = rn(c["E"]) * (0.1 if c["score"] == "sigmoid" else 0.3 / c["E"])
        if own:  # the layer's rule, kept with the model
            import expert_cache_host_amd as m
            st["rule"] = m.RoutingRule(c["k"], score=c["score"], groups=c["groups"], keep_groups=c["keep"],
                                       group_best=c["best"], renorm=c["renorm"], scale=SCALE)
        return st
    T, V = c["T"], c["V"]
    # most tokens far down, a few ahead of them; some are banned
    z = 2 * rn(T, V) + 9 * rand(T, V) ** 12
    z = z.masked_fill_(rand(T, V) < 0.002, -math.inf)
    st["z"] = z.to(TYPES[c["x"]])
    st["u"] = rand(T)
    st["temp"], st["top_k"], st["top_p"], st["min_p"] = c["temp"], c["top_k"], c["top_p"], c["min_p"]
    if c["per_row"]:
        i = torch.arange(T, device=DEV)
        st["temp"] = torch.where(i % 5 == 3, 0.0, c["temp"] * (0.7 + 0.6 * rand(T)))
        st["top_k"] = torch.where(i % 3 == 1, 0, c["top_k"]).to(torch.int32)
        st["top_p"] = torch.where(i % 4 == 2, 1.0, c["top_p"] * (1 - 0.1 * rand(T))) if c["top_p"] < 1 else \
            torch.ones(T, device=DEV)
        st["min_p"] = c["min_p"] * rand(T)
    return st


# ------------------------------------------------------------------------------------------------ one pass

def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def _own(st):
    import expert_cache_host_amd as m
    c = st["case"]
    if c["op"] == "q8":
        return [m.q8_matmul(st["x"], st["w"])]
    if c["op"] == "route":
        return list(m.route_experts(st["z"], st["rule"], bias=st["b"]))
    return list(m.sample_tokens(st["z"], st["u"], temperature=st["temp"], top_k=st["top_k"], top_p=st["top_p"],
                                min_p=st["min_p"]))


def _q8(st):
    c = st["case"]
    x = st["x"].float()
    s = x.abs().amax(1, keepdim=True) / 127
    # a code is decided in 64 bits: a quotient next to a border may round onto it in 32
    a = torch.round(x.double() / torch.where(s == 0, 1.0, s).double()).float()
    b = st["q"].float()
    z = torch.zeros(c["T"], c["rows"], device=DEV, dtype=torch.float64)
    for i in range(0, c["cols"], 1024):  # 1024 products of at most 127^2 sum exactly in 32 bits, all of them do not
        z += a[:, i:i + 1024] @ b[:, i:i + 1024].t()
    return [(z.float() * s * st["s"]).to(TYPES[c["x"]])]


def _route(st):
    c = st["case"]
    T, E, G = c["T"], c["E"], c["groups"]
    z = st["z"].double()  # sums of a score and a bias lie close to each other
    if c["score"] == "softmax":
        s = torch.exp(z - z.amax(1, keepdim=True))
        s = s / s.sum(1, keepdim=True)
    else:
        s = 1 / (1 + torch.exp(-z))
    order = z if st["b"] is None else s + st["b"].double()
    if c["keep"] < G:
        pair = (s if st["b"] is None else order).view(T, G, -1).sort(dim=2, descending=True).values
        value = pair[:, :, 0] + pair[:, :, 1] if c["best"] == 2 else order.view(T, G, -1).amax(2)
        rank = value.sort(dim=1, descending=True, stable=True).indices
        out = torch.ones(T, G, dtype=torch.bool, device=DEV).scatter_(1, rank[:, :c["keep"]], False)
        order = order.masked_fill(out.repeat_interleave(E // G, 1), -math.inf)
    ids = order.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = s.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return [ids.to(torch.int32), (SCALE * w).float()]


def _column(v):
    """A setting of the call, or one of each row, against [T, V]."""
    return v.double().unsqueeze(1) if torch.is_tensor(v) else v


def _sample(st):
    z, ids = st["z"].float().sort(dim=1, descending=True, stable=True)
    temp, k, top_p, min_p = (_column(st[n]) for n in ("temp", "top_k", "top_p", "min_p"))
    rank = torch.arange(z.shape[1], device=DEV).unsqueeze(0)
    greedy = (temp <= 0) if torch.is_tensor(temp) else torch.full((z.shape[0], 1), temp <= 0, device=DEV)
    if torch.is_tensor(temp):
        temp = torch.where(greedy, 1.0, temp)
    # long sums and their borders in 64 bits
    p = torch.exp((z.double() - z[:, :1].double()) / (temp if torch.is_tensor(temp) else temp or 1.0))
    p = p * ((rank < k) | (torch.as_tensor(k, device=DEV) <= 0))
    # the share of top-p is that of the first k, whatever min-p leaves of them
    before = p.cumsum(1) - p
    share = torch.as_tensor(top_p, device=DEV)
    p = p * ((before < share * p.sum(1, keepdim=True)) | (share >= 1)) * (p >= min_p)
    p = torch.where(greedy, (rank == 0).double(), p)
    run_sum = p.cumsum(1)
    at = (run_sum <= st["u"].double().unsqueeze(1) * run_sum[:, -1:]).sum(1, keepdim=True)
    at = torch.minimum(at, (p > 0).sum(1, keepdim=True) - 1)
    prob = p.gather(1, at) / run_sum[:, -1:]
    return [ids.gather(1, at).squeeze(1).to(torch.int32), prob.squeeze(1).float()]


_PLAIN = {"q8": _q8, "route": _route, "sample": _sample}


# ------------------------------------------------------------------------------------------------ what it needs

def work(case):
    c = case
    n = BYTES[c["x"]]
    if c["op"] == "q8":
        return {"bytes": c["T"] * (c["cols"] + c["rows"]) * n + c["rows"] * (c["cols"] + 4),
                "flops": 2 * c["T"] * c["cols"] * c["rows"]}
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * n + 8 * c["k"]) + (4 * c["E"] if c["bias"] else 0),
                "flops": c["T"] * c["E"] * 6}
    return {"bytes": c["T"] * (c["V"] * n + 12 + (16 if c["per_row"] else 0)), "flops": c["T"] * c["V"] * 6}


# ------------------------------------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """From the definitions, a block of rows or one row at a time, in float64 and whole numbers."""
    c, st = case, prepare(case, seed)
    if c["op"] == "q8":
        out = torch.empty(c["T"], c["rows"], dtype=torch.float64, device=DEV)
        w = st["q"].double().mul_(st["s"].double()[:, None])
        for t in range(0, c["T"], 256):
            x = st["x"][t:t + 256].double()
            top = x.abs().max(1, keepdim=True).values
            s = (top / 127).float().double()  # the scale is held in 32 bits
            q = x / s
            low = torch.floor(q)
            # to the nearest, halves to the even neighbour
            up = (q - low > 0.5) | ((q - low == 0.5) & (torch.remainder(low, 2) == 1))
            out[t:t + 256] = (low + up.double()).mul_(s) @ w.T
        return [out]
    if c["op"] == "route":
        z = st["z"].double()
        bias = torch.zeros(c["E"], dtype=torch.float64, device=DEV) if st["b"] is None else st["b"].double()
        s = torch.softmax(z, 1) if c["score"] == "softmax" else torch.sigmoid(z)
        select = s + bias if st["b"] is not None else z.clone()
        left = select.clone()
        if c["keep"] < c["groups"]:
            parts = torch.stack(((s + bias) if c["best"] == 2 else select).chunk(c["groups"], 1), 1)
            value = parts.topk(c["best"], 2).values.sum(2)
            kept = torch.zeros_like(value, dtype=torch.bool)
            for _ in range(c["keep"]):  # the first of the largest, one group at a time
                first = (value == value.max(1, keepdim=True).values).to(torch.int8).argmax(1, keepdim=True)
                kept.scatter_(1, first, True)
                value.scatter_(1, first, -math.inf)
            left[~kept.repeat_interleave(c["E"] // c["groups"], 1)] = -math.inf
        ids = []
        for _ in range(c["k"]):
            first = (left == left.max(1, keepdim=True).values).to(torch.int8).argmax(1, keepdim=True)
            ids.append(first)
            left.scatter_(1, first, -math.inf)
        ids = torch.cat(ids, 1)
        w = torch.gather(s, 1, ids)
        return [ids.to(torch.int32), SCALE * (w / w.sum(1, keepdim=True) if c["renorm"] else w)]
    tokens, probs = [], []
    for t in range(c["T"]):
        temp, k, share, least = (float(v[t]) if torch.is_tensor(v) else float(v)
                                 for v in (st["temp"], st["top_k"], st["top_p"], st["min_p"]))
        z = st["z"][t].double()
        order = torch.argsort(-z, stable=True)
        if temp <= 0:
            tokens.append(int(order[0]))
            probs.append(1.0)
            continue
        p = torch.exp((z[order] - z[order[0]]) / temp)
        n = int((p > 0).sum())
        n = min(n, int(k)) if k > 0 else n
        total = torch.cumsum(p[:n], 0)
        if share < 1:
            n = min(n, int(torch.searchsorted(total, share * total[n - 1])) + 1)
        n = min(n, int((p >= least).sum()))
        at = int(torch.searchsorted(total[:n], float(st["u"][t]) * total[n - 1], right=True))
        at = min(at, n - 1)
        tokens.append(int(order[at]))
        probs.append(float(p[at] / total[n - 1]))
    return [torch.tensor(tokens, dtype=torch.int32, device=DEV), torch.tensor(probs, dtype=torch.float64, device=DEV)]
