"""The decoder-layer operators against the binary64 oracle on the GPU.

Tolerances are worst-case bounds of the float32 steps (u = 2^-24 per rounding)
plus half a step of the output's type; they are derived beside each check."""
import numpy as np
import pytest
import torch

import expert_cache_host_amd as m
from expert_cache_host_amd.binding import MoeError
from oracle import decoder as o

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def strided(t, extra=3, shift=0):
    """The same rows in a wider buffer (row stride shape[1] + extra, offset `shift` elements)."""
    buf = torch.full((t.shape[0], t.shape[1] + extra + shift), 7.5, dtype=t.dtype, device=t.device)
    buf[:, shift:shift + t.shape[1]] = t
    return buf[:, shift:shift + t.shape[1]]


# ------------------------------------------------------------------ norms

def check_norm(h, y, post_w, gate, pre_w, ht, xt, got_h, got_x, a=1.0, b=1.0, eps=1e-6):
    rh, rx = o.block_norm(f64(h), f64(y), f64(post_w), f64(gate), f64(pre_w), a, b, eps)
    d = h.shape[1]
    # a mean of squares: at most 32 sequential adds per thread, 6 lane and 16 wave steps, one division and one
    # add, each within u of a sum of positive terms, the square u: 56 u, halved by the root, 1 ulp (2 u) for the
    # root; four more roundings: 28 + 2 + 4 < 40 u per factor chain
    ha = np.abs(f64(h)) * abs(a)
    nb = np.abs(rh - f64(h) * float(np.float32(a))) if y is not None else 0 * ha
    eh = 2 * U * ha + 40 * U * nb
    if got_h is not None:
        # values below the type's normal range round by its smallest step
        assert np.all(np.abs(f64(got_h) - rh) <= eh + HALF[ht] * (np.abs(rh) + eh) + float(torch.finfo(TYPES[ht]).smallest_normal)), "h'"
    if pre_w is not None:
        w = np.abs(f64(pre_w))
        r = 1 / np.sqrt((rh * rh).mean(1, keepdims=True) + eps)
        # the mean's own relative error: 2 sum(|h'| eh) / sum(h'^2) halved by the root, plus 40 u
        rel = (np.abs(rh) * eh).mean(1, keepdims=True) / ((rh * rh).mean(1, keepdims=True) + eps) + 40 * U
        ex = w * r * (eh + np.abs(rh) * rel) * (1 + 1e-3)
        assert np.all(np.abs(f64(got_x) - rx) <= ex + HALF[xt] * (np.abs(rx) + ex) + float(torch.finfo(TYPES[xt]).smallest_normal)), "x"


@pytest.mark.parametrize("d", [1, 3, 64, 65, 1000, 2045, 2816, 4096, 5003, 6144, 8193, 20000, 32768])
@pytest.mark.parametrize("ht,yt", [("f32", "f32"), ("bf16", "f32"), ("f16", "bf16"), ("bf16", "f16")])
def test_norm_sizes(d, ht, yt):
    g = gen(d)
    for T, gk in ((1, "channel"), (3, "full"), (70, "none")):
        h, y = rnd(g, T, d, scale=3, dtype=TYPES[ht]), rnd(g, T, d, dtype=TYPES[yt])
        pw, qw = 1 + rnd(g, d, scale=0.1), 1 + rnd(g, d, scale=0.1)
        gate = {"none": None, "channel": torch.sigmoid(rnd(g, d)), "full": torch.sigmoid(rnd(g, T, d)).to(TYPES[yt])}[gk]
        gh, gx = m.block_norm(h, y, pw, gate, qw, res_scale=0.75, block_scale=1.25)
        assert gh.dtype == TYPES[ht] and gx.dtype == TYPES[yt]
        check_norm(h, y, pw, gate, qw, ht, yt, gh, gx, 0.75, 1.25)


@pytest.mark.parametrize("parts", ["pre", "post", "sum", "both"])
@pytest.mark.parametrize("extra,shift", [(0, 0), (4, 0), (3, 0), (4, 4), (2, 1)])
def test_norm_parts_and_strides(parts, extra, shift):
    g = gen(7)
    T, d = 5, 96
    h, y = strided(rnd(g, T, d), extra, shift), strided(rnd(g, T, d, dtype=torch.bfloat16), extra, shift)
    w1, w2 = 1 + rnd(g, d + shift, scale=0.1)[shift:], 1 + rnd(g, d + shift, scale=0.1)[shift:]
    gate = strided(rnd(g, T, d, dtype=torch.float16), extra, shift)
    ho, xo = strided(torch.zeros(T, d, device="cuda"), extra, shift), strided(torch.zeros(T, d, device="cuda"), extra, shift)
    if parts == "pre":
        gh, gx = m.block_norm(h, pre_w=w2, x_out=xo)
        assert gh is h
        check_norm(h, None, None, None, w2, "f32", "f32", None, gx)
    elif parts == "post":
        gh, gx = m.block_norm(h, y, w1, gate, h_out=ho)
        assert gx is None
        check_norm(h, y, w1, gate, None, "f32", "f32", gh, None)
    elif parts == "sum":  # no norm of the block, no gate
        gh, gx = m.block_norm(h, y, pre_w=w2, h_out=ho, x_out=xo, block_scale=-2.0)
        check_norm(h, y, None, None, w2, "f32", "f32", gh, gx, 1.0, -2.0)
    else:
        gh, gx = m.block_norm(h, y, w1, gate, w2, h_out=ho, x_out=xo)
        check_norm(h, y, w1, gate, w2, "f32", "f32", gh, gx)
    for t in (ho, xo):  # nothing beside the rows is touched
        base = t._base
        assert bool((base[:, :shift] == 7.5).all()) and bool((base[:, shift + d:] == 7.5).all())


def test_norm_more_rows_than_a_grid_dimension():
    """Small rows by the million (a norm per head, say): the rows on both sides of 2^21 and the last ones."""
    T, d = (1 << 22) + 5, 8
    g = gen(3)
    h, y = rnd(g, T, d, dtype=torch.bfloat16), rnd(g, T, d, dtype=torch.bfloat16)
    w = rnd(g, d)
    gh, gx = m.block_norm(h, y, w, None, w)
    at = torch.tensor([0, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, (1 << 22) - 1, 1 << 22, T - 1], device="cuda")
    check_norm(h[at], y[at], w, None, w, "bf16", "bf16", gh[at], gx[at])


def test_norm_in_place():
    g = gen(3)
    h, y, w1, w2 = rnd(g, 9, 2816), rnd(g, 9, 2816), 1 + rnd(g, 2816), 1 + rnd(g, 2816)
    want = m.block_norm(h, y, w1, None, w2)
    hh, yy = h.clone(), y.clone()
    got = m.block_norm(hh, yy, w1, None, w2, h_out=hh, x_out=yy)
    assert got[0] is hh and got[1] is yy
    assert torch.equal(hh, want[0]) and torch.equal(yy, want[1])


def test_norm_special_rows():
    g = gen(4)
    h, y, w = rnd(g, 6, 300), rnd(g, 6, 300), torch.ones(300, device="cuda")
    h[1] = 0
    y[1] = 0            # an all-zero row: eps alone
    y[2, 7] = float("nan")
    h[3, 5] = float("inf")
    gh, gx = m.block_norm(h, y, w, None, w)
    assert bool((gh[1] == 0).all()) and bool((gx[1] == 0).all())
    assert bool(gh[2].isnan().all()) and bool(gx[2].isnan().all())
    for r in (0, 4, 5):
        check_norm(h[r:r + 1], y[r:r + 1], w, None, w, "f32", "f32", gh[r:r + 1], gx[r:r + 1])
    assert bool(torch.isinf(gh[3, 5])) and bool(gx[3, 5].isnan())
    e = m.block_norm(h[:0], y[:0], w, None, w)
    assert e[0].shape == (0, 300) and e[1].shape == (0, 300)


def test_norm_refusals():
    g = gen(5)
    h, w = rnd(g, 2, 64), rnd(g, 64)
    with pytest.raises(ValueError):
        m.block_norm(h, rnd(g, 2, 65), w, None, w)
    with pytest.raises(ValueError):
        m.block_norm(h, h.double(), w, None, w)
    with pytest.raises(ValueError):
        m.block_norm(h, None, w, None, w)
    with pytest.raises(ValueError):
        m.block_norm(h)
    with pytest.raises(ValueError):
        m.block_norm(h.t(), pre_w=w)
    with pytest.raises(ValueError):
        m.block_norm(h, pre_w=w.half())
    with pytest.raises(ValueError):
        m.block_norm(h, pre_w=w, x_out=torch.empty(3, 64, device="cuda"))
    with pytest.raises(MoeError):
        m.block_norm(h, pre_w=w, eps=-1.0)


# ------------------------------------------------------------------ matrix-vector products

def make_q4(g, rows, cols, group, size=0.01):
    codes = torch.randint(0, 256, (rows, cols // 32, 16), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand((rows, cols // group), generator=g, device="cuda") - 0.5) * 2 * size
    return codes, s.half()


def check_matvec(x, codes, scales, got, ty):
    w = torch.from_numpy(o.q4_values(codes.cpu().numpy(), scales.cpu().numpy())).cuda()
    xd = x.double()
    ref, mag = xd @ w.t(), xd.abs() @ w.abs().t()
    nb = codes.shape[1]
    # x as a pair of binary16 parts keeps 2^-22 of each element, or 2^-38 of the token's largest; 32 to 128
    # products of a group, one scaled add a group, then at most 16 waves and 3 lane steps in float32
    n = 128 + nb + 24
    tiny = xd.abs().amax(1, keepdim=True) * 2.0 ** -38 * w.abs().sum(1)
    tol = (n * U + 2.0 ** -22) * mag + tiny
    tol = tol + HALF[ty] * (ref.abs() + tol) + float(torch.finfo(TYPES[ty]).smallest_normal)
    bad = ((got.double() - ref).abs() > tol)
    assert not bool(bad.any()), ((got.double() - ref).abs() / tol).max()


@pytest.mark.parametrize("rows,cols,group", [
    (1, 32, 32), (15, 64, 32), (16, 96, 32), (17, 128, 128), (100, 160, 32), (1003, 2144, 32), (48, 2816, 64),
    (33, 4160, 64), (64, 6144, 128), (40, 8192, 32), (31, 8256, 64), (20, 12288, 128), (8, 28672, 32), (5003, 704, 32)])
@pytest.mark.parametrize("ty", list(TYPES))
def test_matvec_shapes(rows, cols, group, ty):
    g = gen(rows + cols)
    codes, scales = make_q4(g, rows, cols, group)
    w = m.Q4Matrix(codes, scales)
    for T in (1, 3, 8, 17):
        x = rnd(g, T, cols, scale=2, dtype=TYPES[ty])
        check_matvec(x, codes, scales, m.q4_matvec(x, w), ty)


@pytest.mark.parametrize("T", [2, 4, 5, 7, 9, 12, 16, 31, 32, 33, 63, 64, 65, 100, 257])
@pytest.mark.parametrize("ty", list(TYPES))
def test_matvec_tokens(T, ty):
    g = gen(T)
    codes, scales = make_q4(g, 70, 1184, 32)
    x = rnd(g, T, 1184, dtype=TYPES[ty])
    check_matvec(x, codes, scales, m.q4_matvec(x, m.Q4Matrix(codes, scales)), ty)


@pytest.mark.parametrize("ty,size", [("f32", 1e-30), ("f32", 1e30), ("bf16", 1e-30), ("bf16", 1e30), ("f16", 1e-3),
                                     ("f16", 1e3)])
def test_matvec_magnitudes(ty, size):
    """Any input magnitude; one channel a thousand times the rest; an all-zero token."""
    g = gen(11)
    codes, scales = make_q4(g, 64, 1024, 32)
    x = rnd(g, 4, 1024).float() * size
    x[1, 77] *= 1000 if ty != "f16" else 30
    x[2] = 0
    x = x.to(TYPES[ty])
    got = m.q4_matvec(x, m.Q4Matrix(codes, scales))
    check_matvec(x, codes, scales, got, ty)
    assert bool((got[2] == 0).all())


@pytest.mark.parametrize("ty", list(TYPES))
def test_matvec_strides_and_offsets(ty):
    g = gen(12)
    codes, scales = make_q4(g, 37, 320, 64)
    w = m.Q4Matrix(codes, scales)
    x = rnd(g, 6, 320, dtype=TYPES[ty])
    want = m.q4_matvec(x, w)
    for extra, shift in ((3, 0), (8, 0), (1, 1), (5, 3)):
        out = strided(torch.zeros(6, 37, device="cuda", dtype=TYPES[ty]), extra, shift)
        got = m.q4_matvec(strided(x, extra, shift), w, out=out)
        assert torch.equal(got, want)
        assert bool((out._base[:, :shift] == 7.5).all()) and bool((out._base[:, shift + 37:] == 7.5).all())
    assert torch.equal(m.q4_matvec(x[:1].expand(6, 320), w), want[:1].expand(6, 37))  # row stride 0


@pytest.mark.parametrize("ty", list(TYPES))
def test_matvec_non_finite_tokens(ty):
    """An infinite or NaN element makes its own token's outputs what the formula gives, and no other's."""
    g = gen(13)
    codes, scales = make_q4(g, 40, 256, 32)
    scales = torch.where(scales == 0, 0.001, scales)
    x = rnd(g, 5, 256, dtype=TYPES[ty])
    clean = m.q4_matvec(x, m.Q4Matrix(codes, scales))
    y = x.clone()
    y[1, 10] = float("inf")
    y[3, 200] = float("nan")
    got = m.q4_matvec(y, m.Q4Matrix(codes, scales))
    for t in (0, 2, 4):
        assert torch.equal(got[t], clean[t])
    assert bool(got[3].isnan().all())
    wv = o.q4_values(codes.cpu().numpy(), scales.cpu().numpy())[:, 10]
    e = got[1].double().cpu().numpy()
    assert np.all(np.isnan(e[wv == 0])) and np.all(e[wv > 0] == np.inf) and np.all(e[wv < 0] == -np.inf)


def test_matvec_from_blocks():
    """The interchange layout's bytes (Q4_0 for group 32), split on the host."""
    rng = np.random.default_rng(5)
    for group in (32, 64, 128):
        rows, cols = 19, 384
        codes = rng.integers(0, 256, (rows, cols // 32, 16), dtype=np.uint8)
        s = (rng.standard_normal((rows, cols // group)) * 0.01).astype(np.float16)
        per = group // 32
        raw = np.concatenate([s.view(np.uint8).reshape(rows, -1, 2), codes.reshape(rows, -1, 16 * per)], 2)
        w = m.Q4Matrix.from_blocks(raw, rows, cols, group)
        assert np.array_equal(w.codes.cpu().numpy(), codes) and np.array_equal(w.scales.cpu().numpy(), s)
        x = rnd(gen(1), 2, cols)
        check_matvec(x, w.codes, w.scales, m.q4_matvec(x, w), "f32")


def test_matvec_refusals():
    g = gen(14)
    codes, scales = make_q4(g, 8, 128, 64)
    w = m.Q4Matrix(codes, scales)
    with pytest.raises(ValueError):
        m.Q4Matrix(codes, scales[:, :1].float())
    with pytest.raises(ValueError):
        m.Q4Matrix(codes, torch.zeros(8, 3, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        m.Q4Matrix(codes.transpose(0, 1), scales)
    with pytest.raises(ValueError):
        m.q4_matvec(rnd(g, 1, 127), w)
    with pytest.raises(ValueError):
        m.q4_matvec(rnd(g, 1, 128).double(), w)
    with pytest.raises(ValueError):
        m.q4_matvec(rnd(g, 1, 128).cpu(), w)
    with pytest.raises(ValueError):
        m.q4_matvec(rnd(g, 2, 128), w, out=torch.empty(2, 8, device="cuda", dtype=torch.float16))
    assert m.q4_matvec(rnd(g, 0, 128), w).shape == (0, 8)


# ------------------------------------------------------------------ the cache

def make_batch(new, past, P, seed, slack=2, max_pages=None):
    """pages, start, past tensors; every sequence on its own pages in a shuffled order."""
    rng = np.random.default_rng(seed)
    n = [(a + b + P - 1) // P for a, b in zip(new, past)]
    order = rng.permutation(sum(n) + slack)
    pages = np.full((len(new), max_pages or max(max(n), 1) + 1), -1, np.int32)
    at = 0
    for s, k in enumerate(n):
        pages[s, :k] = order[at:at + k]
        at += k
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    return t(pages), t(start), t(past), int(sum(n) + slack)


def where(pages, past, new, P):
    """(page, offset) of every new token; page -1 where there is none."""
    pg = pages.cpu().numpy()
    out = []
    for s, n in enumerate(new):
        for i in range(n):
            p = int(past[s]) + i
            ok = 0 <= p // P < pg.shape[1]
            out.append((int(pg[s, p // P]) if ok else -1, p % P))
    return out


def cache_bytes(c):
    return [t.clone() for t in c.tensors]


@pytest.mark.parametrize("D,Hkv,G,P", [(64, 1, 1, 16), (64, 3, 2, 48), (128, 8, 4, 64), (128, 2, 5, 16), (256, 4, 2, 32)])
@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("rot,inter", [(0, False), (None, False), (None, True), (32, False), (2, True)])
def test_append_and_read(D, Hkv, G, P, ty, rot, inter):
    """Codes and scales bit for bit, everything else in the pool untouched, rows behind the last sequence too."""
    g = gen(D + P)
    rot = D if rot is None else rot
    new, past = [1, 17, 0, 3, 40], [0, 5, 9, 100003, P - 1]
    pages, start, pst, n = make_batch(new, past, P, D)
    T, pad = sum(new), 3
    c = m.KVCache.create(n, P, Hkv, D)
    for t in c.tensors:
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.view(torch.uint8).shape, generator=g, device="cuda", dtype=torch.uint8))
    before = cache_bytes(c)
    qkv = rnd(g, T + pad, (G * Hkv + 2 * Hkv) * D, scale=2, dtype=TYPES[ty])
    a, b = G * Hkv * D, (G * Hkv + Hkv) * D
    q, k, v = qkv[:, :a], qkv[:, a:b], qkv[:, b:]
    f = torch.from_numpy((10000.0 ** (-np.arange(rot // 2) * 2 / max(rot, 1))).astype(np.float32)).cuda() if rot else None
    qo = torch.full((T + pad, a), 7.5, device="cuda", dtype=TYPES[ty])
    assert c.append(k, v, pages, start, pst, q=q, inv_freq=f, interleaved=inter, q_out=qo) is qo
    pos = np.concatenate([np.arange(p, p + w) for p, w in zip(past, new)])
    inv = None if f is None else f.cpu().numpy()
    rk = o.rotate(f64(k[:T]).reshape(T, Hkv, D), pos, inv, inter)
    rq = o.rotate(f64(q[:T]).reshape(T, G * Hkv, D), pos, inv, inter).reshape(T, -1)
    got = qo[:T].float().cpu().numpy()
    # binary64 rounded to float32 (half a step of it), then to the type; sines may differ in the last place of
    # binary64, far below
    assert np.all(np.abs(got - rq) <= (HALF[ty] + 2 * U) * np.abs(rq) + 2e-7 * (ty == "f16"))
    assert bool((qo[T:] == 7.5).all())
    kc, ks = o.q4_encode(rk)
    vc, vs = o.q4_encode(f64(v[:T]).reshape(T, Hkv, D).astype(np.float32))
    want = [t.cpu().numpy() for t in before]
    for t, (pg, off) in enumerate(where(pages, past, new, P)):
        want[0][pg, :, off] = kc[t, :, :, :16] | (kc[t, :, :, 16:] << 4)
        want[1][pg, :, off] = ks[t]
        want[2][pg, :, off] = (vc[t, :, :, :16] | (vc[t, :, :, 16:] << 4)).transpose(0, 2, 1)
        want[3][pg, :, off] = vs[t]
    for name, t, w in zip(("k_codes", "k_scales", "v_codes", "v_scales"), c.tensors, want):
        assert np.array_equal(t.view(torch.uint8).cpu().numpy(), np.ascontiguousarray(w).view(np.uint8).reshape(t.view(torch.uint8).shape)), name
    gk, gv = c.read(pages, start, pst, T + pad)
    assert np.array_equal(gk[:T].double().cpu().numpy(), o.q4_decode(kc, ks))
    assert np.array_equal(gv[:T].double().cpu().numpy(), o.q4_decode(vc, vs))


def test_append_hard_values():
    """Ties in magnitude, borders between codes, zeros, subnormal and saturating scales, NaN and infinities."""
    D, P = 64, 16
    rows = []
    x = np.zeros(32, np.float32)
    rows.append(x.copy())                                        # all zero
    x[:] = 1.0; x[3] = -8.0; x[9] = 8.0; rows.append(x.copy())   # tie: the first one, -8, gives scale +1
    x[:] = 0.0; x[3] = 8.0; x[9] = -8.0; rows.append(x.copy())   # the first one, +8, gives scale -1
    x[:] = np.arange(32) / 2 - 8; rows.append(x.copy())          # every border n - 1/2 of scale 1, exactly
    rows.append(-x)
    rows.append(np.nextafter(x, np.float32(9)))
    rows.append(np.nextafter(x, np.float32(-9)))
    rows.append((x * 2.0 ** -26).astype(np.float32))             # subnormal scale
    rows.append((x * 2.0 ** -40).astype(np.float32))             # scale rounds to zero
    rows.append((x * np.float32(1e30)).astype(np.float32))       # scale saturates
    y = x.copy(); y[5] = np.nan; rows.append(y)
    y = x.copy(); y[6] = np.inf; rows.append(y)
    y = x.copy(); y[7] = -np.inf; y[8] = np.inf; rows.append(y)
    rows.append(np.full(32, np.nan, np.float32))
    if len(rows) % 2:
        rows.append(np.zeros(32, np.float32))
    X = np.stack(rows).reshape(-1, 1, D)
    T = X.shape[0]
    pages, start, past, n = make_batch([T], [0], P, 1)
    c = m.KVCache.create(n, P, 1, D)
    k = torch.from_numpy(X.reshape(T, D)).cuda()
    c.append(k, k.clone(), pages, start, past)
    code, s = o.q4_encode(X)
    gk, gv = c.read(pages, start, past, T)
    want = o.q4_decode(code, s)
    assert np.array_equal(gk.double().cpu().numpy(), want) and np.array_equal(gv.double().cpu().numpy(), want)
    assert np.all(np.isfinite(want))


def test_append_holes():
    """Bad pages, positions past the table and negative pasts write nothing; q is rotated for valid pasts all the same."""
    D, P, Hkv = 64, 16, 2
    g = gen(2)
    new, past = [40, 4, 4], [0, -3, 60]
    pages = torch.tensor([[0, 99, 2], [3, 4, 5], [6, 7, -7]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 40, 44, 48], dtype=torch.int32, device="cuda")
    pst = torch.tensor(past, dtype=torch.int32, device="cuda")
    c = m.KVCache.create(8, P, Hkv, D)
    k = rnd(g, 48, Hkv * D)
    c.append(k, k, pages, start, pst)
    gk, _ = c.read(pages, start, pst, 48)
    wrote = {(pg, off) for t, (pg, off) in enumerate(where(pages, past, new, P)) if t < 40 and 0 <= pg < 8}
    s = c.tensors[1]
    for pg in range(8):
        for off in range(P):
            assert bool((s[pg, :, off] != 0).any()) == ((pg, off) in wrote), (pg, off)
    assert bool((gk[16:32] == 0).all()) and bool((gk[44:] == 0).all()) and bool((gk[:16] != 0).any())


def test_read_and_append_with_a_negative_past():
    """Rows of a negative past read 0, whatever stood in the output; their queries have no position and stay."""
    from expert_cache_host_amd.decoder import _library
    D, P, Hkv = 64, 16, 2
    g = gen(6)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    pages, start, past = t([[0, 1], [2, 3], [4, 5]]), t([0, 3, 8, 10]), t([4, -2, 0])
    c = m.KVCache.create(6, P, Hkv, D)
    k = rnd(g, 12, Hkv * D)
    for freq in (None, torch.ones(32, device="cuda"), torch.ones(3, device="cuda")):
        q_out = torch.full((12, Hkv * D), 7.5, device="cuda")
        c.append(k, k, pages, start, past, q=k, inv_freq=freq, q_out=q_out)
        kept = (q_out == 7.5).all(1)
        assert kept.tolist() == [False] * 3 + [True] * 5 + [False] * 2 + [True] * 2
        out = torch.full((2, 12, Hkv * D), 7.5, device="cuda")
        b = c._batch(pages, start, past, 12)
        assert _library().moe_kv_read(c._cp, b, out[0].data_ptr(), out[1].data_ptr(),
                                      torch.cuda.current_stream().cuda_stream) == 0
        assert bool((out[:, 3:8] == 0).all()) and bool((out[:, 10:] == 7.5).all())
        assert bool((out[:, :3] != 7.5).all()) and bool((out[:, 8:10] != 7.5).all())


# ------------------------------------------------------------------ attention

def fill_cache(g, n, P, Hkv, D, garbage=True, size=0.3):
    """A pool of random codes; with `garbage`, places the batch does not hold carry NaN and infinite scales."""
    c = m.KVCache.create(n, P, Hkv, D)
    for t in (c.tensors[0], c.tensors[2]):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device="cuda", dtype=torch.uint8))
    for t in (c.tensors[1], c.tensors[3]):
        t.copy_((torch.rand(t.shape, generator=g, device="cuda") - 0.5) * 2 * size)
    return c


def spoil(c, pages, total, P):
    """NaN and infinite scales everywhere no key of the batch lies."""
    held = torch.zeros(c.n_pages, P, dtype=torch.bool)
    pg = pages.cpu().numpy()
    for s, n in enumerate(total):
        for p in range(n):
            if 0 <= p // P < pg.shape[1] and 0 <= pg[s, p // P] < c.n_pages:
                held[int(pg[s, p // P]), p % P] = True
    out = ~held.cuda()
    for t in (c.tensors[1], c.tensors[3]):
        t[out.unsqueeze(1).expand(-1, c.kv_heads, -1)] = float("nan")
    c.tensors[3][out.unsqueeze(1).expand(-1, c.kv_heads, -1)] = float("inf")


def check_attend(c, q, pages, start, past, scale, window, got, ty, rows=None):
    P, D, Hkv = c.page_tokens, c.head_dim, c.kv_heads
    H = q.shape[1] // D
    pg, st, ps = pages.cpu().numpy(), start.cpu().numpy(), past.cpu().numpy()
    kq, ks, vq, vs = (t.cpu().numpy() for t in c.tensors)
    qn, gn = f64(q).reshape(-1, H, D), f64(got).reshape(-1, H, D)
    for s in range(len(ps)):
        L = max(0, min(int(ps[s]) + int(st[s + 1] - st[s]), pg.shape[1] * P)) if ps[s] >= 0 else 0
        at = np.arange(L)
        page = pg[s, at // P] if L else np.zeros(0, np.int32)
        ok = (page >= 0) & (page < c.n_pages)
        pc = np.where(ok, page, 0)
        kk = o.q4_decode(np.concatenate([kq[pc, :, at % P] & 15, kq[pc, :, at % P] >> 4], -1), ks[pc, :, at % P])
        vt = vq[pc, :, at % P].transpose(0, 1, 3, 2)
        vv = o.q4_decode(np.concatenate([vt & 15, vt >> 4], -1), vs[pc, :, at % P])
        sk, sv = (np.repeat(np.abs(a[pc, :, at % P].astype(np.float64)), 32, -1) for a in (ks, vs))
        for t in range(int(st[s]), int(st[s + 1])):
            if rows is not None and t not in rows:
                continue
            pos = int(ps[s]) + t - int(st[s])
            seen = ok & (at <= pos) & ((at > pos - window) if window else True) if ps[s] >= 0 else ok
            ref = o.attend(qn[t], kk, vv, seen, scale)
            if not seen.any():
                assert np.all(gn[t] == 0)
                continue
            G = H // Hkv
            idx = np.nonzero(seen)[0]
            n = len(idx)
            for h in range(H):
                kh, vh = kk[idx, h // G], vv[idx, h // G]
                mag = np.abs(kh) @ np.abs(qn[t, h]) * abs(scale)
                z = kh @ qn[t, h] * scale
                p = np.exp(z - z.max())
                p /= p.sum()
                # a score: 32 products a block, D / 32 scaled adds, the pair of query parts (2^-22) and three
                # factors; its exponential carries the absolute error of score and reference plus 2 ulp.
                # The products are of codes 0..15 as stored and the offset of 8 is subtracted as a sum of its
                # own, so a rounding is u of up to (15 + 8) scale |q|, whatever |code - 8| is
                raw = 23 * sk[idx, h // G] @ np.abs(qn[t, h]) * abs(scale)
                dz = (32 + D // 32 + 8) * U
                ep = 2 * (dz * raw + 2.0 ** -22 * mag + 4 * U * (np.abs(z) + np.abs(z.max()))) + 8 * U
                # the weighted sum: probabilities times scales in binary16 (one part for half-width types, a
                # pair for float32), sums of n terms; both sums share the probabilities' error
                part = 2.0 ** -11 if ty != "f32" else 2.0 ** -21
                avg = np.abs(vh).T @ (p * (2 * ep + 2 * (ep * p).sum() + part))
                # its roundings likewise: u of up to 23 scale p a term
                avg += 2 * (n + 40) * U * 23 * (sv[idx, h // G].T @ p)
                tol = avg + n * 2.0 ** -32 * np.abs(vh).max() * p.max()
                tol = tol + HALF[ty] * (np.abs(ref[h]) + tol) + float(torch.finfo(TYPES[ty]).smallest_normal)
                bad = np.abs(gn[t, h] - ref[h]) / tol
                assert bad.max() <= 1, (s, t, h, bad.max())


@pytest.mark.parametrize("D,Hkv,G,P", [(64, 2, 1, 16), (64, 1, 3, 48), (128, 2, 4, 64), (128, 1, 8, 16), (128, 1, 17, 32),
                                       (256, 2, 2, 32), (256, 1, 5, 16)])
@pytest.mark.parametrize("ty", list(TYPES))
def test_attend_decode(D, Hkv, G, P, ty):
    """One token per sequence, contexts from the token alone to a few thousand keys, garbage all around."""
    g = gen(D + G)
    past = [0, 1, 14, 15, 16, 31, 32, 63, 255, 700, 2500]
    new = [1] * len(past)
    pages, start, pst, n = make_batch(new, past, P, G)
    c = fill_cache(g, n, P, Hkv, D)
    spoil(c, pages, [a + 1 for a in past], P)
    q = rnd(g, len(past), Hkv * G * D, scale=1.5, dtype=TYPES[ty])
    got = c.attend(q, pages, start, pst, D ** -0.5)
    check_attend(c, q, pages, start, pst, D ** -0.5, 0, got, ty)


@pytest.mark.parametrize("D,Hkv,G,P,window", [(128, 2, 4, 32, 0), (128, 1, 5, 16, 7), (64, 2, 1, 16, 33), (256, 1, 8, 48, 64),
                                              (64, 1, 16, 64, 1), (256, 1, 1, 16, 100)])
@pytest.mark.parametrize("ty", list(TYPES))
def test_attend_chunks(D, Hkv, G, P, window, ty):
    """Ragged chunks of new tokens, empty sequences among them, with and without a window, strided rows."""
    g = gen(D + window)
    new, past = [1, 0, 37, 5, 130], [9, 3, 0, 333, 64]
    pages, start, pst, n = make_batch(new, past, P, D)
    c = fill_cache(g, n, P, Hkv, D)
    spoil(c, pages, [a + b for a, b in zip(new, past)], P)
    T = sum(new)
    q = strided(rnd(g, T, Hkv * G * D, dtype=TYPES[ty]), 8)
    out = strided(torch.zeros(T, Hkv * G * D, dtype=TYPES[ty], device="cuda"), 3)
    got = c.attend(q, pages, start, pst, 0.2, window=window, out=out)
    check_attend(c, q, pages, start, pst, 0.2, window, got, ty)
    assert bool((out._base[:, -3:] == 7.5).all())


def test_attend_rows_of_no_sequence_and_holes():
    D, P, Hkv, G = 128, 16, 2, 2
    g = gen(8)
    pages = torch.tensor([[3, -1, 5, 1000], [-1, -1, -1, -1], [2, 4, 6, 7], [0, 1, 8, 9]], dtype=torch.int32, device="cuda")
    past = torch.tensor([61, 20, -5, 70], dtype=torch.int32, device="cuda")
    start = torch.tensor([1, 4, 6, 8, 9], dtype=torch.int32, device="cuda")
    c = fill_cache(g, 10, P, Hkv, D)
    T = 12
    q = rnd(g, T, Hkv * G * D)
    out = torch.full((T, Hkv * G * D), 7.5, device="cuda")
    c.attend(q, pages, start, past, 0.1, out=out)
    # the last sequence stands past its table: it sees all 64 keys of it, not its own
    check_attend(c, q, pages, start, past, 0.1, 0, out, "f32")
    assert bool((out[0] == 7.5).all()) and bool((out[9:] == 7.5).all())
    assert bool((out[4:8] == 0).all())
    # a window that lies wholly in a hole leaves the row empty
    out2 = c.attend(q[:1], pages[:1].contiguous(), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                    torch.tensor([30], dtype=torch.int32, device="cuda"), 0.1, window=9)
    assert bool((out2 == 0).all())


@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("ksize,vsize,qsize", [(3.0, 1e-4, 1.0), (1e-4, 900.0, 1.0), (0.3, 0.3, 100.0), (0.3, 6e-8, 1e-3)])
def test_attend_magnitudes(ty, ksize, vsize, qsize):
    """Peaked and flat rows, tiny and large values: the precision does not depend on the values' size."""
    D, P, Hkv, G = 128, 32, 1, 4
    g = gen(21)
    new, past = [2, 1], [800, 50]
    pages, start, pst, n = make_batch(new, past, P, 3)
    c = fill_cache(g, n, P, Hkv, D)
    c.tensors[1].copy_(((torch.rand(c.tensors[1].shape, generator=g, device="cuda") - 0.5) * 2 * ksize))
    c.tensors[3].copy_(((torch.rand(c.tensors[3].shape, generator=g, device="cuda") - 0.5) * 2 * vsize))
    c.tensors[3][::2] *= 0.01  # pages of very different size
    q = rnd(g, 3, Hkv * G * D, scale=qsize, dtype=TYPES[ty])
    got = c.attend(q, pages, start, pst, D ** -0.5)
    check_attend(c, q, pages, start, pst, D ** -0.5, 0, got, ty)


@pytest.mark.parametrize("ty,qsize,ksize,scale", [
    (ty, *a) for a in [(1e3, 30.0, 0.1), (6e4, 500.0, 0.1), (6e4, 500.0, -0.1), (1e12, 0.3, 0.1), (1e30, 0.3, 0.1),
                       (3e38, 0.3, 0.1), (3e38, 0.3, -1e-30), (1e-30, 500.0, 1e38)]
    for ty in TYPES if ty != "f16" or a[0] < 65504 and a[0] > 1e-7])
def test_attend_scores_beyond_an_exponential(ty, qsize, ksize, scale):
    """Scores so far apart that the softmax is the largest one's key alone, up to where float32 cannot hold them."""
    for D, Hkv, G in ((64, 1, 2), (128, 1, 4), (256, 2, 1)):
        P, g = 32, gen(D + 1)
        new, past = [3, 1], [700, 90]
        pages, start, pst, n = make_batch(new, past, P, 7)
        c = fill_cache(g, n, P, Hkv, D)
        c.tensors[1].copy_((torch.rand(c.tensors[1].shape, generator=g, device="cuda") - 0.5) * 2 * ksize)
        q = ((torch.rand(4, Hkv * G * D, generator=g, device="cuda") - 0.5) * 2 * qsize).to(TYPES[ty])
        got = f64(c.attend(q, pages, start, pst, scale)).reshape(4, Hkv * G, D)
        total = torch.tensor([a + b for a, b in zip(new, past)])
        every = torch.tensor([0, int(total[0]), int(total.sum())], dtype=torch.int32, device="cuda")
        kk, vv = (f64(x) for x in c.read(pages, every, torch.zeros_like(pst), int(every[-1])))
        qn, checked = f64(q).reshape(4, Hkv * G, D), 0
        for t in range(4):
            s, i = (0, t) if t < 3 else (1, 0)
            at = slice(int(every[s]), int(every[s]) + past[s] + i + 1)
            for h in range(Hkv * G):
                k, v = kk[at, h // G], vv[at, h // G]
                z, mag = k @ qn[t, h] * scale, np.abs(k) @ np.abs(qn[t, h]) * abs(scale)
                top = int(z.argmax())
                # float32 sums: see check_attend, 8 times the magnitudes stands for codes as stored; 100 apart
                # leaves e^-100
                if not (np.delete(z, top) + 100 + 64 * U * 8 * (mag.max() + np.abs(z).max()) < z[top]).all():
                    continue
                checked += 1
                part = 2.0 ** -11 if ty != "f32" else 2.0 ** -21
                assert np.all(np.abs(got[t, h] - v[top]) <= (part + 40 * U + HALF[ty]) * 1.01 * np.abs(v[top])
                              + 8 * U * 23 * 0.3), (D, t, h)
        assert checked >= 2 * Hkv * G


def test_attend_shared_prefix_and_many_sequences():
    """300 sequences in one call (more than one probe of the search), many of them on the same prefix pages."""
    D, P, Hkv, G, S = 64, 16, 2, 2, 300
    g = gen(23)
    rng = np.random.default_rng(3)
    past = rng.integers(0, 90, S)
    pages = np.full((S, 6), -1, np.int32)
    for s in range(S):
        k = (past[s] + P) // P
        pages[s, :k] = [(s % 7) * 6 + j if j + 1 < k else 42 + s for j in range(k)]
    new = np.ones(S, np.int64)
    new[[5, 100, 299]] = 0
    new[[50, 250]] = 7
    start = np.concatenate([[0], np.cumsum(new)])
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    c = fill_cache(g, 42 + S, P, Hkv, D)
    q = rnd(g, int(start[-1]), Hkv * G * D)
    got = c.attend(q, t(pages), t(start), t(past), D ** -0.5)
    check_attend(c, q, t(pages), t(start), t(past), D ** -0.5, 0, got, "f32")


def test_rows_past_the_tensors_are_not_touched():
    """start may promise more rows than the tensors hold (n_rows): those are neither read nor written."""
    D, P, Hkv, G = 128, 16, 1, 2
    g = gen(24)
    pages = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
    start = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    past = torch.tensor([3], dtype=torch.int32, device="cuda")
    c = fill_cache(g, 8, P, Hkv, D)
    before = [t.clone() for t in c.tensors]
    q, k = rnd(g, 64, Hkv * G * D), rnd(g, 64, Hkv * D)
    full = torch.full((64, Hkv * G * D), 7.5, device="cuda")
    c.append(k[:10], k[:10], pages, start, past, q=q[:10], q_out=full[:10])
    assert bool((full[10:] == 7.5).all())
    for t, b in zip(c.tensors, before):
        flat, old = t.transpose(1, 2).reshape(8 * P, -1), b.transpose(1, 2).reshape(8 * P, -1)
        assert torch.equal(flat[:3], old[:3]) and torch.equal(flat[13:], old[13:])
    full.fill_(7.5)
    c.attend(q[:10], pages, start, past, 0.1, out=full[:10])
    assert bool((full[10:] == 7.5).all())
    check_attend(c, q, pages, torch.tensor([0, 10], dtype=torch.int32), past, 0.1, 0, full, "f32")


@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (256, 2)])
@pytest.mark.parametrize("ty", list(TYPES))
def test_attend_garbage_beside_the_window_and_past_the_rows(D, G, ty):
    """Keys on valid pages that no row sees (left of every row's window, or of tokens that the tensors do not
    hold) may carry NaN and infinite scales: the result is the same bit for bit."""
    P, Hkv = 32, 2
    g = gen(D + 5)
    new, past, window = [3, 1, 2, 40], [70, 45, 5, 90], 20
    pages, start, pst, n = make_batch(new, past, P, 5)
    c = fill_cache(g, n, P, Hkv, D)
    T = sum(new) - 33  # of the last sequence's tokens the tensors hold 7
    q = rnd(g, T, Hkv * G * D, dtype=TYPES[ty])
    for w in (window, 0):
        want = c.attend(q, pages, start, pst, D ** -0.5, window=w)
        bad = m.KVCache(*(t.clone() for t in c.tensors))
        pg = pages.cpu().numpy()
        for s, (a, b) in enumerate(zip(new, past)):
            b_live = b + (a if s < 3 else 7)
            unseen = list(range(max(0, b + 1 - w))) if w else []
            for p in unseen + list(range(b_live, b + a)):
                bad.tensors[1][int(pg[s, p // P]), :, p % P] = float("nan")
                bad.tensors[3][int(pg[s, p // P]), :, p % P] = float("inf" if p % 3 else "nan")
        got = bad.attend(q, pages, start, pst, D ** -0.5, window=w)
        assert bool(got.isfinite().all()) and torch.equal(got, want), w


def test_workspace_stays_bounded():
    """A long prompt over a long table asks for no workspace that grows with both."""
    from expert_cache_host_amd.decoder import _KvBatch, _library
    c = m.KVCache.create(4, 64, 8, 128)
    for rows, seqs in ((1, 1), (32, 32), (512, 1), (8192, 1), (100000, 64), (4096, 4096)):
        b = _KvBatch(4096, 4096, 4096, seqs, 4096, rows)
        for ty in (0, 1):
            n = _library().moe_kv_attend_workspace(c._cp, b, ty, 64, 0)
            assert 0 <= n <= 300 << 20, (rows, seqs, ty, n)


def test_attend_long():
    """Long contexts (many splits), a few rows checked in full."""
    D, P, Hkv, G = 128, 64, 2, 4
    g = gen(31)
    new, past = [1, 1, 3], [70000, 3, 33333]
    pages, start, pst, n = make_batch(new, past, P, 3)
    c = fill_cache(g, n, P, Hkv, D)
    q = rnd(g, 5, Hkv * G * D, scale=2)
    got = c.attend(q, pages, start, pst, D ** -0.5)
    check_attend(c, q, pages, start, pst, D ** -0.5, 0, got, "f32")


def test_cache_offsets_past_32_bits():
    """A pool whose code and scale offsets pass 2^32: append, read and attend on its last pages."""
    D, P, Hkv = 256, 64, 8
    n = (1 << 32) // (Hkv * P * D // 2) + 9     # codes past 4 GiB
    c = m.KVCache(*(torch.empty(s, dtype=t, device="cuda") for s, t in (
        ((n, Hkv, P, 8, 16), torch.uint8), ((n, Hkv, P, 8), torch.float16),
        ((n, Hkv, P, 16, 8), torch.uint8), ((n, Hkv, P, 8), torch.float16))))
    pages = torch.tensor([[n - 1, n - 3, 0]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    past = torch.tensor([0], dtype=torch.int32, device="cuda")
    g = gen(41)
    k, v = rnd(g, 100, Hkv * D), rnd(g, 100, Hkv * D)
    c.append(k, v, pages, start, past)
    gk, gv = c.read(pages, start, past, 100)
    kc, ks = o.q4_encode(k.cpu().numpy().reshape(100, Hkv, D))
    vc, vs = o.q4_encode(v.cpu().numpy().reshape(100, Hkv, D))
    kd, vd = o.q4_decode(kc, ks), o.q4_decode(vc, vs)
    assert np.array_equal(gk.double().cpu().numpy(), kd) and np.array_equal(gv.double().cpu().numpy(), vd)
    q = rnd(g, 100, Hkv * D)
    out = c.attend(q, pages, start, past, D ** -0.5)
    for t in (0, 63, 64, 99):
        ref = o.attend(f64(q[t]).reshape(Hkv, D), kd, vd, np.arange(100) <= t, D ** -0.5)
        assert np.abs(f64(out[t]).reshape(Hkv, D) - ref).max() < 1e-4 * np.abs(ref).max()


# ------------------------------------------------------------------ streams, graphs, together

def small_layer(seed):
    """A decoder layer's parts at a small size, Q4 projections, a paged cache and the MoE layer's operands."""
    g = gen(seed)
    d, Hkv, G, D, P = 256, 2, 2, 64, 16
    n = (G + 2) * Hkv * D
    qkv = make_q4(g, n, d, 32, 0.02)
    out = make_q4(g, d, G * Hkv * D, 64, 0.02)
    return dict(g=g, d=d, Hkv=Hkv, G=G, D=D, P=P, qkv=qkv, o=out, w=[1 + rnd(g, d, scale=0.1) for _ in range(4)],
                f=torch.from_numpy((10000.0 ** (-np.arange(D // 2) * 2 / D)).astype(np.float32)).cuda())


def attention_half(L, cache, h, pages, start, past):
    """norm -> projections -> append -> attend -> projection -> residual and the next norm."""
    a, b = L["G"] * L["Hkv"] * L["D"], (L["G"] + 1) * L["Hkv"] * L["D"]
    _, x = m.block_norm(h, pre_w=L["w"][0])
    qkv = m.q4_matvec(x, m.Q4Matrix(*L["qkv"]))
    q = cache.append(qkv[:, a:b], qkv[:, b:], pages, start, past, q=qkv[:, :a], inv_freq=L["f"])
    att = cache.attend(q, pages, start, past, L["D"] ** -0.5)
    y = m.q4_matvec(att, m.Q4Matrix(*L["o"]))
    return m.block_norm(h, y, L["w"][1], None, L["w"][2])


def test_a_whole_layer_with_the_moe_block():
    """The operators around moe_layer_forward as a decode loop uses them, against binary64 end to end."""
    import synth
    from oracle.layer import moe_layer
    wl = synth.WORKLOADS["tiny"]
    L = small_layer(51)
    assert L["d"] == wl.d_model
    weights = synth.gen_experts(wl, 0)
    w_r, bias = synth.gen_router(wl, 0)
    moe = m.MoECache(1, wl.n_experts, wl.slots, wl.d_model, wl.d_ff, weights, top_k=wl.top_k, miss_mode="host")
    w_d = torch.from_numpy(w_r).cuda()
    cache = m.KVCache.create(16, L["P"], L["Hkv"], L["D"])
    pages = torch.tensor([[1, 3, 5], [2, 8, 9]], dtype=torch.int32, device="cuda")
    past = [0, 0]
    Hkv, G, D = L["Hkv"], L["G"], L["D"]
    keys, vals = [[], []], [[], []]
    wq, wo = (o.q4_values(c.cpu().numpy(), s.cpu().numpy()) for c, s in (L["qkv"], L["o"]))
    wn = [f64(w) for w in L["w"]]
    for step, new in enumerate(([19, 2], [1, 1], [1, 1], [1, 1])):
        T = sum(new)
        start = torch.tensor([0, new[0], T], dtype=torch.int32, device="cuda")
        pst = torch.tensor(past, dtype=torch.int32, device="cuda")
        h = rnd(L["g"], T, L["d"])
        h1, x = attention_half(L, cache, h, pages, start, pst)
        y = moe.forward(0, x, w_d, None)
        h2, _ = m.block_norm(h1, y, L["w"][3])
        # the oracle's layer; the 4-bit codes are taken from the cache (checked bit for bit elsewhere): the
        # projections feeding them differ from binary64 by float32 rounding and may fall on the other side of a border
        gk, gv = cache.read(pages, start, pst, T)
        _, ox = o.block_norm(f64(h), pre_w=wn[0])
        pr = ox @ wq.T
        pos = np.concatenate([np.arange(p, p + n) for p, n in zip(past, new)])
        oq = o.rotate(pr[:, :G * Hkv * D].reshape(T, G * Hkv, D), pos, L["f"].cpu().numpy(), False).astype(np.float64)
        att = np.zeros((T, G * Hkv * D))
        row = 0
        for s in range(2):
            keys[s] += list(f64(gk)[row:row + new[s]])
            vals[s] += list(f64(gv)[row:row + new[s]])
            for i in range(new[s]):
                K, V = np.stack(keys[s]), np.stack(vals[s])
                att[row + i] = o.attend(oq[row + i], K, V, np.arange(len(K)) <= past[s] + i, D ** -0.5).ravel()
            row += new[s]
        oh1, ox2 = o.block_norm(f64(h), att @ wo.T, wn[1], None, wn[2])
        assert np.abs(f64(h1) - oh1).max() < 1e-4 * np.abs(oh1).max()
        assert np.abs(f64(x) - ox2).max() < 1e-4 * np.abs(ox2).max()
        ref = moe_layer(f64(x).astype(np.float32), w_r, bias, weights, wl.d_model, wl.d_ff, wl.n_experts, wl.top_k)["out64"]
        oh2, _ = o.block_norm(f64(h1), ref, wn[3])
        # the MoE layer's own bar is 2e-3 of its output's RMS; the norm brings that RMS to about 1
        assert np.abs(f64(h2) - oh2).max() < 1e-2
        past = [p + n for p, n in zip(past, new)]
    moe.close()


def test_same_call_twice_is_bit_equal():
    L = small_layer(52)
    pages = torch.tensor([[1, 3, 5], [2, 8, 9]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 20, 23], dtype=torch.int32, device="cuda")
    past = torch.tensor([11, 0], dtype=torch.int32, device="cuda")
    h = rnd(L["g"], 23, L["d"])
    res = []
    for _ in range(3):
        cache = m.KVCache.create(16, L["P"], L["Hkv"], L["D"])
        res.append([*attention_half(L, cache, h, pages, start, past), *cache.tensors])
    for r in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, res[0]))


def test_other_stream():
    L = small_layer(53)
    pages = torch.tensor([[1, 3], [2, 8]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    past = torch.tensor([17, 4], dtype=torch.int32, device="cuda")
    h = rnd(L["g"], 2, L["d"])
    c1, c2 = (m.KVCache.create(16, L["P"], L["Hkv"], L["D"]) for _ in range(2))
    want = attention_half(L, c1, h, pages, start, past)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = attention_half(L, c2, h, pages, start, past)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the same by the stream argument
    x = rnd(L["g"], 3, L["d"])
    w = m.Q4Matrix(*L["qkv"])
    ref = m.q4_matvec(x, w)
    torch.cuda.synchronize()
    got = m.q4_matvec(x, w, stream=s)
    q = c2.attend(ref[:2, :256].contiguous(), pages, start, past, 0.1, stream=s)
    s.synchronize()
    assert torch.equal(got, ref) and torch.equal(q, c2.attend(ref[:2, :256].contiguous(), pages, start, past, 0.1))


def test_graph_replays():
    """A decode step captured once and replayed with new inputs and positions, eager work between the replays;
    two captured graphs on different streams hold their own workspaces."""
    L = small_layer(54)
    cap, eager = (m.KVCache.create(16, L["P"], L["Hkv"], L["D"]) for _ in range(2))
    pages = torch.tensor([[1, 3, 4], [2, 8, 7]], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    past = torch.tensor([0, 0], dtype=torch.int32, device="cuda")
    h = rnd(L["g"], 2, L["d"])
    attention_half(L, cap, h, pages, start, past)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = attention_half(L, cap, h, pages, start, past)
    for t in cap.tensors:
        t.zero_()
    for step in range(40):
        h.copy_(rnd(L["g"], 2, L["d"]))
        graph.replay()
        want = attention_half(L, eager, h, pages, start, past)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), step
        past += 1
    assert all(torch.equal(a, b) for a, b in zip(cap.tensors, eager.tensors))


def test_two_graphs_at_once():
    D, P, Hkv, G = 128, 64, 2, 4
    g = gen(61)
    new, past = [1, 1], [9000, 7000]
    pages, start, pst, n = make_batch(new, past, P, 3)
    c = fill_cache(g, n, P, Hkv, D)
    qs = [rnd(g, 2, Hkv * G * D) for _ in range(2)]
    want = [c.attend(q, pages, start, pst, 0.1).clone() for q in qs]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for q in qs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(c.attend(q, pages, start, pst, 0.1))
        graphs.append(gr)
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()


def test_cache_refusals():
    g = gen(71)
    c = m.KVCache.create(4, 16, 2, 64)
    pages = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    past = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = rnd(g, 1, 128)
    for bad in (dict(k=rnd(g, 1, 127)), dict(v=k.half()), dict(v=rnd(g, 2, 128)), dict(pages=pages.long()),
                dict(pages=pages.cpu()), dict(start=start[:1]), dict(past=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(q=rnd(g, 1, 192)), dict(q=rnd(g, 1, 128).half()), dict(q_out=k), dict(inv_freq=rnd(g, 33)),
                dict(inv_freq=rnd(g, 16).double())):
        a = dict(k=k, v=k, pages=pages, start=start, past=past)
        a.update(bad)
        with pytest.raises(ValueError):
            c.append(**a)
    for bad in (dict(q=rnd(g, 1, 64)), dict(q=rnd(g, 1, 128).double()), dict(out=rnd(g, 1, 128).half()),
                dict(start=start.long())):
        a = dict(q=k, pages=pages, start=start, past=past, scale=1.0)
        a.update(bad)
        with pytest.raises(ValueError):
            c.attend(**a)
    for w in (-1, 1 << 31, (1 << 32) + 5):
        with pytest.raises(ValueError):
            c.attend(k, pages, start, past, 1.0, window=w)
    with pytest.raises(ValueError):
        c.read(pages, start, past, -1)
    with pytest.raises(MoeError):
        c.attend(k, pages, start, past, float("nan"))
    with pytest.raises(ValueError):
        m.KVCache(c.tensors[0], c.tensors[1].float(), c.tensors[2], c.tensors[3])
    with pytest.raises(ValueError):
        m.KVCache(c.tensors[0][:, :, :8].contiguous(), *(t[:, :, :8].contiguous() for t in c.tensors[1:]))
