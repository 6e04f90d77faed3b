"""Corners of the decoder-layer operators on the GPU, against binary64.

Tolerances are derived beside each check, as in test_gpu_decoder.py (u = 2^-24 per
float32 rounding, half a step of the output's type)."""
import numpy as np
import pytest
import torch

import expert_cache_host_amd as m
from oracle import decoder as o
from test_gpu_decoder import (HALF, TYPES, U, check_attend, check_matvec, f64, fill_cache, gen, make_batch, make_q4,
                              rnd, spoil)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ attention: scores and value scales far apart

# what the probability times its value scale is rounded to: one binary16 part, or a pair
PART = {"f32": 2.0 ** -21, "bf16": 2.0 ** -11, "f16": 2.0 ** -11}


@pytest.mark.parametrize("n,at", [(250, (10, 20)), (250, (3, 200)), (250, (70, 130, 249)), (6000, (5, 40, 5900)),
                                  (6000, (1000, 3000, 3001, 5999))])
@pytest.mark.parametrize("D,ty,q0,scale,steps", [
    (D, ty, *a) for a in [(2.0 ** 15, 0.5, True), (2.0 ** 15, -0.5, True), (2.0 ** 15, 64.0, False), (2.0 ** 27, 8.0, False)]
    for D, ty in [(64, "f32"), (128, "f32"), (256, "f32"), (64, "bf16"), (128, "bf16"), (128, "f16"), (256, "f16")]
    if ty != "f16" or a[0] < 65504])
def test_attend_close_scores_far_from_zero(D, ty, q0, scale, steps, n, at):
    """Keys whose scores tie, or lie half a unit apart (`steps`), at scores of millions to billions, in one wave, in
    several, and in several parts; the value scales' powers of two differ from wave to wave."""
    P, G, g = 64, 3, gen(n + D)
    pages, start, past, n_pages = make_batch([1], [n - 1], P, 1)
    c = m.KVCache.create(n_pages, P, 1, D)
    pg = pages.cpu().numpy()[0]
    kc = np.full((n, D // 32, 32), 8, np.uint8)      # all other keys score 0
    sign = 1 if scale > 0 else -1
    for i, p in enumerate(at):
        kc[p, 0] = 8 + 7 * sign                      # 32 * 7 * q0, an integer below 2^24 times q0's power of two
        if steps:
            kc[p, 1, 0] = 8 + sign * (i % 3)         # and one more per step: the scores are exact in float32
    vc = torch.randint(0, 16, (n, D // 32, 32), generator=g, device="cuda").cpu().numpy().astype(np.uint8)
    vs = (0.7 * 2.0 ** -(np.arange(n) // 64 * 5 % 13))[:, None].repeat(D // 32, 1).astype(np.float16)
    for p in range(n):
        where = (int(pg[p // P]), 0, p % P)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        if p % P == 0:
            b = min(P, n - p)
            rows = slice(p, p + b)
            c.tensors[0][where[0], 0, :b] = t(kc[rows, :, :16] | kc[rows, :, 16:] << 4)
            c.tensors[1][where[0], 0, :b] = 1.0
            c.tensors[2][where[0], 0, :b] = t((vc[rows, :, :16] | vc[rows, :, 16:] << 4).transpose(0, 2, 1))
            c.tensors[3][where[0], 0, :b] = t(vs[rows])
    q = torch.zeros(1, G, D, device="cuda")
    q[:, :, :32] = q0
    q[:, :, 32] = 1.0
    got = f64(c.attend(q.to(TYPES[ty]).view(1, -1), pages, start, past, scale)).reshape(G, D)
    k, v = o.q4_decode(kc, np.ones_like(vs)), o.q4_decode(vc, vs)
    z = (k @ f64(q)[0, 0]) * scale
    p = np.exp(z - z.max())
    p /= p.sum()
    ref = p @ v
    # scores and their differences are exact; an exponent of at most 32 (64 for the larger scale) carries 2 u of
    # itself twice (unit and product), an exponential and its sums 12 u, twice for numerator and denominator; the
    # parts' rounding, and a product below the largest value scale keeps 2^-36 of that
    mag = p @ np.abs(v)
    tol = (PART[ty] + (4 * 32 + 24) * U) * mag + len(at) * 2.0 ** -35 * 8 * float(vs.max())
    tol = tol + HALF[ty] * (np.abs(ref) + tol)
    assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / tol).max()


def one_sequence(g, n, P, D, ks, vs, Hkv=1):
    """A cache of one sequence of n keys with random codes and the given scales [n, Hkv, D / 32]; what it holds."""
    pages, start, past, n_pages = make_batch([1], [n - 1], P, 1)
    c = fill_cache(g, n_pages, P, Hkv, D)
    pg = pages.cpu().numpy()[0, np.arange(n) // P].astype(np.int64)
    at = (torch.from_numpy(pg).cuda(), slice(None), torch.arange(n, device="cuda") % P)
    c.tensors[1][at] = torch.from_numpy(np.ascontiguousarray(ks.astype(np.float16))).cuda()
    c.tensors[3][at] = torch.from_numpy(np.ascontiguousarray(vs.astype(np.float16))).cuda()
    kq, kf, vq, vf = (t[at].cpu().numpy() for t in c.tensors)
    vq = vq.transpose(0, 1, 3, 2)
    k = o.q4_decode(np.concatenate([kq & 15, kq >> 4], -1), kf)
    v = o.q4_decode(np.concatenate([vq & 15, vq >> 4], -1), vf)
    return c, pages, start, past, k, v


@pytest.mark.parametrize("n", [40, 300, 5000])
@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("D,spread", [(64, 13), (64, 20), (128, 13), (128, 20), (256, 20), (128, 26)])
def test_attend_value_blocks_of_very_different_size(D, spread, ty, n):
    """Blocks of 32 value elements up to 2^spread apart: each keeps its relative precision down to 2^-35 of the
    largest value scale per key."""
    g, nb = gen(n + D), D // 32
    rng = np.random.default_rng(n)
    size = 2.0 ** (spread - 17 - (np.arange(nb) * spread // (nb - 1))[::-1 if n == 300 else 1])
    vs = rng.uniform(0.5, 1, (n, 1, nb)) * size
    c, pages, start, past, k, v = one_sequence(g, n, 32, D, np.zeros((n, 1, nb)), vs)  # all scores are 0
    q = torch.randn(1, 3 * D, generator=g, device="cuda").to(TYPES[ty])
    got = f64(c.attend(q, pages, start, past, D ** -0.5)).reshape(3, D)
    ref, mag, per = v[:, 0].mean(0), np.abs(v[:, 0]).mean(0), np.repeat(size, 32)
    # equal probabilities: the parts' rounding, sums of n terms of codes 0..15 as stored and of their offset of 8
    # (23 value scales a term), and the stated bound
    tol = PART[ty] * mag + 2 * (n + 40) * U * 23 * per + 23 * 2.0 ** -35 * size.max()
    tol = tol + HALF[ty] * (np.abs(ref) + tol) + (2.0 ** -25 if ty == "f16" else 0)
    for h in range(3):
        assert np.all(np.abs(got[h] - ref) <= tol), (h, (np.abs(got[h] - ref) / tol).reshape(nb, 32).max(1))


@pytest.mark.parametrize("ratio", [12, 20, 28])
@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attend_a_large_value_without_weight(D, ty, ratio):
    """A visible key whose value scales are 2^ratio times the others' but whose probability is nothing: the others
    keep what 2^-35 of that scale per key leaves them."""
    n, nb, g = 200, D // 32, gen(D + ratio)
    rng = np.random.default_rng(ratio)
    ks, vs = np.zeros((n, 1, nb)), rng.uniform(0.5, 1, (n, 1, nb)) * 2.0 ** -13
    c, pages, start, past, k, v = one_sequence(g, n, 32, D, ks, vs)
    for p in (3, 90, 150):
        # the first element's key code 0 (value -8) at scale 8: score -64 * 60 against 0
        pg = int(pages[0, p // 32])
        c.tensors[0][pg, 0, p % 32, 0, 0] &= 0xf0
        c.tensors[1][pg, 0, p % 32, 0] = 8.0
        c.tensors[3][pg, 0, p % 32] = 2.0 ** (ratio - 13)
    q = torch.zeros(1, D, device="cuda")
    q[0, 0] = 60
    got = f64(c.attend(q.to(TYPES[ty]), pages, start, past, 1.0)).reshape(D)
    rest = np.setdiff1d(np.arange(n), [3, 90, 150])
    ref = v[rest, 0].mean(0)
    # equal probabilities, exact scores: the parts' rounding, sums of n terms of raw codes, the stated bound
    mag = np.abs(v[rest, 0]).mean(0)
    tol = PART[ty] * mag + 2 * (n + 40) * U * 23 * 2.0 ** -13 + 23 * 2.0 ** (ratio - 13) * 2.0 ** -35
    tol = tol + HALF[ty] * (np.abs(ref) + tol) + (2.0 ** -25 if ty == "f16" else 0)
    assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / tol).max()


# ------------------------------------------------------------------ batches that pass the tensors' ends

@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("D,G,window", [(64, 1, 0), (128, 4, 0), (128, 5, 9), (256, 2, 40)])
def test_sequences_that_begin_before_the_tensors(D, G, window, ty):
    """start may begin below 0: append, read and attention take the rows that the tensors hold, each at its
    position, as the same rows in a longer batch."""
    P, Hkv, g, before = 16, 2, gen(D + G), 150
    start = torch.tensor([-150, -141, -30, 40, 41, 43], dtype=torch.int32, device="cuda")
    past = torch.tensor([4, 9, 33, 70, -3], dtype=torch.int32, device="cuda")
    pages = torch.arange(5 * 16, dtype=torch.int32, device="cuda").view(5, 16)
    T = 47  # four rows of no sequence at the end
    k, v = (torch.randn(before + T, Hkv * D, generator=g, device="cuda").to(TYPES[ty]) for _ in range(2))
    q = torch.randn(before + T, Hkv * G * D, generator=g, device="cuda").to(TYPES[ty])
    f = torch.full((D // 2,), 0.01, device="cuda")
    whole = fill_cache(g, 80, P, Hkv, D)
    held = m.KVCache(*(t.clone() for t in whole.tensors))
    want_q = torch.full_like(q, 7.5)
    whole.append(k, v, pages, start + before, past, q=q, inv_freq=f, q_out=want_q)
    got_q = torch.full_like(q[before:], 7.5)
    held.append(k[before:], v[before:], pages, start, past, q=q[before:], inv_freq=f, q_out=got_q)
    assert torch.equal(got_q, want_q[before:])
    for a, b in zip(whole.read(pages, start + before, past, before + T), held.read(pages, start, past, T)):
        assert torch.equal(a[before:before + 43], b[:43])
    # attention over the whole batch's cache: the same rows in both calls
    want, got = torch.full_like(q, 7.5), torch.full_like(q[before:], 7.5)
    whole.attend(q, pages, start + before, past, 0.1, window=window, out=want)
    whole.attend(q[before:], pages, start, past, 0.1, window=window, out=got)
    assert bool((got[43:] == 7.5).all()) and bool((got[41:43] == 0).all())
    # tiles are cut at other rows, so sums may be joined in another order: see check_attend for the parts
    check_attend(whole, q, pages, start + before, past, 0.1, window, want, ty, rows=range(before, before + 43))
    shifted = torch.cat([want[:before], got])
    check_attend(whole, q, pages, start + before, past, 0.1, window, shifted, ty, rows=range(before, before + 43))


# ------------------------------------------------------------------ the caller's surroundings

def test_an_earlier_error_of_the_caller_fails_no_call():
    """A HIP error that the caller has not fetched yet is neither a call's result nor taken away by it."""
    import ctypes
    hip = ctypes.CDLL(m.lib_path())  # the runtime the library is linked to
    D, P, g = 64, 16, gen(91)
    x, w, out = torch.randn(2, D, generator=g, device="cuda"), torch.ones(D, device="cuda"), torch.empty(2, D, device="cuda")
    c = m.KVCache.create(2, P, 1, D)
    mat = m.Q4Matrix(torch.full((D, D // 32, 16), 0x99, dtype=torch.uint8, device="cuda"),
                     torch.ones(D, D // 32, dtype=torch.float16, device="cuda"))
    pages, start, past = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([[1]], [0, 2], [0]))
    k, f = x.clone(), torch.ones(3, device="cuda")
    read = c.read(pages, start, past, 2)  # allocations are cached from here on
    att = c.attend(x, pages, start, past, 1.0, out=out).clone()
    torch.cuda.synchronize()
    del read, att
    calls = [lambda: m.block_norm(x, pre_w=w, x_out=out), lambda: m.q4_matvec(x, mat, out=out),
             lambda: c.append(k, k, pages, start, past, q=x, q_out=out), lambda: c.read(pages, start, past, 2),
             lambda: c.append(k, k, pages, start, past, inv_freq=f),
             lambda: c.attend(x, pages, start, past, 1.0, out=out)]
    try:
        for call in calls:
            hip.hipGetLastError()
            assert hip.hipSetDevice(4096) != 0
            call()
            assert hip.hipGetLastError() != 0
    finally:
        hip.hipGetLastError()
        torch.cuda.synchronize()
    want = x.double().sum(1, keepdim=True)  # 64 weights of 1: see check_matvec's 160 roundings
    assert bool(((m.q4_matvec(x, mat) - want).abs() <= 160 * U * x.abs().sum(1, keepdim=True)).all())


@pytest.mark.parametrize("op", ["norm", "matvec", "append", "read", "attend"])
def test_tensors_dropped_while_another_stream_reads_them(op):
    """Inputs of a call on another stream may be dropped at once: their memory is not given out before it has run."""
    s, g = torch.cuda.Stream(), gen(92)
    D, T = 64, 513
    new = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    busy = torch.zeros(8192, 8192, device="cuda")
    c = m.KVCache.create(40, 16, 1, D)
    start, past = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([0, T], [0]))
    pages = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40)
    ops = {"norm": lambda t: m.block_norm(t[0], t[1], pre_w=t[2], gate=t[3], post_w=t[4], h_out=t[5], x_out=t[6], stream=s),
           "matvec": lambda t: m.q4_matvec(t[0], m.Q4Matrix(t[1], t[2]), out=t[3], stream=s),
           "append": lambda t: c.append(t[0], t[1], t[2], t[3], t[4], q=t[5], inv_freq=t[6], q_out=t[7], stream=s),
           "read": lambda t: m.KVCache(*t[:4]).read(t[4], t[5], t[6], T, stream=s),
           "attend": lambda t: c.attend(t[0], t[1], t[2], t[3], 1.0, out=t[4], stream=s)}
    make = {"norm": lambda: [new(T, D), new(T, D), new(D), new(T, D), new(D), new(T, D), new(T, D)],
            "matvec": lambda: [new(3, 1024), torch.zeros(512, 32, 16, dtype=torch.uint8, device="cuda"),
                               torch.ones(512, 32, dtype=torch.float16, device="cuda"), new(3, 512)],
            "append": lambda: [new(T, D), new(T, D), pages.clone(), start.clone(), past.clone(), new(T, D),
                               new(D // 2), new(T, D)],
            "read": lambda: [t.clone() for t in c.tensors] + [pages.clone(), start.clone(), past.clone()],
            "attend": lambda: [new(T, D), pages.clone(), start.clone(), past.clone(), new(T, D)]}
    ops[op](make[op]())  # what is loaded at first use
    torch.cuda.synchronize()
    inputs = make[op]()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(30):  # some 10 ms each
            torch.mm(busy, busy)
        done = torch.cuda.Event()
        done.record()
    held = {t.data_ptr(): (t.shape, t.dtype) for t in inputs}
    kept = ops[op](inputs)
    del inputs
    # the same sizes again from the same pool, never written
    again = [torch.empty(shape, dtype=dtype, device="cuda") for shape, dtype in held.values()]
    early = not done.query()
    taken = {t.data_ptr() for t in again} & set(held)
    torch.cuda.synchronize()
    del kept
    assert early, "the stream was not kept busy long enough"
    assert not taken


# ------------------------------------------------------------------ launch shapes of large calls

@pytest.mark.parametrize("rows,cols,group", [(70001, 512, 32), (9001, 4096, 64), (9001, 6144, 128), (6017, 2144, 32),
                                             (9001, 8192, 32), (9001, 8256, 64), (8200, 12288, 128)])
@pytest.mark.parametrize("ty", list(TYPES))
def test_matvec_several_tiles_a_workgroup(rows, cols, group, ty):
    """More tiles of rows than workgroups fit the chip: each takes several in turn, with the next one's loads in
    flight; above 6144 columns one or four tiles a visit (from 5 parts of tokens on), the last visit not full."""
    g = gen(rows + cols)
    codes, scales = make_q4(g, rows, cols, group)
    w = m.Q4Matrix(codes, scales)
    for T in (1, 4, 8, 16, 37):
        x = rnd(g, T, cols, scale=2, dtype=TYPES[ty])
        out = torch.full((T, rows + 3), 7.5, device="cuda", dtype=TYPES[ty])
        m.q4_matvec(x, w, out=out[:, :rows])
        check_matvec(x, codes, scales, out[:, :rows], ty)
        assert bool((out[:, rows:] == 7.5).all())


@pytest.mark.parametrize("D,Hkv,G", [(256, 32, 2), (128, 8, 4), (64, 1, 3)])
@pytest.mark.parametrize("ty", list(TYPES))
@pytest.mark.parametrize("rot,inter", [(64, False), (64, True), (6, False)])
def test_append_and_read_of_long_prompts(D, Hkv, G, ty, rot, inter):
    """More than 512 tokens in a call: fewer workgroups a token, each with several chunks of heads."""
    g, P = gen(D + rot), 48
    new, past = [300, 1, 291], [7, 100, 0]
    pages, start, pst, n = make_batch(new, past, P, D)
    T = sum(new)
    c = m.KVCache.create(n, P, Hkv, D)
    q, k, v = (rnd(g, T, h * D, scale=2, dtype=TYPES[ty]) for h in (G * Hkv, Hkv, Hkv))
    f = torch.from_numpy((1000.0 ** (-np.arange(rot // 2) * 2 / rot)).astype(np.float32)).cuda()
    got = c.append(k, v, pages, start, pst, q=q, inv_freq=f, interleaved=inter).float().cpu().numpy()
    pos = np.concatenate([np.arange(p, p + w) for p, w in zip(past, new)])
    turn = lambda t, h: o.rotate(f64(t).reshape(T, h, D), pos, f.cpu().numpy(), inter)  # noqa: E731
    ref = turn(q, G * Hkv).reshape(T, -1)
    # as in test_append_and_read: binary64 rounded to float32, then to the type
    assert np.all(np.abs(got - ref) <= (HALF[ty] + 2 * U) * np.abs(ref) + 2e-7 * (ty == "f16"))
    gk, gv = c.read(pages, start, pst, T)
    assert np.array_equal(gk.double().cpu().numpy(), o.q4_decode(*o.q4_encode(turn(k, Hkv))))
    assert np.array_equal(gv.double().cpu().numpy(),
                          o.q4_decode(*o.q4_encode(f64(v).reshape(T, Hkv, D).astype(np.float32))))


@pytest.mark.parametrize("ty", list(TYPES))
def test_attend_garbage_around_many_sequences(ty):
    """Shared prefixes, hundreds of sequences and a long one: scales that are NaN or infinite wherever no key of the
    batch lies stay out of every result."""
    D, P, Hkv, G, S = 64, 16, 2, 2, 300
    g, rng = gen(93), np.random.default_rng(4)
    past = rng.integers(0, 90, S)
    past[17] = 9000
    pages = np.full((S, 564), -1, np.int32)
    for s in range(S):
        k = (past[s] + P) // P
        pages[s, :k] = [(s % 7) * 6 + j if j + 1 < k else 42 + s for j in range(k)] if s != 17 else 342 + np.arange(k)
    start = np.arange(S + 1)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    pages, start, past_d = t(pages), t(start), t(past)
    c = fill_cache(g, 342 + 563, P, Hkv, D)
    q = rnd(g, S, Hkv * G * D, dtype=TYPES[ty])
    want = c.attend(q, pages, start, past_d, D ** -0.5)
    # pages 0 .. 41 are shared by sequences of different lengths: those are full up to their last shared page
    spoil(c, pages, [int(p) + 1 for p in past], P)
    got = c.attend(q, pages, start, past_d, D ** -0.5)
    assert torch.equal(got, want)
    check_attend(c, q, pages, start, past_d, D ** -0.5, 0, got, ty, rows=[0, 5, 17, 100, 299])


@pytest.mark.parametrize("D,G", [(64, 1), (128, 4), (256, 2)])
@pytest.mark.parametrize("ty", list(TYPES))
def test_attend_non_finite_queries(D, G, ty):
    """An infinite or NaN element of a query makes that row's head NaN (every visible key's score is infinite or NaN,
    all minus infinity among them) and no other's; a row that sees no key is 0 all the same."""
    P, Hkv, g = 16, 2, gen(94)
    new, past = [1, 1, 4, 1, 1], [0, 3, 60, 2500, -7]
    pages, start, pst, n = make_batch(new, [max(p, 0) for p in past], P, 5)
    pst = torch.tensor(past, dtype=torch.int32, device="cuda")
    c = fill_cache(g, n, P, Hkv, D)
    q = rnd(g, 8, Hkv * G * D, dtype=TYPES[ty])
    sound = q.clone()
    bad = [(t, h, e) for t, h, e in ((0, 0, 3), (1, 0, 0), (3, Hkv * G - 1, D - 1), (4, 0, 17), (6, Hkv * G - 1, 40), (7, 0, 1))]
    for i, (t, h, e) in enumerate(bad):
        for value in (float("inf"), float("-inf"), float("nan")):
            q.copy_(sound)
            q[t, h * D + e] = value
            for scale in (0.1, -0.1):
                got = c.attend(q, pages, start, pst, scale)
                own = got.view(8, Hkv * G, D)[t, h]
                assert bool((own == 0).all() if t == 7 else own.isnan().all()), (t, h, value, scale)
                if i % 2 == 0 and scale > 0:
                    got.view(8, Hkv * G, D)[t, h] = c.attend(sound, pages, start, pst, scale).view(8, Hkv * G, D)[t, h]
                    check_attend(c, sound, pages, start, pst, scale, 0, got, ty, rows=[0, 1, 2, 3, 4, 5])


def test_captured_calls_on_a_given_stream():
    """Calls with a stream argument inside a capture, on the capturing stream and with inputs dropped meanwhile."""
    D, P, g = 64, 16, gen(95)
    codes, scales = make_q4(g, D, D, 32)
    c = m.KVCache.create(4, P, 1, D)
    pages, start, past = (torch.tensor(a, dtype=torch.int32, device="cuda") for a in ([[1, 2], [0, 3]], [0, 2, 3], [0, 17]))
    x, w = rnd(g, 3, D), torch.ones(D, device="cuda")

    def chain(x, w, s):
        _, y = m.block_norm(x, pre_w=w, stream=s)
        y = m.q4_matvec(y, m.Q4Matrix(codes.clone() if s is None else kept[0], scales if s is None else kept[1]), stream=s)
        q = c.append(y, y, pages, start, past, q=y, stream=s)
        return c.attend(q, pages, start, past, 0.1, stream=s), *c.read(pages, start, past, 3, stream=s)

    kept = [codes.clone(), scales.clone()]
    chain(x, w, torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(x, w, torch.cuda.current_stream())
    for _ in range(4):
        x.copy_(rnd(g, 3, D))
        want = chain(x, w, None)
        torch.cuda.synchronize()
        for t in c.tensors:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
