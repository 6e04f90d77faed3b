"""Corners of the decoder-layer operators on the GPU, against binary64.

Tolerances are derived beside each check, as in test_gpu_decoder.py (u = 2^-24 per
float32 rounding, half a step of the output's type)."""
import numpy as np
import pytest
import torch

import expert_cache_host_amd as m
from oracle import decoder as o
from test_gpu_decoder import HALF, TYPES, U, f64, fill_cache, gen, make_batch

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
