"""The oracle of the operators between a prompt and its next token, against brute force."""
import itertools

import numpy as np
import pytest

from oracle import step as o


def test_q8_rows_nearest():
    r = np.random.default_rng(1)
    x = (r.standard_normal((20, 37)) * 5).astype(np.float32).astype(np.float64)
    x[3] = 0
    x[4, 5] = np.inf
    x[5, 6] = np.nan
    q, s = o.q8_rows(x)
    assert s[3] == 0 and not q[3].any() and np.isnan(s[4]) and np.isnan(s[5]) and not q[4:6].any()
    for i in [0, 1, 2, 6, 19]:
        err = np.abs(x[i, :, None] - np.arange(-127, 128) * float(s[i]))
        assert np.array_equal(err.argmin(1) - 127, q[i])


def test_q8_rows_halves_go_to_the_even_code():
    x = np.array([[127, 0.5, 1.5, 2.5, -0.5, -1.5, -126.5, 126.5]]) * 2.0 ** -5
    q, s = o.q8_rows(x)
    assert s[0] == 2.0 ** -5 and q.tolist() == [[127, 0, 2, 2, 0, -2, -126, 126]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
def test_route_brute_force(score, best):
    r = np.random.default_rng(2)
    for _ in range(20):
        z = np.round(r.standard_normal((1, 8)), 1)
        b = np.round(r.standard_normal(8) * 0.2, 1)
        s = np.exp(z[0]) / np.exp(z[0]).sum() if score == "softmax" else 1 / (1 + np.exp(-z[0]))
        c = s + b
        val = {g: sorted(c[2 * g:2 * g + 2])[-1] if best == 1 else c[2 * g:2 * g + 2].sum() for g in range(4)}
        # the pair of groups, then the pair of experts in it, that no other pair beats
        groups = max(itertools.combinations(range(4), 2), key=lambda p: sum(sorted(val[g] for g in p)))
        best_groups = sorted(val, key=lambda g: -val[g])[:2]
        assert sum(val[g] for g in groups) == pytest.approx(sum(val[g] for g in best_groups))
        idx, w = o.route(z, b, 2, score, 4, 2, best, True, 2.0)
        inside = [e for e in range(8) if val[e // 2] >= val[best_groups[1]]]
        want = sorted(inside, key=lambda e: (-c[e], e))[:2]
        assert idx[0].tolist() == want
        np.testing.assert_allclose(w[0], 2 * s[want] / s[want].sum())


def test_route_masks():
    z = np.array([[-np.inf, 1.0, np.nan, 0.0], [-np.inf] * 4, [np.inf, 0, np.inf, 1]])
    idx, w = o.route(z, None, 3)
    assert idx.tolist() == [[1, 3, 0], [0, 1, 2], [0, 2, 3]]
    assert w[0, 2] == 0 and not w[1].any() and w[2].tolist() == [0.5, 0.5, 0]


def test_sample_by_hand():
    z = np.log(np.array([[0.1, 0.4, 0.2, 0.3]]))
    pick = lambda u, **kw: int(o.sample(z, [u], **kw)[0][0])  # noqa: E731
    assert [pick(u) for u in (0.0, 0.39, 0.41, 0.69, 0.71, 0.89, 0.91, 0.999)] == [1, 1, 3, 3, 2, 2, 0, 0]
    assert [pick(u, top_k=2) for u in (0.0, 0.57, 0.572, 0.999)] == [1, 1, 3, 3]
    assert [pick(u, top_p=0.65) for u in (0.57, 0.572, 0.999)] == [1, 3, 3]
    assert pick(0.999, top_p=0.39) == 1 and pick(0.999, top_p=0.0) == 1 and pick(0.999, min_p=1.0) == 1
    assert pick(0.999, min_p=0.45) == 2 and pick(0.999, temperature=0.0) == 1
    assert pick(0.999, top_k=3, top_p=0.75) == 3  # 0.7 / 0.9 reaches 0.75
    assert o.sample(np.full((1, 3), -np.inf), [0.5])[0][0] == -1


def test_sample_frequencies():
    r = np.random.default_rng(3)
    z = np.tile(r.standard_normal(50) * 2, (4000, 1))
    u = (np.arange(4000) + 0.5) / 4000
    tok, prob = o.sample(z, u, temperature=0.7)
    p = np.exp(z[0] / 0.7) / np.exp(z[0] / 0.7).sum()
    assert np.abs(np.bincount(tok, minlength=50) / 4000 - p).max() <= 1 / 4000
    np.testing.assert_allclose(prob, p[tok], rtol=1e-9)
