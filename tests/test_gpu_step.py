"""The operators between a prompt and its next token against the binary64 oracle on the
GPU.  Codes, products of 8-bit rows, selected experts and tokens are equal bit for bit;
other tolerances are derived beside their checks."""
import numpy as np
import pytest
import torch

import expert_cache_host_amd as m
import synth
from expert_cache_host_amd.binding import MoeError
from layer_check import check_close
from oracle import step as o
from oracle.layer import expert_output
from oracle.routing import router_logits_fp32

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def strided(t, extra=3, shift=0):
    """The same rows in a wider buffer (row stride shape[1] + extra + shift, offset `shift` elements)."""
    buf = torch.full((t.shape[0], t.shape[1] + extra + shift), 7.5, device=t.device).to(t.dtype)
    buf[:, shift:shift + t.shape[1]] = t
    return buf[:, shift:shift + t.shape[1]]


# ------------------------------------------------------------------ 8-bit rows and products

def check_rows(x):
    q = m.q8_rows(x)
    codes, scales = o.q8_rows(f64(x))
    assert q.codes.shape == (x.shape[0], -(-x.shape[1] // 128) * 128)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.codes[:, :x.shape[1]].cpu().numpy(), codes)
    assert not q.codes[:, x.shape[1]:].any()
    return q


@pytest.mark.parametrize("cols", [1, 3, 64, 127, 128, 129, 1000, 2045, 6144, 8192, 8200, 20001, 131072])
@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
def test_q8_rows_sizes(cols, ty):
    g = gen(cols)
    n = 5 if cols < 20000 else 2
    x = rnd(g, n, cols, scale=3, dtype=TYPES[ty])
    check_rows(x)
    for extra, shift in ((4, 0), (3, 0), (4, 4), (2, 1)):
        check_rows(strided(x, extra, shift))


def test_q8_rows_values():
    g = gen(2)
    x = rnd(g, 14, 300)
    x[1] = 0
    x[2, 299] = float("inf")
    x[3, 7] = float("-inf")
    x[4, 8] = float("nan")
    x[5] *= 1e-44 / x[5].abs().max()          # subnormals: the scale too
    x[6] *= 1e-45 / x[6].abs().max()          # the scale is 0
    x[7] *= 3e38 / x[7].abs().max()
    x[8] = (torch.arange(300, device="cuda") - 150 + 0.5) * 2.0 ** -9  # halves of the scale 2^-9
    x[8, 0], x[8, 277:] = 127 * 2.0 ** -9, 0
    x[9] = torch.arange(300, device="cuda") / 299
    x[10] = -1.0
    x[11] *= 1e-37 / x[11].abs().max()        # a subnormal scale with digits left
    x[12, 1:] = 0
    x[13, 3] = -0.0
    check_rows(x)
    check_rows(x[:, :277])
    # values next to a border: every float32 neighbour of (n + 1/2) s
    s = torch.tensor(0.0123, device="cuda")
    b = (torch.arange(-127, 127, device="cuda") + 0.5) * s
    rows = torch.stack([torch.nextafter(b, torch.full_like(b, d)) if d else b for d in (-9.0, 0.0, 9.0)])
    rows = torch.cat([rows, (127 * s).expand(3, 1)], 1)
    check_rows(rows)


def test_q8_rows_many_and_none():
    g = gen(3)
    check_rows(rnd(g, 70000, 5))
    assert m.q8_rows(rnd(g, 0, 64)).codes.shape == (0, 128)


def check_product(x, w, codes, scales, **kw):
    """Bit for bit: the sum is exact, then two float32 products and one rounding to the type."""
    got = m.q8_matmul(x, w, **kw)
    q, s = o.q8_rows(f64(x))
    want = torch.from_numpy(o.q8_matmul(q, s, codes.cpu().numpy(), scales.cpu().numpy())).to(got.dtype)
    assert got.shape == want.shape
    assert torch.equal(torch.nan_to_num(got.cpu(), nan=123.0), torch.nan_to_num(want, nan=123.0))
    return got


def matrix(g, rows, cols):
    codes = torch.randint(-128, 128, (rows, cols), generator=g, device="cuda").to(torch.int8)
    return codes, 1e-3 * (1 + torch.rand(rows, generator=g, device="cuda"))


@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 17, 31, 33, 64, 65, 100, 128, 130, 257])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 16), (16, 64), (17, 100), (64, 128), (100, 129), (250, 640),
                                       (257, 1000), (513, 2045), (1030, 513)])
def test_q8_matmul_sizes(T, rows, cols):
    g = gen(T * 7 + rows)
    codes, scales = matrix(g, rows, cols)
    w = m.Q8Matrix(codes, scales)
    ty = ("f32", "bf16", "f16")[(T + rows) % 3]
    check_product(rnd(g, T, cols, dtype=TYPES[ty]), w, codes, scales)


@pytest.mark.parametrize("T,rows,cols", [(300, 1300, 4096), (1000, 520, 2100), (515, 5003, 384), (2100, 257, 130),
                                         (64, 20000, 260), (1, 40000, 512), (24, 4096, 6144), (700, 2816, 2816)])
@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
def test_q8_matmul_large(T, rows, cols, ty):
    g = gen(T + cols)
    codes, scales = matrix(g, rows, cols)
    check_product(rnd(g, T, cols, dtype=TYPES[ty]), m.Q8Matrix(codes, scales), codes, scales)


@pytest.mark.parametrize("T", [1, 3, 20, 70, 300])
def test_q8_matmul_strides_and_types(T):
    g = gen(T)
    rows, cols = 333, 777
    codes, scales = matrix(g, rows, cols)
    wide = torch.zeros(rows, 816, dtype=torch.int8, device="cuda")
    wide[:, :cols] = codes
    wide[:, cols:] = 77  # what stands behind a row has no effect
    for w in (m.Q8Matrix(codes, scales), m.Q8Matrix(wide[:, :cols], scales), m.Q8Matrix(strided(codes, 3, 2), scales)):
        for x, dt in ((rnd(g, T, cols), torch.bfloat16), (strided(rnd(g, T, cols, dtype=torch.float16), 5, 1), torch.float32)):
            check_product(x, w, codes, scales, dtype=dt)
        x = rnd(g, T, cols)
        buf = torch.full((T + 2, rows + 9), -5.0, device="cuda", dtype=torch.float16)
        check_product(x, w, codes, scales, out=buf[1:T + 1, 3:rows + 3])
        assert (buf[0] == -5).all() and (buf[-1] == -5).all() and (buf[:, :3] == -5).all() and (buf[:, rows + 3:] == -5).all()
        q = m.q8_rows(x)
        assert torch.equal(m.q8_matmul(q, w), m.q8_matmul(x, w))
        assert torch.equal(m.q8_matmul(q, w, dtype=torch.bfloat16), m.q8_matmul(x, w, dtype=torch.bfloat16))


@pytest.mark.parametrize("T", [1, 18, 130])
def test_q8_matmul_largest_sums(T):
    """131072 products of 127 and -128: within 32 bits."""
    x = torch.ones(T, 131072, device="cuda")
    x[T // 2] = -1
    codes = torch.full((20, 131072), -128, dtype=torch.int8, device="cuda")
    codes[7] = 127
    check_product(x, m.Q8Matrix(codes, torch.ones(20, device="cuda")), codes, torch.ones(20))


@pytest.mark.parametrize("T", [1, 4, 33, 300])
def test_q8_matmul_rows_that_are_not_finite(T):
    g = gen(5)
    codes, scales = matrix(g, 70, 200)
    w = m.Q8Matrix(codes, scales)
    x = rnd(g, T, 200)
    x[T // 2, 3] = float("nan")
    x[0, 199] = float("inf") if T > 1 else x[0, 199]
    got = check_product(x, w, codes, scales)
    assert torch.isnan(got[T // 2]).all()
    assert not torch.isnan(got).any(1).cpu().numpy()[[i for i in range(T) if i not in (0, T // 2)]].any()
    x = rnd(g, T, 200) * 1e30
    check_product(x, w, codes, scales, dtype=torch.float16)  # past the type's largest: infinities


@pytest.mark.parametrize("rows,cols,T", [(1, 131072, 300), (1, 5000, 1), (70, 131056, 33), (5000, 1, 700), (10240, 16, 16),
                                         (10239, 127, 32), (4097, 300, 17), (4096, 300, 32), (3, 40000, 4)])
def test_q8_matmul_thin(rows, cols, T):
    g = gen(rows + T)
    codes, scales = matrix(g, rows, cols)
    check_product(rnd(g, T, cols), m.Q8Matrix(codes, scales), codes, scales)


def test_q8_matmul_empty():
    g = gen(6)
    codes, scales = matrix(g, 70, 200)
    assert m.q8_matmul(rnd(g, 0, 200), m.Q8Matrix(codes, scales)).shape == (0, 70)
    assert m.q8_matmul(m.q8_rows(rnd(g, 0, 200)), m.Q8Matrix(codes, scales)).shape == (0, 70)


@pytest.mark.parametrize("ty", ["f32", "bf16"])
def test_q8_from_weights(ty):
    g = gen(8)
    for cols in (256, 300):
        w = rnd(g, 90, cols, dtype=TYPES[ty])
        q = m.Q8Matrix.from_weights(w)
        assert (q.rows, q.cols) == (90, cols)
        codes, scales = o.q8_rows(f64(w))
        check_product(rnd(g, 40, cols), q, torch.from_numpy(codes), torch.from_numpy(scales))


def test_q8_matrix_over_two_gigabytes():
    """Offsets past 32 bits in the matrix and in the output."""
    g = gen(9)
    rows, cols = 1 << 20, 2304
    codes = torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)
    scales = torch.full((rows,), 1e-3, device="cuda")
    w = m.Q8Matrix(codes, scales)
    pick = torch.tensor([0, 5, 931000, 931999, 1000003, rows - 1], device="cuda")
    for T in (1, 40, 2500):
        x = rnd(g, T, cols)
        out = m.q8_matmul(x, w, dtype=torch.bfloat16)
        at = [0, T // 2, T - 1]
        q, s = o.q8_rows(f64(x[at]))
        want = o.q8_matmul(q, s, codes[pick].cpu().numpy(), scales[pick].cpu().numpy())
        assert torch.equal(out[at][:, pick].cpu(), torch.from_numpy(want).bfloat16()), T


def test_q8_refusals():
    g = gen(10)
    codes, scales = matrix(g, 64, 128)
    w = m.Q8Matrix(codes, scales)
    x = rnd(g, 3, 128)
    for bad in (dict(x=rnd(g, 3, 127)), dict(x=x.double()), dict(x=x.cpu()), dict(x=rnd(g, 128, 3).t()), dict(x=x[0]),
                dict(out=torch.empty(3, 63, device="cuda")), dict(out=torch.empty(2, 64, device="cuda")),
                dict(out=torch.empty(3, 64, device="cuda").double()), dict(dtype=torch.int32),
                dict(out=torch.empty(3, 64, device="cuda"), dtype=torch.float16), dict(x=m.q8_rows(rnd(g, 3, 127)))):
        with pytest.raises(ValueError):
            m.q8_matmul(**{**dict(x=x, w=w), **bad})
    for args in ((codes.float(), scales), (codes[0], scales), (codes, scales[:3]), (codes, scales.double()),
                 (codes, scales.cpu()), (codes.t(), scales), (codes[:0], scales[:0])):
        with pytest.raises(ValueError):
            m.Q8Matrix(*args)
    q = m.q8_rows(x)
    for args in ((q.codes[:, :64], q.scales, 64), (q.codes, q.scales, 129), (q.codes, q.scales[:2], 128)):
        with pytest.raises(ValueError):
            m.Q8Rows(*args)


# ------------------------------------------------------------------ routing

def check_route(z, bias, **rule):
    got_i, got_w = m.route_experts(z, m.RoutingRule(rule["k"], rule.get("score", "softmax"), rule.get("groups", 1),
                                                    rule.get("keep"), rule.get("best", 1), rule.get("renorm", True),
                                                    rule.get("scale", 1.0)), bias)
    idx, w = o.route(f64(z), None if bias is None else bias.cpu().numpy(), **rule)
    np.testing.assert_array_equal(got_i.cpu().numpy(), idx)
    # scores in binary64 (errors near 2^-50), one rounding to float32
    assert np.all(np.abs(got_w.double().cpu().numpy() - w) <= (U + 2.0 ** -45) * np.abs(w) + 2.0 ** -149)
    return got_i, got_w


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (8, 2), (8, 8), (60, 4), (64, 8), (65, 6), (128, 8), (200, 16),
                                 (256, 8), (257, 3), (384, 12), (512, 10), (512, 64)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_sizes(E, k, score):
    g = gen(E)
    for T, ty, b, renorm in ((1, "f32", True, True), (5, "bf16", False, True), (67, "f16", True, False),
                             (130, "f32", False, False), (33, "bf16", True, True)):
        bias = rnd(g, E, scale=0.1) if b else None
        check_route(rnd(g, T, E, scale=2, dtype=TYPES[ty]), bias, k=k, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("E,groups,keep,k", [(8, 2, 1, 4), (16, 8, 3, 6), (64, 4, 2, 8), (96, 24, 5, 8), (128, 64, 9, 7),
                                             (256, 8, 4, 8), (320, 5, 4, 64), (512, 16, 1, 32), (512, 2, 1, 3),
                                             (510, 51, 7, 20), (64, 64, 9, 9)])
@pytest.mark.parametrize("best", [1, 2])
def test_route_groups(E, groups, keep, k, best):
    if best == 2 and E == groups:
        pytest.skip("a group of one expert has no second")
    g = gen(E + groups)
    for T, ty, score, b in ((1, "f32", "sigmoid", True), (40, "bf16", "sigmoid", False), (65, "f32", "softmax", True),
                            (9, "f16", "softmax", False)):
        bias = rnd(g, E, scale=0.2) if b else None
        check_route(rnd(g, T, E, scale=1.5, dtype=TYPES[ty]), bias, k=k, score=score, groups=groups, keep=keep, best=best)


@pytest.mark.parametrize("size", [50.0, 1e4, 1e30])
def test_route_groups_whose_pairs_cancel(size):
    """A group's two best of opposite signs: their sum is far smaller than what float32 rounds off either."""
    g = gen(5)
    E, groups = 64, 8
    bias = torch.full((E,), -size, device="cuda")
    bias[::E // groups] = size
    z = 1e-5 * rnd(g, 200, E)
    for score in ("sigmoid", "softmax"):
        check_route(z, bias, k=4, score=score, groups=groups, keep=3, best=2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_whose_pairs_pass_float32(score):
    """A bias near the lowest float32, a mask that many use: pairs sum to less than float32 holds, yet their groups come
    before one with a single expert left."""
    inf, low = float("inf"), -3.4028234e38
    t = lambda v: torch.tensor(v, device="cuda")  # noqa: E731
    for b in ([0.0, 0.0, -3.4e38, -3.4e38], [0.0, 0.0, low, low], [0.0, 0.0, -1.8e38, -1.8e38]):
        idx, _ = check_route(t([[0.0, -inf, 0.0, 0.0]]), t(b), k=1, score=score, groups=2, keep=1, best=2)
        assert idx.tolist() == [[2]]
    # groups of such pairs among themselves, beside ordinary and excluded ones
    g = gen(12)
    for k, groups, keep in ((2, 8, 3), (9, 16, 5)):
        z = rnd(g, 60, 64)
        z[torch.rand(60, 64, generator=g, device="cuda") < 0.3] = -inf
        bias = rnd(g, 64, scale=0.2)
        bias[8:40] = low
        bias[16:24] = -1.75e38
        bias[40:48] = -inf
        bias[50] = inf
        check_route(z, bias, k=k, score=score, groups=groups, keep=keep, best=2)
        check_route(z, bias, k=k, score=score, groups=groups, keep=keep, best=1)
        check_route(z, -bias, k=k, score=score, groups=groups, keep=keep, best=2)


@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_ties_and_close_values(groups, keep, score):
    """Equal values go to the lower ids; values that differ by less than float32 can tell are told apart."""
    g = gen(4)
    E, k = 64, 10
    z = torch.round(rnd(g, 50, E) * 2) / 2
    check_route(z, None, k=k, score=score, groups=groups, keep=keep, best=2)
    check_route(z, torch.round(rnd(g, E) * 4) / 8, k=k, score=score, groups=groups, keep=keep, best=2)
    check_route(torch.zeros(3, E, device="cuda"), torch.zeros(E, device="cuda"), k=k, score=score, groups=groups, keep=keep)
    # scores one float32 step apart under a large bias, which float32 sums cannot hold
    z = 1 + torch.randint(0, 40, (50, E), generator=g, device="cuda") * 2.0 ** -23
    check_route(z, torch.full((E,), 100.0, device="cuda"), k=k, score=score, groups=groups, keep=keep, best=2)
    check_route(-z * 20, torch.full((E,), 1.0, device="cuda"), k=k, score=score, groups=groups, keep=keep, best=1)
    # more equal values than a wave has lanes
    b = torch.zeros(512, device="cuda")
    b[7] = 1
    check_route(torch.ones(3, 512, device="cuda"), b, k=k, score=score, groups=groups, keep=keep, best=2)
    check_route(torch.round(rnd(g, 20, 512) / 2), b, k=63, score=score, groups=groups, keep=keep, best=2)
    check_route(torch.round(rnd(g, 20, 512) / 2), None, k=64, score=score, groups=groups, keep=keep)
    # +0 and -0 are equal
    z = torch.zeros(2, E, device="cuda")
    z[:, ::2] = -0.0
    check_route(z, None, k=k, score=score, groups=groups, keep=keep)


@pytest.mark.parametrize("groups,keep,best", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_masked(groups, keep, best, score, with_bias):
    g = gen(6)
    E, k = 96, 12
    inf = float("inf")
    z = rnd(g, 12, E, scale=2)
    z[0] = -inf
    z[1, 5:] = -inf
    z[2, :60] = float("nan")
    z[3, 7] = z[3, 50] = inf
    z[4] = inf
    z[5, 3:] = -3.4028234e38
    z[6] = float("nan")
    z[7, ::2] = -inf
    z[8, torch.arange(E, device="cuda") % 12 != 4] = -inf  # one expert a group
    z[9] = -1e30
    z[10] *= 500  # scores that underflow
    bias = None
    if with_bias:
        bias = rnd(g, E, scale=0.3)
        bias[11], bias[30], bias[31], bias[70] = -inf, float("nan"), -inf, 1e30
    for renorm in (True, False):
        i, w = check_route(z, bias, k=k, score=score, groups=groups, keep=keep, best=best, renorm=renorm)
        assert torch.isfinite(w).all() and (w[0] == 0).all() and (w[6] == 0).all()
        assert all(len(set(r)) == k for r in i.cpu().tolist())


def test_route_infinite_bias():
    g = gen(7)
    b = rnd(g, 32, scale=0.1)
    b[9] = b[20] = float("inf")
    for best in (1, 2):
        check_route(rnd(g, 9, 32), b, k=5, score="sigmoid", groups=4, keep=2, best=best)


def test_route_strides_many_and_none():
    g = gen(8)
    z = rnd(g, 301, 130)
    for extra, shift in ((3, 0), (4, 4), (2, 1)):
        check_route(strided(z, extra, shift), None, k=6)
    zh = rnd(g, 70001, 16, dtype=torch.bfloat16)
    check_route(zh, rnd(g, 16), k=2, score="sigmoid")
    i, w = m.route_experts(rnd(g, 0, 64), m.RoutingRule(4))
    assert i.shape == w.shape == (0, 4)
    row = z[:1].expand(5, 130)  # one row for all (stride 0)
    check_route(row, None, k=6)


def test_route_refusals():
    g = gen(9)
    z, r = rnd(g, 3, 64), m.RoutingRule(4)
    for bad in (dict(logits=z.double()), dict(logits=z.t()), dict(logits=z[0]), dict(bias=rnd(g, 63)),
                dict(bias=rnd(g, 64).half()), dict(bias=rnd(g, 64).cpu())):
        with pytest.raises(ValueError):
            m.route_experts(**{**dict(logits=z, rule=r), **bad})
    with pytest.raises(MoeError):
        m.route_experts(rnd(g, 3, 513), r)
    with pytest.raises(MoeError):
        m.route_experts(z, m.RoutingRule(4, groups=3, keep_groups=1))


# ------------------------------------------------------------------ the MoE layer with a rule

@pytest.mark.parametrize("mode", ["stream", "host"])
@pytest.mark.parametrize("T", [1, 2, 4, 5, 17])
def test_layer_with_a_rule(mode, T):
    """The MoE layer's output with the rule's experts and weights, and its slots' log, which is that of the same experts
    through the planner."""
    wl = synth.WORKLOADS["tiny"]
    buf = synth.gen_experts(wl, 0)
    c = m.MoECache(1, wl.n_experts, 4, wl.d_model, wl.d_ff, buf, top_k=wl.top_k, miss_mode=mode)
    plan = m.Planner(wl.n_experts, 4, mode)
    w_r, b = synth.gen_router(wl, 0)
    g = gen(T)
    for call in range(6):
        rule = dict(k=wl.top_k, score=("sigmoid", "softmax")[call % 2], groups=4, keep=2, best=1 + call // 2 % 2,
                    renorm=call != 3, scale=1.5)
        r = m.RoutingRule(rule["k"], rule["score"], 4, 2, rule["best"], rule["renorm"], 1.5)
        sb = rnd(g, wl.n_experts, scale=0.3) if call != 1 else None
        x = rnd(g, T, wl.d_model)
        if call == 4:  # the plain path between them, on the same cache
            c.forward(0, x, torch.from_numpy(w_r).cuda())
            plan.plan(c.routing(0)[0].ravel().tolist(), T)
            continue
        out = c.forward(0, x, torch.from_numpy(w_r).cuda(), None if b is None else torch.from_numpy(b).cuda(), rule=r,
                        select_bias=sb)
        torch.cuda.synchronize()
        z = router_logits_fp32(x.cpu().numpy(), w_r, b)
        idx, w = o.route(z, None if sb is None else sb.cpu().numpy(), **rule)
        got_i, got_w = c.routing(0)
        np.testing.assert_array_equal(got_i, idx)
        assert np.all(np.abs(got_w - w) <= 1.001 * U * np.abs(w))
        plan.plan(idx.ravel().tolist(), T)
        want = np.zeros((T, wl.d_model))
        for e in np.unique(idx):
            tok, j = np.nonzero(idx == e)
            want[tok] += w[tok, j][:, None] * expert_output(buf, int(e), wl.d_model, wl.d_ff, f64(x)[tok])
        check_close(out.cpu().numpy(), want)
    assert c.evictions(0) == plan.evictions()
    c.close()


@pytest.mark.parametrize("T", [1, 6])
def test_layer_with_a_rule_timed_and_on_another_stream(T):
    """Timing, partial results and logits as without a rule; calls on changing streams."""
    wl = synth.WORKLOADS["tiny"]
    c = m.MoECache(1, wl.n_experts, 4, wl.d_model, wl.d_ff, synth.gen_experts(wl, 0), top_k=wl.top_k, miss_mode="host",
                   keep_debug=True)
    c.set_timing(True)
    g = gen(T)
    w_r = rnd(g, wl.n_experts, wl.d_model, scale=0.1)
    r = m.RoutingRule(wl.top_k, "sigmoid", scale=2.0)
    streams = [torch.cuda.current_stream(), torch.cuda.Stream()]
    x = rnd(g, T, wl.d_model)
    torch.cuda.synchronize()
    outs = []
    for call in range(4):
        with torch.cuda.stream(streams[call % 2]):
            outs.append(c.forward(0, x, w_r, rule=r))
        torch.cuda.synchronize()
        gpu, host = c.partials(0)
        np.testing.assert_array_equal(gpu + host, outs[-1].cpu().numpy())
        z = router_logits_fp32(x.cpu().numpy(), w_r.cpu().numpy(), None)
        idx, w = o.route(z, None, wl.top_k, "sigmoid", scale=2.0)
        np.testing.assert_array_equal(c.routing(0)[0], idx)
    assert c.kernel_stats()["router"][0] == 4
    check_close(outs[3].cpu().numpy(), f64(outs[0]))
    c.close()


@pytest.mark.parametrize("T", [1, 3, 6])
@pytest.mark.parametrize("with_bias", [False, True])
def test_layer_with_a_rule_kernel_stats(T, with_bias):
    """The rule's kernel counts as the top-k, with the bytes it moves; the buckets of decode calls as the remap."""
    wl = synth.WORKLOADS["tiny"]
    E, k = wl.n_experts, wl.top_k
    c = m.MoECache(1, E, E, wl.d_model, wl.d_ff, synth.gen_experts(wl, 0), top_k=k)
    g = gen(T)
    x, w_r = rnd(g, T, wl.d_model), rnd(g, E, wl.d_model, scale=0.1)
    bias = rnd(g, E, scale=0.1) if with_bias else None
    r = m.RoutingRule(k, "sigmoid")
    c.forward(0, x, w_r, rule=r, select_bias=bias)
    c.sync()
    for plain in (False, True):
        c.set_timing(True)
        c.reset_stats()
        for _ in range(5):
            if plain:
                c.forward(0, x, w_r)
            else:
                c.forward(0, x, w_r, rule=r, select_bias=bias)
        c.sync()
        ks = c.kernel_stats()
        n, sec, by = ks["topk"]
        # logits, then ids and weights twice: on the device and in page-locked memory
        assert (n, by) == (5, 5 * 4 * (T * E + 4 * T * k + (E if with_bias and not plain else 0))) and sec > 0
        n, sec, by = ks["remap"]
        if T <= 4:  # the plain path's top-k lists the buckets itself
            assert (n, by) == ((0, 0) if plain else (5, 5 * 8 * T * k)) and (sec > 0) == (not plain)
        else:
            assert n >= 5 and by == n * 8 * T * k and sec > 0
        c.set_timing(False)
    # a rule alone, which times nothing, between timed calls
    c.set_timing(True)
    c.reset_stats()
    m.route_experts(x @ w_r.t(), r, bias)
    c.forward(0, x, w_r, rule=r)
    c.sync()
    assert c.kernel_stats()["topk"][0] == 1
    c.close()


def test_layer_rule_refusals():
    wl = synth.WORKLOADS["tiny"]
    c = m.MoECache(1, wl.n_experts, 4, wl.d_model, wl.d_ff, synth.gen_experts(wl, 0), top_k=wl.top_k)
    g = gen(1)
    x, w = rnd(g, 1, wl.d_model), rnd(g, wl.n_experts, wl.d_model)
    with pytest.raises(MoeError, match="top_k"):
        c.forward(0, x, w, rule=m.RoutingRule(wl.top_k + 1))
    with pytest.raises(MoeError, match="divide"):
        c.forward(0, x, w, rule=m.RoutingRule(wl.top_k, groups=3))
    with pytest.raises(ValueError):
        c.forward(0, x, w, select_bias=w[:, 0].contiguous())
    with pytest.raises(ValueError):
        c.forward(0, x, w, rule=m.RoutingRule(wl.top_k), select_bias=rnd(g, wl.n_experts + 1))
    with pytest.raises(ValueError):
        c.forward(0, x, w, rule=m.RoutingRule(wl.top_k), out=torch.empty_like(x), noalloc=True)
    c.close()


# ------------------------------------------------------------------ sampling

def cpu(v):
    return f64(v) if torch.is_tensor(v) else v


def check_sample(z, u, **kw):
    tok, prob = m.sample_tokens(z, u, **kw)
    want, p = o.sample(f64(z), f64(u), **{n: cpu(v) for n, v in kw.items()})
    np.testing.assert_array_equal(tok.cpu().numpy(), want)
    # the weight and the sum in binary64, the quotient rounded to float32
    assert np.all(np.abs(f64(prob) - p) <= (U + 2.0 ** -40) * p + 2.0 ** -149)
    return tok, prob


@pytest.mark.parametrize("V", [1, 2, 63, 64, 65, 1000, 4096, 5003, 32000, 65003, 131072, 262144])
@pytest.mark.parametrize("ty", ["f32", "bf16", "f16"])
def test_sample_sizes(V, ty):
    g = gen(V)
    T = 6 if V < 60000 else 3
    z = (2 * rnd(g, T, V) + 9 * torch.rand((T, V), generator=g, device="cuda") ** 12).to(TYPES[ty])
    u = torch.rand(T, generator=g, device="cuda")
    for kw in (dict(), dict(temperature=0.0), dict(temperature=0.7, top_k=50, top_p=0.9), dict(top_p=0.6),
               dict(min_p=0.05), dict(temperature=1.3, top_k=1000, top_p=0.97, min_p=0.01), dict(top_k=1),
               dict(temperature=2.5, top_k=V // 2 + 1)):
        check_sample(z, u, **kw)


@pytest.mark.parametrize("V", [16383, 16384, 16385, 20001])
def test_sample_around_the_short_rows(V):
    """Rows that one workgroup takes and rows that several launches take; many rows of one segment each."""
    g = gen(V)
    for T in (2, 600 if V > 16384 else 40):
        z, u = rnd(g, T, V, scale=2.5), torch.rand(T, generator=g, device="cuda")
        check_sample(z, u, temperature=0.9, top_k=77, top_p=0.9, min_p=0.01)


@pytest.mark.parametrize("V", [9000, 40000])
@pytest.mark.parametrize("n", [255, 256, 257, 2047, 2048, 2049, 2500])
def test_sample_around_the_sorted_tokens(V, n):
    """n equal tokens ahead of the others: as many as are sorted by counting, in LDS, or not at all."""
    g = gen(n)
    T = 9
    z = rnd(g, T, V) - 20
    for t in range(T):
        z[t, torch.randperm(V, generator=g, device="cuda")[:n]] = 1.5
    u = torch.linspace(0, 0.9999999, T, device="cuda")
    for kw in (dict(), dict(top_k=n - 1), dict(top_k=n + 1), dict(top_p=0.5), dict(min_p=0.9, top_k=n // 2)):
        check_sample(z, u, **kw)


def test_sample_settings_per_row():
    g = gen(3)
    T, V = 37, 3001
    z = rnd(g, T, V, scale=2)
    u = torch.rand(T, generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    t = torch.where(i % 4 == 1, 0.0, 0.5 + 0.05 * i)
    t[9], t[13] = float("nan"), -1.0
    k = torch.where(i % 3 == 0, 0, i * 7).to(torch.int32)
    k[20], k[21] = -5, 2 ** 31 - 1
    p = torch.where(i % 5 == 2, 1.0, 0.3 + 0.02 * i).clamp(max=0.999)
    p[4], p[5], p[6], p[7] = 1.5, -0.5, 0.0, float("nan")
    mp = 0.01 * (i % 7).float()
    mp[10], mp[11], mp[12] = 2.0, -1.0, float("nan")
    check_sample(z, u, temperature=t, top_k=k, top_p=p, min_p=mp)
    check_sample(z, u, temperature=0.8, top_k=k)
    check_sample(z, u, top_p=p, min_p=0.02)


@pytest.mark.parametrize("V", [7, 2000, 70000])
def test_sample_random_numbers_cover_the_tokens(V):
    """A grid of random numbers, the smallest and the largest among them, and numbers outside of the range."""
    g = gen(V)
    T = 200
    z = rnd(g, 1, V, scale=1.5).expand(T, V)
    u = torch.linspace(0, 1, T, device="cuda")
    u[0], u[-1], u[-2], u[-3], u[-4] = 0.0, 1.0 - 2.0 ** -24, 1.0, float("nan"), -0.5
    check_sample(z, u, temperature=0.9)
    check_sample(z, u, temperature=0.9, top_k=5, top_p=0.99)
    check_sample(z, u, min_p=0.2)


@pytest.mark.parametrize("V", [64, 5000, 66000])
def test_sample_ties(V):
    """Equal logits stand in the order of their ids: all equal, few values, and a tie that a filter's border cuts."""
    g = gen(V)
    T = 24
    u = torch.rand(T, generator=g, device="cuda")
    check_sample(torch.full((T, V), -3.25, device="cuda"), u)
    check_sample(torch.full((T, V), 2.0, device="cuda"), u, top_k=V // 3 + 1, top_p=0.7)
    z = torch.randint(-2, 3, (T, V), generator=g, device="cuda").float() * 0.5
    for kw in (dict(), dict(top_k=V // 10 + 1), dict(top_p=0.37), dict(top_k=V // 2, top_p=0.5, min_p=0.3)):
        check_sample(z.half(), u, **kw)
    z = torch.zeros(T, V, device="cuda")
    z[:, ::2] = -0.0
    check_sample(z, u, top_p=0.5)


def test_sample_flat_and_steep():
    """Nearly flat rows (every token within a small part of a temperature) and rows with one token far ahead."""
    g = gen(11)
    T, V = 8, 50000
    u = torch.rand(T, generator=g, device="cuda")
    z = rnd(g, T, V)
    for s in (1e-6, 1e-3, 0.05, 40.0, 1e4, 1e30):
        check_sample(z * s, u)
        check_sample(z * s, u, top_k=300, top_p=0.9)
        check_sample(z * s, u, top_p=0.9, min_p=0.5)
    check_sample(z, u, temperature=1e-3)
    check_sample(z, u, temperature=1e-30)
    check_sample(z, u, temperature=1e30, top_p=0.9)
    check_sample(z + 1e6, u, temperature=1e-2, top_k=9)


@pytest.mark.parametrize("V", [700, 20000])
def test_sample_temperatures_at_the_ends(V):
    """Temperatures whose inverse passes binary64, infinite ones, and those at the ends of float32."""
    g = gen(19)
    T = 6
    u = torch.rand(T, generator=g, device="cuda")
    z = rnd(g, T, V)
    z[2, :5] = z[2].max() + 1  # equal largest tokens
    for t in (5e-324, 1e-310, 1e-306, 1e300):
        for kw in (dict(), dict(top_k=3), dict(top_p=0.7), dict(min_p=0.4)):
            check_sample(z, u, temperature=t, **kw)
    t = torch.full_like(u, float("inf"))
    t[::3] = 1e-45
    t[1::3] = 3.4e38
    check_sample(z, u, temperature=t)
    check_sample(z, u, temperature=t, top_k=50, top_p=0.6, min_p=0.2)


def test_sample_masked():
    g = gen(12)
    inf = float("inf")
    T, V = 12, 3000
    z = rnd(g, T, V, scale=2)
    z[0] = -inf
    z[1] = float("nan")
    z[2, 1:] = -inf
    z[3, :2990] = -inf
    z[4, ::3] = float("nan")
    z[5, 17] = inf
    z[6, 10:20] = inf
    z[7] = inf
    z[8] = -3.4028234e38
    z[9, 5:] = -3.4028234e38
    z[10, 4] = 3.4028234e38
    u = torch.rand(T, generator=g, device="cuda")
    for kw in (dict(), dict(top_k=20), dict(top_p=0.5), dict(min_p=0.1), dict(temperature=0.0), dict(temperature=3.0, top_k=2500)):
        tok, prob = check_sample(z, u, **kw)
        assert tok[:2].tolist() == [-1, -1] and prob[:2].tolist() == [0, 0] and tok[2] == 0
        tok, _ = check_sample(z.to(torch.bfloat16), u, **kw)
        assert tok[1] == -1


def test_sample_strides_rows_and_none():
    g = gen(13)
    z = rnd(g, 33, 2050, scale=2)
    u = torch.rand(33, generator=g, device="cuda")
    for extra, shift in ((3, 0), (4, 4), (2, 1)):
        check_sample(strided(z, extra, shift), u, top_p=0.9)
        check_sample(strided(z.half(), extra, shift), u, top_k=40)
    zb, ub = rnd(g, 1500, 129), torch.rand(1500, generator=g, device="cuda")
    check_sample(zb, ub, top_p=0.8)
    tok, prob = m.sample_tokens(rnd(g, 0, 50), u[:0])
    assert tok.shape == prob.shape == (0,)
    zz = rnd(g, 2, 1 << 20, scale=3)
    for kw in (dict(), dict(top_k=100000, top_p=0.95)):
        check_sample(zz, u[:2], **kw)


def test_sample_refusals():
    g = gen(14)
    z, u = rnd(g, 3, 64), torch.rand(3, device="cuda")
    for bad in (dict(logits=z.double()), dict(logits=z.t()), dict(logits=z[0]), dict(u=u[:2]), dict(u=u.double()),
                dict(u=u.cpu()), dict(temperature=u[:2]), dict(temperature=u.double()), dict(top_k=u),
                dict(top_k=-1), dict(top_k=torch.ones(3, dtype=torch.int64, device="cuda")), dict(top_p=u.half()),
                dict(min_p=u.cpu())):
        with pytest.raises(ValueError):
            m.sample_tokens(**{**dict(logits=z, u=u), **bad})
    for bad in (dict(temperature=-1.0), dict(temperature=float("nan")), dict(top_p=1.5), dict(min_p=-0.1)):
        with pytest.raises(MoeError):
            m.sample_tokens(z, u, **bad)


# ------------------------------------------------------------------ together

class Head:
    """The end of a step: a prompt's projection, the vocabulary's product, and the next tokens."""

    def __init__(self, seed, T=6, d=512, V=3000):
        g = self.g = gen(seed)
        self.proj, self.vocab = (m.Q8Matrix(*matrix(g, r, d)) for r in (d, V))
        self.norm = 1 + 0.1 * rnd(g, d)
        self.rule = m.RoutingRule(4, "sigmoid", 4, 2, 2, True, 2.5)
        self.router, self.bias = m.Q8Matrix(*matrix(g, 32, d)), rnd(g, 32, scale=0.1)
        self.T, self.d = T, d

    def __call__(self, h, u):
        h, x = m.block_norm(h, m.q8_matmul(h, self.proj), pre_w=self.norm, block_scale=0.01)
        xq = m.q8_rows(x)
        idx, w = m.route_experts(m.q8_matmul(xq, self.router), self.rule, self.bias)
        tok, prob = m.sample_tokens(m.q8_matmul(xq, self.vocab) * 0.1, u, temperature=0.8, top_k=40, top_p=0.9)
        return h, idx, w, tok, prob


def test_steps_captured_and_replayed():
    """A step in a graph, replayed with eager steps of the same operators between the replays."""
    head = Head(21)
    h, u = rnd(head.g, 6, 512), torch.rand(6, generator=head.g, device="cuda")
    head(h, u)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = head(h, u)
    for step in range(8):
        h.copy_(rnd(head.g, 6, 512))
        u.copy_(torch.rand(6, generator=head.g, device="cuda"))
        graph.replay()
        want = head(h, u)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), step
        x = f64(want[0]) / np.sqrt((f64(want[0]) ** 2).mean(1, keepdims=True))
        assert np.isfinite(x).all()
        check_route(rnd(head.g, 3, 32), head.bias, k=4)  # eager work of another size between the replays


def test_two_graphs_and_streams_at_once():
    head = Head(22)
    streams = [torch.cuda.Stream() for _ in range(2)]
    inputs = [(rnd(head.g, 6, 512), torch.rand(6, generator=head.g, device="cuda")) for _ in range(2)]
    want = [tuple(t.clone() for t in head(*i)) for i in inputs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in inputs:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(head(*i))
        graphs.append(gr)
    for _ in range(5):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for got, ref in zip(outs, want) for a, b in zip(got, ref))
        for t in outs[0] + outs[1]:
            t.zero_()
        torch.cuda.synchronize()
    for _ in range(3):
        got = []
        for i, s in zip(inputs, streams):
            with torch.cuda.stream(s):
                got.append(head(*i))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for r, ref in zip(got, want) for a, b in zip(r, ref))


def test_calls_on_a_given_stream():
    """Inputs dropped right after a call on another stream keep their memory until it has run."""
    g = gen(23)
    s = torch.cuda.Stream()
    codes, scales = matrix(g, 700, 1024)
    w = m.Q8Matrix(codes, scales)
    keep = rnd(g, 300, 1024)
    u = torch.rand(300, generator=g, device="cuda")
    bias = rnd(g, 700)[:512].contiguous()
    rule = m.RoutingRule(8, "sigmoid")
    want = m.q8_matmul(keep, w), *m.route_experts(keep[:, :512], rule, bias), *m.sample_tokens(keep, u, top_p=0.9)
    for _ in range(5):
        x = keep.clone()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            for _ in range(20):
                torch.mm(keep.t(), keep)
        got = m.q8_matmul(x, w, stream=s), *m.route_experts(x[:, :512], rule, bias, stream=s), \
            *m.sample_tokens(x, u, top_p=0.9, stream=s)
        del x
        junk = torch.full((300, 1024), 1e9, device="cuda")
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        del junk


def test_layer_from_prompt_to_token():
    """A projection in 8 bits, the MoE layer by a rule, norms, the vocabulary in 4 bits and the next token, next to the
    same steps in plain torch: the routing decides equally, outputs agree to the layer's tolerance."""
    wl = synth.WORKLOADS["tiny"]
    d, T, V = wl.d_model, 5, 512
    g = gen(31)
    buf = synth.gen_experts(wl, 0)
    c = m.MoECache(1, wl.n_experts, 4, d, wl.d_ff, buf, top_k=wl.top_k)
    wq = m.Q8Matrix.from_weights(rnd(g, d, d, scale=d ** -0.5))
    router, bias = rnd(g, wl.n_experts, d, scale=0.1), rnd(g, wl.n_experts, scale=0.1)
    rule = m.RoutingRule(wl.top_k, "sigmoid", scale=1.5)
    vocab = m.Q4Matrix(torch.randint(0, 256, (V, d // 32, 16), generator=g, device="cuda", dtype=torch.uint8),
                       torch.full((V, d // 32), 0.01, device="cuda", dtype=torch.float16))
    nw = torch.ones(d, device="cuda")
    for step in range(3):
        h, u = rnd(g, T, d), torch.rand(T, generator=g, device="cuda")
        y = m.q8_matmul(h, wq)
        h1, x = m.block_norm(h, y, pre_w=nw)
        moe = c.forward(0, x, router, rule=rule, select_bias=bias)
        _, x2 = m.block_norm(h1, moe, pre_w=nw)
        logits = m.q4_matvec(x2, vocab)
        tok, prob = m.sample_tokens(logits, u, temperature=0.7, top_k=50, top_p=0.95)
        torch.cuda.synchronize()
        q, s = o.q8_rows(f64(h))
        assert torch.equal(y.cpu(), torch.from_numpy(o.q8_matmul(q, s, wq.codes[:, :d].cpu().numpy(), wq.scales.cpu().numpy())))
        idx, wt = o.route(router_logits_fp32(x.cpu().numpy(), router.cpu().numpy(), None), bias.cpu().numpy(), wl.top_k,
                          "sigmoid", scale=1.5)
        np.testing.assert_array_equal(c.routing(0)[0], idx)
        want = np.zeros((T, d))
        for e in np.unique(idx):
            t, j = np.nonzero(idx == e)
            want[t] += wt[t, j][:, None] * expert_output(buf, int(e), d, wl.d_ff, f64(x)[t])
        check_close(moe.cpu().numpy(), want)
        want_tok, _ = o.sample(f64(logits), f64(u), 0.7, 50, 0.95)
        assert tok.tolist() == want_tok.tolist()
    c.close()
