"""The operators between a prompt and its next token refuse what they cannot compute,
before any GPU work (the pointers below are never read)."""
import ctypes

import pytest
import torch

import expert_cache_host_amd as m
from expert_cache_host_amd import step
from expert_cache_host_amd.binding import RouteRule

P = 4096  # an aligned address; no refused call looks at it
EINVAL = -1


def refused(rc, msg):
    text = m.load_library().moe_last_error().decode()
    assert rc == EINVAL and msg in text, (rc, text)


@pytest.mark.parametrize("kw,msg", [
    (dict(t=3), "element type"), (dict(cols=0), "cols"), (dict(cols=131073, ldc=131200), "cols"), (dict(n=-1), "n_rows"),
    (dict(n=(1 << 24) + 1), "n_rows"), (dict(ldx=-1), "x_stride"), (dict(x=None), "NULL"), (dict(codes=None), "NULL"),
    (dict(scales=None), "NULL"), (dict(codes=P + 8), "16-byte"), (dict(ldc=112), "padded"), (dict(ldc=136), "multiple of 16"),
    (dict(x=P + 2), "aligned"), (dict(x=P + 1, t=1), "aligned"), (dict(scales=P + 2), "aligned"),
])
def test_q8_rows(kw, msg):
    a = dict(x=P, t=0, ldx=100, n=2, cols=100, codes=P, ldc=128, scales=P)
    a.update(kw)
    refused(step._library().moe_q8_rows(*a.values(), None), msg)


SIZES = [
    (dict(t=-1), "element type"), (dict(cols=0), "cols"), (dict(cols=131073, ldw=131088), "cols"), (dict(rows=0), "rows"),
    (dict(rows=(1 << 24) + 1, ldo=1 << 25), "rows"), (dict(T=-1), "n_tokens"), (dict(T=(1 << 20) + 1), "n_tokens"),
    (dict(T=1 << 20, rows=1 << 18, ldo=1 << 18), "2^22"), (dict(ldw=(1 << 22) + 16), "2^22"),
    (dict(ldo=39), "out_stride"), (dict(w=None), "NULL"), (dict(w=P + 8), "16-byte"), (dict(ldw=96), "multiple of 16"),
    (dict(ldw=120), "multiple of 16"), (dict(ws=None), "NULL"), (dict(out=None), "NULL"), (dict(ws=P + 2), "aligned"),
    (dict(out=P + 2), "aligned"),
]


@pytest.mark.parametrize("kw,msg", SIZES + [
    (dict(x=None), "NULL"), (dict(x=P + 4), "16-byte"), (dict(ldx=112), "padded"), (dict(xs=None), "NULL"),
    (dict(xs=P + 1), "aligned"),
])
def test_q8_matmul(kw, msg):
    a = dict(x=P, ldx=128, xs=P, T=2, w=P, ldw=112, ws=P, rows=40, cols=100, out=P, t=0, ldo=40)
    a.update(kw)
    refused(step._library().moe_q8_matmul(*a.values(), None), msg)


@pytest.mark.parametrize("kw,msg", SIZES + [
    (dict(xt=5), "element type"), (dict(x=None), "NULL"), (dict(x=P + 2), "aligned"), (dict(ldx=-1), "x_stride"),
    (dict(work=None), "workspace"), (dict(size=263), "workspace"), (dict(work=P + 8), "16-byte"),
])
def test_q8_linear(kw, msg):
    a = dict(x=P, xt=0, ldx=100, T=2, w=P, ldw=112, ws=P, rows=40, cols=100, out=P, t=0, ldo=40, work=P, size=1 << 20)
    a.update(kw)
    refused(step._library().moe_q8_linear(*a.values(), None), msg)


def test_q8_linear_workspace():
    ws = step._library().moe_q8_linear_workspace
    assert ws(0, 40, 100) >= 0 and ws(3, 40, 129) >= 3 * (256 + 4)
    for T, rows, cols in ((1, 1, 1), (7, 300, 128), (1 << 20, 64, 131072), (4000, 9000, 6145)):  # what the binding gives
        assert ws(T, rows, cols) == T * (-(-cols // 128) * 128 + 4)
    refused(ws(-1, 40, 100), "n_tokens")
    refused(ws(1, 0, 100), "rows")
    refused(ws(1, 1, 0), "cols")


RULES = [
    (dict(top_k=0), "top_k"), (dict(top_k=65), "top_k"), (dict(E=4, groups=1, keep=1, top_k=5), "top_k"),
    (dict(score=2), "score"), (dict(groups=0), "groups"), (dict(groups=5), "groups"), (dict(E=130, groups=65), "groups"),
    (dict(keep=0), "keep_groups"), (dict(keep=5), "keep_groups"), (dict(keep=1, top_k=17), "fewer"),
    (dict(best=0), "group_best"), (dict(best=3), "group_best"), (dict(groups=64, keep=9, best=2), "two experts"),
    (dict(renorm=2), "renorm"), (dict(scale=float("inf")), "scale"), (dict(scale=float("nan")), "scale"),
    (dict(E=513), "n_experts"), (dict(E=0), "n_experts"),
]


def rule(E=64, top_k=8, score=0, groups=4, keep=2, best=2, renorm=1, scale=1.0):
    return RouteRule(top_k, score, groups, keep, best, renorm, scale), E


@pytest.mark.parametrize("kw,msg", RULES)
def test_rule(kw, msg):
    r, E = rule(**kw)
    refused(step._library().moe_route(P, 0, E, P, 2, E, ctypes.byref(r), P, P, None), msg)


@pytest.mark.parametrize("kw,msg", [
    (dict(t=3), "element type"), (dict(rule=None), "rule"), (dict(T=-1), "n_tokens"), (dict(T=(1 << 24) + 1), "n_tokens"),
    (dict(ld=-1), "stride"), (dict(z=None), "NULL"), (dict(idx=None), "NULL"), (dict(w=None), "NULL"),
    (dict(z=P + 2), "aligned"), (dict(b=P + 2), "aligned"), (dict(idx=P + 1), "aligned"), (dict(w=P + 2), "aligned"),
])
def test_route(kw, msg):
    a = dict(z=P, t=0, ld=64, b=P, T=2, E=64, rule=ctypes.byref(rule()[0]), idx=P, w=P)
    a.update(kw)
    refused(step._library().moe_route(*a.values(), None), msg)


def test_forward_ruled():
    r, _ = rule()
    fn = m.load_library().moe_layer_forward_ruled
    refused(fn(None, 0, P, 1, P, None, ctypes.byref(r), None, P, None), "cache is NULL")


@pytest.mark.parametrize("kw,msg", [
    (dict(t=3), "element type"), (dict(T=-1), "n_rows"), (dict(T=65536), "n_rows"), (dict(V=0), "vocab"),
    (dict(V=(1 << 20) + 1), "vocab"), (dict(ld=-1), "stride"), (dict(z=None), "NULL"), (dict(u=None), "NULL"),
    (dict(tok=None), "NULL"), (dict(z=P + 2), "aligned"), (dict(u=P + 1), "aligned"), (dict(tok=P + 2), "aligned"),
    (dict(prob=P + 2), "aligned"), (dict(temp=-0.1), "temperature"), (dict(temp=float("inf")), "temperature"),
    (dict(temp=float("nan")), "temperature"), (dict(k=-1), "top_k"), (dict(p=1.1), "top_p"), (dict(p=-0.1), "top_p"),
    (dict(p=float("nan")), "top_p"), (dict(mp=-0.1), "min_p"), (dict(mp=1.5), "min_p"), (dict(mp=float("nan")), "min_p"),
    (dict(temps=P + 2), "aligned"), (dict(ks=P + 1), "aligned"), (dict(work=P + 8), "16-byte"),
])
def test_sample(kw, msg):
    a = dict(z=P, t=0, ld=64, T=2, V=64, u=P, temp=1.0, p=1.0, mp=0.0, k=0, temps=None, ps=None, mps=None, ks=None, tok=P,
             prob=P, work=P, size=1 << 30)
    a.update(kw)
    o = step._SampleOpts(*(a.pop(n) for n in ("temp", "p", "mp", "k", "temps", "ps", "mps", "ks")))
    head = [a.pop(n) for n in ("z", "t", "ld", "T", "V", "u")]
    refused(step._library().moe_sample(*head, ctypes.byref(o), *a.values(), None), msg)


def test_sample_opts_and_workspace():
    lib = step._library()
    refused(lib.moe_sample(P, 0, 64, 2, 64, P, None, P, P, None, 0, None), "opts")
    refused(lib.moe_sample_workspace(1, 0), "vocab")
    refused(lib.moe_sample_workspace(65536, 5), "n_rows")
    need = lib.moe_sample_workspace(2, 64)
    if need > 0:
        o = step._SampleOpts(1.0, 1.0, 0.0, 0, None, None, None, None)
        refused(lib.moe_sample(P, 0, 64, 2, 64, P, ctypes.byref(o), P, P, P, need - 1, None), "workspace")
        refused(lib.moe_sample(P, 0, 64, 2, 64, P, ctypes.byref(o), P, P, None, need, None), "workspace")


def test_tensors_must_be_on_the_gpu():
    t = torch.zeros(4, 64)
    for call in (lambda: m.q8_rows(t), lambda: m.Q8Matrix(t.to(torch.int8), t[:, 0]),
                 lambda: m.route_experts(t, m.RoutingRule(2)), lambda: m.sample_tokens(t, t[:, 0])):
        with pytest.raises(ValueError, match="GPU"):
            call()
    with pytest.raises(ValueError, match="score"):
        m.RoutingRule(2, score="tanh")
    for k in (0, -1, 65):
        with pytest.raises(ValueError, match="top_k"):
            m.RoutingRule(k)
    with pytest.raises(AttributeError):
        m.RoutingRule(2).top_k = 3


@pytest.mark.parametrize("kw", [dict(groups=2 ** 32 + 1), dict(keep_groups=2 ** 32 + 1), dict(group_best=2 ** 32 + 1),
                                dict(groups=-2 ** 32 + 1), dict(groups=8, keep_groups=2 ** 33 + 4), dict(group_best=2 ** 33)])
def test_rule_counts_that_pass_32_bits(kw):
    """Not taken for their low 32 bits, which would be a rule of their own."""
    with pytest.raises(ValueError, match=next(reversed(kw))):
        m.RoutingRule(2, **kw)
