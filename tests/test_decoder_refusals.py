"""The decoder-layer operators refuse what they cannot compute, before any GPU work
(the pointers below are never read)."""
import ctypes

import pytest

import expert_cache_host_amd as m
from expert_cache_host_amd import decoder
from expert_cache_host_amd.decoder import _KvBatch, _KvCache

P = 4096  # an aligned address; no refused call looks at it
EINVAL = -1


def _err():
    return m.load_library().moe_last_error().decode()


def norm(**kw):
    a = dict(h=P, ht=0, ldh=64, y=P, yt=0, ldy=64, post=P, gate=P, gt=0, ldg=0, pre=P, T=2, d=64, rs=1.0, bs=1.0,
             eps=1e-6, ho=P, ldho=64, x=P, xt=0, ldx=64)
    a.update(kw)
    return decoder._library().moe_block_norm(*a.values(), None)


@pytest.mark.parametrize("kw,msg", [
    (dict(T=-1), "n_tokens"), (dict(d=0), "d must"), (dict(d=32769), "d must"), (dict(ht=3), "element type"),
    (dict(yt=-1), "element type"), (dict(gt=7), "element type"), (dict(xt=3), "element type"),
    (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"), (dict(eps=float("inf")), "eps"),
    (dict(y=None), "need y"), (dict(y=None, gate=None), "need y"), (dict(pre=None), "together"),
    (dict(x=None), "together"), (dict(ho=None, x=None, pre=None), "nothing to write"),
    (dict(ldh=-1), "strides"), (dict(ldy=-64), "strides"), (dict(ldg=-1), "strides"),
    (dict(ldho=63), "strides"), (dict(ldx=63), "strides"), (dict(h=None), "h is NULL"), (dict(h=P + 2), "aligned"),
    (dict(y=P + 1, yt=1), "aligned"), (dict(post=P + 2), "aligned"), (dict(x=P + 1, xt=2), "aligned"),
])
def test_block_norm(kw, msg):
    assert norm(**kw) == EINVAL and msg in _err()


def matvec(**kw):
    a = dict(q=P, s=P, rows=16, cols=128, group=32, x=P, t=0, ldx=128, T=2, out=P, ldo=16)
    a.update(kw)
    return decoder._library().moe_q4_matvec(*a.values(), None)


@pytest.mark.parametrize("kw,msg", [
    (dict(t=3), "element type"), (dict(group=16), "group"), (dict(group=256), "group"), (dict(rows=0), "rows"),
    (dict(rows=(1 << 30) + 1, ldo=1 << 31), "rows"),
    (dict(cols=0), "cols"), (dict(cols=96, group=64), "cols"), (dict(cols=48), "cols"), (dict(T=-1), "n_tokens"),
    (dict(T=65537), "n_tokens"), (dict(ldx=-1), "x_stride"), (dict(ldo=15), "out_stride"), (dict(q=None), "NULL"),
    (dict(s=None), "NULL"), (dict(x=None), "NULL"), (dict(out=None), "NULL"), (dict(q=P + 8), "16-byte"),
    (dict(s=P + 1), "aligned"), (dict(x=P + 2), "aligned"), (dict(out=P + 1, t=1), "aligned"),
])
def test_q4_matvec(kw, msg):
    assert matvec(**kw) == EINVAL and msg in _err()


def cache(**kw):
    a = dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, n_pages=4, page_tokens=16, kv_heads=2, head_dim=64)
    a.update(kw)
    return _KvCache(*a.values())


def batch(**kw):
    a = dict(pages=P, start=P, past=P, n_seqs=1, max_pages=2, n_rows=2)
    a.update(kw)
    return _KvBatch(*a.values())


def append(c=None, b=None, **kw):
    a = dict(t=0, k=P, ldk=128, v=P, ldv=128, f=P, rot=64, il=0, q=P, ldq=256, heads=4, qo=P + 64, ldqo=256)
    a.update(kw)
    return decoder._library().moe_kv_append(c or cache(), b or batch(), *a.values(), None)


def attend(c=None, b=None, **kw):
    a = dict(t=0, q=P, ldq=256, heads=4, scale=0.125, window=0, out=P, ldo=256, ws=P, wsb=1 << 40)
    a.update(kw)
    return decoder._library().moe_kv_attend(c or cache(), b or batch(), *a.values(), None)


def read(c=None, b=None, k=P, v=P):
    return decoder._library().moe_kv_read(c or cache(), b or batch(), k, v, None)


def need(c=None, b=None, t=0, heads=4, window=0):
    return decoder._library().moe_kv_attend_workspace(c or cache(), b or batch(), t, heads, window)


CACHES = [(dict(k_codes=None), "NULL"), (dict(v_scales=None), "NULL"), (dict(n_pages=0), "n_pages"),
          (dict(page_tokens=8), "page_tokens"), (dict(page_tokens=24), "page_tokens"),
          (dict(page_tokens=65552), "page_tokens"), (dict(kv_heads=0), "kv_heads"), (dict(kv_heads=1025), "kv_heads"),
          (dict(head_dim=32), "head_dim"), (dict(head_dim=96), "head_dim"), (dict(head_dim=512), "head_dim"),
          (dict(v_codes=P + 8), "16-byte"), (dict(k_scales=P + 2), "16-byte")]
BATCHES = [(dict(pages=None), "NULL"), (dict(start=None), "NULL"), (dict(past=None), "NULL"), (dict(n_seqs=0), "n_seqs"),
           (dict(max_pages=0), "max_pages"), (dict(n_rows=-1), "n_rows"), (dict(past=P + 2), "aligned")]


@pytest.mark.parametrize("fn", [append, attend, read, need])
@pytest.mark.parametrize("kw,msg", CACHES)
def test_cache(fn, kw, msg):
    assert fn(c=cache(**kw)) == EINVAL and msg in _err()


@pytest.mark.parametrize("fn", [append, attend, read, need])
def test_too_many_rows(fn):
    assert fn(b=batch(n_rows=(1 << 23) + 1)) == EINVAL and "n_rows" in _err()


@pytest.mark.parametrize("fn", [attend, need])
@pytest.mark.parametrize("b,heads", [(dict(n_rows=1 << 23), 32), (dict(n_seqs=1 << 24), 4),
                                     (dict(n_rows=1 << 23, n_seqs=(1 << 24) - (1 << 21)), 4)])
def test_more_tiles_than_a_grid(fn, b, heads):
    assert fn(b=batch(**b), heads=heads, **(dict(ldo=heads * 64) if fn is attend else {})) == EINVAL
    assert "2^24" in _err()


@pytest.mark.parametrize("fn", [append, attend, read, need])
@pytest.mark.parametrize("kw,msg", BATCHES)
def test_batch(fn, kw, msg):
    assert fn(b=batch(**kw)) == EINVAL and msg in _err()


def test_null_structs():
    lib = decoder._library()
    for c, b in ((None, batch()), (cache(), None)):
        assert lib.moe_kv_read(c, b, P, P, None) == EINVAL and "NULL" in _err()


@pytest.mark.parametrize("kw,msg", [
    (dict(t=3), "element type"), (dict(rot=63), "rot_dim"), (dict(rot=66), "rot_dim"), (dict(rot=-2), "rot_dim"),
    (dict(f=None), "inv_freq"), (dict(f=P + 2), "inv_freq"), (dict(il=2), "interleaved"), (dict(q=None), "together"),
    (dict(qo=None), "together"), (dict(qo=P), "must not be q"), (dict(heads=0), "q_heads"), (dict(heads=3), "q_heads"),
    (dict(heads=1026), "q_heads"), (dict(ldq=-1), "strides"), (dict(ldqo=255), "q_out_stride"),
    (dict(ldk=-1), "strides"), (dict(ldv=-1), "strides"), (dict(k=None), "NULL"), (dict(v=None), "NULL"),
    (dict(k=P + 2), "aligned"), (dict(qo=P + 1, t=2), "aligned"),
])
def test_append(kw, msg):
    assert append(**kw) == EINVAL and msg in _err()


@pytest.mark.parametrize("kw,msg", [
    (dict(t=3), "element type"), (dict(heads=3), "q_heads"), (dict(scale=float("nan")), "scale"),
    (dict(scale=float("inf")), "scale"), (dict(window=-1), "window"), (dict(ldq=-1), "strides"),
    (dict(ldo=255), "out_stride"), (dict(q=None), "NULL"), (dict(out=None), "NULL"), (dict(q=P + 2), "aligned"),
    (dict(ws=P + 8), "16-byte"),
])
def test_attend(kw, msg):
    assert attend(**kw) == EINVAL and msg in _err()


@pytest.mark.parametrize("kw", [dict(t=3), dict(heads=5), dict(window=-1)])
def test_workspace(kw):
    assert need(**kw) == EINVAL


def test_read_pointers():
    assert read(k=None) == EINVAL and read(v=P + 2) == EINVAL


def test_no_tokens_is_no_work():
    b0 = batch(n_rows=0)
    assert norm(T=0, h=None) == 0 and matvec(T=0, x=None) == 0
    assert append(b=b0, k=None) == 0 and attend(b=b0, q=None) == 0 and read(b=b0, k=None) == 0


def test_binding_refuses_host_tensors():
    import torch
    z = torch.zeros
    with pytest.raises(ValueError, match="GPU"):
        m.block_norm(z(1, 64), pre_w=z(64))
    with pytest.raises(ValueError, match="GPU"):
        m.Q4Matrix(z(4, 2, 16, dtype=torch.uint8), z(4, 2, dtype=torch.float16))
    with pytest.raises(ValueError, match="GPU"):
        m.KVCache(z(1, 1, 16, 2, 16, dtype=torch.uint8), None, None, None)
    with pytest.raises(ValueError, match="head_dim"):
        m.KVCache.create(1, 16, 1, 96, device="cpu")


def test_from_blocks_sizes():
    import numpy as np
    with pytest.raises(ValueError, match="needed"):
        m.Q4Matrix.from_blocks(np.zeros(17, np.uint8), 1, 32, device="cpu")
    with pytest.raises(ValueError, match="multiple of group"):
        m.Q4Matrix.from_blocks(np.zeros(18, np.uint8), 1, 32, 64, device="cpu")


def test_struct_sizes_match_the_header():
    assert ctypes.sizeof(_KvCache) == 48 and ctypes.sizeof(_KvBatch) == 40
