"""Refusals of the norm append, shared prefixes, weighed attention and eviction, on the host before any
launch (no GPU needed): the pointers here are never dereferenced."""
import ctypes as C

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build

FAKE, ODD = 1 << 20, (1 << 20) + 4


@pytest.fixture(scope="module")
def L():
    build()
    return B.lib()


def params(**over):
    kw = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, n_tokens=1000, block_size=32, num_pages=100,
              window_tokens=0, topk=4, num_queries=5, capacity_tokens=1005)
    kw.update(over)
    return B.make_params(**kw)


def append(L, p=None, rows=10, cu=None, lens=FAKE, pos=FAKE, axes=3, axis=FAKE, rotary=128, pairing=1, freq=FAKE, qw=FAKE,
           qws=0, kw=FAKE, kws=128, eps=1e-6, q=FAKE, qs=1024, k=FAKE, ks=256, v=FAKE, vs=256, qo=FAKE, kp=FAKE, vp=FAKE,
           bt=FAKE, lo=None, hi=None, ws=FAKE, n=256):
    p = params() if p is None else p
    return L.sparse_attn_append_kv_norm(C.byref(p), rows, cu, lens, pos, axes, axis, rotary, pairing, freq, qw, qws, kw, kws,
                                        eps, q, qs, k, ks, v, vs, qo, kp, vp, bt, lo, hi, ws, n, None)


def test_append_norm_refusals(L):
    bad = [dict(axes=0), dict(axes=9), dict(axis=None), dict(pos=None), dict(rotary=0, freq=None), dict(axis=FAKE + 2),
           dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(qws=64), dict(kws=-128),
           dict(qw=ODD), dict(kw=ODD), dict(q=None, qo=None),                # a weight for queries that are not there
           dict(rows=-1), dict(rows=9), dict(rotary=24), dict(pairing=0), dict(freq=None), dict(cu=FAKE, lens=None),
           dict(lo=FAKE), dict(k=None), dict(kp=None), dict(bt=None), dict(qo=ODD), dict(ks=255), dict(vs=128), dict(ws=None),
           dict(n=255), dict(pos=FAKE + 1)]
    for change in bad:
        assert append(L, **change) == B.INVALID_ARG, change
    assert append(L, p=params(head_dim=96)) == B.UNSUPPORTED
    assert append(L, rows=0, k=None, v=None, kp=None, vp=None, bt=None) == B.OK
    assert append(L, p=params(batch=0)) == B.OK


def shared(L, p=None, q=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, lens=FAKE, groups=2, cu=FAKE, pre=FAKE, mask=None, out=FAKE, ws=FAKE,
           n=1 << 40):
    p = params() if p is None else p
    return L.sparse_attn_shared_decode(C.byref(p), q, kp, vp, bt, lens, groups, cu, pre, mask, out, ws, n, None)


def test_shared_refusals(L):
    size = B.sparse_attn_shared_workspace_size(params(), 2)
    bad = [dict(q=None), dict(kp=None), dict(vp=None), dict(bt=None), dict(out=None), dict(ws=None), dict(ws=ODD),
           dict(n=size - 1), dict(q=ODD), dict(kp=ODD), dict(out=ODD), dict(bt=FAKE + 1), dict(lens=FAKE + 2),
           dict(mask=FAKE + 1), dict(groups=0), dict(groups=-1), dict(cu=None), dict(pre=None), dict(cu=FAKE + 2),
           dict(pre=FAKE + 1), dict(p=params(capacity_tokens=1004))]
    for change in bad:
        assert shared(L, **change) == B.INVALID_ARG, change
    assert shared(L, p=params(num_queries=1025, capacity_tokens=4000)) == B.UNSUPPORTED
    assert shared(L, groups=1 << 30) == B.UNSUPPORTED
    assert shared(L, p=params(batch=0)) == B.OK
    # one size for every context length
    assert size == B.sparse_attn_shared_workspace_size(params(n_tokens=0), 2) == \
        B.sparse_attn_shared_workspace_size(params(n_tokens=100000, capacity_tokens=200000), 2)


def weigh(L, p=None, q=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, lens=FAKE, w=FAKE, out=FAKE, ws=FAKE, n=1 << 40):
    p = params() if p is None else p
    return L.sparse_attn_weigh_decode(C.byref(p), q, kp, vp, bt, lens, w, out, ws, n, None)


def test_weigh_refusals(L):
    size = B.sparse_attn_weigh_workspace_size(params())
    bad = [dict(q=None), dict(kp=None), dict(vp=None), dict(bt=None), dict(out=None), dict(w=None), dict(ws=None),
           dict(ws=ODD), dict(n=size // 2), dict(q=ODD), dict(vp=ODD), dict(w=ODD), dict(out=ODD), dict(bt=FAKE + 1),
           dict(lens=FAKE + 2), dict(p=params(capacity_tokens=1004)), dict(p=params(softmax_scale=float("nan")))]
    for change in bad:
        assert weigh(L, **change) == B.INVALID_ARG, change
    assert weigh(L, p=params(num_queries=1025, capacity_tokens=4000)) == B.UNSUPPORTED
    assert weigh(L, p=params(batch=0)) == B.OK


def evict(L, p=None, lens=FAKE, keep=200, keep_lens=None, sinks=4, recent=32, w=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, nt=FAKE,
          lo=None, hi=None, ids=FAKE, new=2 * FAKE, ws=FAKE, n=1 << 40):
    p = params() if p is None else p
    return L.sparse_attn_evict_tokens(C.byref(p), lens, keep, keep_lens, sinks, recent, w, kp, vp, bt, nt, lo, hi, ids, new,
                                      ws, n, None)


def test_evict_refusals(L):
    size = B.sparse_attn_evict_workspace_size(params(), 200)
    bad = [dict(w=None), dict(kp=None), dict(vp=None), dict(bt=None), dict(nt=None), dict(ids=None), dict(new=None),
           dict(ws=None), dict(ws=ODD), dict(n=size - 1), dict(w=ODD), dict(kp=ODD), dict(vp=ODD), dict(lo=FAKE),
           dict(hi=FAKE), dict(lo=ODD, hi=FAKE), dict(bt=FAKE + 1), dict(nt=FAKE + 2), dict(ids=FAKE + 1), dict(new=FAKE + 2),
           dict(keep=0), dict(keep=-5), dict(sinks=-1), dict(recent=-1), dict(sinks=170), dict(recent=197),
           dict(sinks=2**31 - 1, recent=2**31 - 1), dict(new=FAKE), dict(new=FAKE + 4), dict(new=FAKE - 4),
           dict(lens=None, keep_lens=FAKE, new=FAKE + 4), dict(keep_lens=FAKE + 1)]
    for change in bad:
        assert evict(L, **change) == B.INVALID_ARG, change
    assert evict(L, p=params(capacity_tokens=32 * 16384 + 1)) == B.UNSUPPORTED
    assert evict(L, p=params(batch=1 << 20), keep=1 << 20) == B.UNSUPPORTED
    assert evict(L, p=params(batch=0)) == B.OK


def test_binding_wants_tensors_of_the_problems_shapes():
    p = params()
    cpu = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    pool = torch.zeros(1)
    with pytest.raises(ValueError, match="CUDA"):
        B.sparse_attn_shared_decode(p, cpu, pool, pool, i, i, i[:2], cpu, ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.sparse_attn_weigh_decode(p, cpu, pool, pool, i, pool, cpu, ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.sparse_attn_evict_tokens(p, 10, 0, 0, pool, pool, pool, i, i, i, i, ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.sparse_attn_append_kv_norm(p, cpu, cpu, cpu, None, None, 1e-6, None, cpu, pool, pool, i, ws)
