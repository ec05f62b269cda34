"""Refusals of the cache-growing and draft-tree calls, on the host before any launch (no GPU
needed): the pointers here are never dereferenced."""
import ctypes as C

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case

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


def append(L, p=None, rows=10, cu=None, lens=FAKE, pos=None, rotary=128, pairing=1, freq=FAKE, q=FAKE, qs=1024, k=FAKE,
           ks=256, v=FAKE, vs=256, qo=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, lo=None, hi=None, ws=FAKE, n=256):
    p = params() if p is None else p
    return L.sparse_attn_append_kv(C.byref(p), rows, cu, lens, pos, rotary, pairing, freq, q, qs, k, ks, v, vs, qo, kp, vp,
                                   bt, lo, hi, ws, n, None)


def test_append_refusals(L):
    bad = [dict(rows=-1), dict(rows=9), dict(rotary=-16), dict(rotary=144), dict(rotary=24), dict(pairing=0),
           dict(pairing=3), dict(freq=None), dict(freq=ODD), dict(cu=FAKE, lens=None), dict(q=None), dict(qo=None),
           dict(lo=FAKE), dict(hi=FAKE), dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(bt=None),
           dict(k=ODD), dict(q=ODD), dict(qo=ODD), dict(kp=ODD), dict(lo=ODD, hi=FAKE), dict(ks=255), dict(ks=260),
           dict(vs=128), dict(qs=1023), dict(qs=1028), dict(ws=None), dict(ws=ODD), dict(n=255),
           dict(lens=None, rows=2002), dict(cu=FAKE + 1), dict(lens=FAKE + 2), dict(pos=FAKE + 1),
           dict(q=FAKE, qo=FAKE, qs=2048), dict(p=params(num_pages=0, n_tokens=0, capacity_tokens=0))]
    for change in bad:
        assert append(L, **change) == B.INVALID_ARG, change
    assert append(L, p=params(head_dim=96)) == B.UNSUPPORTED
    assert append(L, p=params(num_q_heads=6)) == B.UNSUPPORTED
    assert append(L, p=params(capacity_tokens=32 * 16384 + 1)) == B.UNSUPPORTED
    assert append(L, p=params(num_pages=2**30 + 1)) == B.UNSUPPORTED       # page x head beyond 32 bits
    # nothing to do: no pointer is looked at
    assert append(L, rows=0, k=None, v=None, kp=None, vp=None, bt=None) == B.OK
    assert append(L, p=params(batch=0), rows=10) == B.OK


def tree(L, p=None, q=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, lens=FAKE, ids=None, cnt=None, mask=None, out=FAKE, ws=FAKE, n=None):
    p = params() if p is None else p
    n = 1 << 40 if n is None else n
    return L.sparse_attn_tree_decode(C.byref(p), q, kp, vp, bt, lens, ids, cnt, mask, out, ws, n, None)


def test_tree_refusals(L):
    size = B.sparse_attn_tree_workspace_size(params())
    bad = [dict(q=None), dict(kp=None), dict(vp=None), dict(bt=None), dict(out=None), dict(ws=None), dict(ws=ODD),
           dict(n=size - 1), dict(q=ODD), dict(kp=ODD), dict(vp=ODD), dict(out=ODD), dict(bt=FAKE + 1), dict(lens=FAKE + 2),
           dict(mask=FAKE + 1), dict(ids=FAKE), dict(cnt=FAKE), dict(ids=FAKE + 1, cnt=FAKE),
           dict(p=params(capacity_tokens=1004)), dict(p=params(capacity_tokens=0)),
           dict(p=params(softmax_scale=float("inf")))]
    for change in bad:
        assert tree(L, **change) == B.INVALID_ARG, change
    assert tree(L, p=params(num_queries=1025, capacity_tokens=4000)) == B.UNSUPPORTED
    assert tree(L, p=params(batch=0)) == B.OK


def test_tree_workspace(L):
    """One size for every context length, any K/V type and selection kind; refused past 1024 drafts."""
    size = B.sparse_attn_tree_workspace_size(params())
    assert size == B.sparse_attn_tree_workspace_size(params(n_tokens=0)) == \
        B.sparse_attn_tree_workspace_size(params(n_tokens=100000, capacity_tokens=200000))
    assert B.sparse_attn_tree_workspace_size(params(kv_dtype=torch.float32, q_dtype=torch.float32)) > 0
    assert B.sparse_attn_tree_workspace_size(params(two_level=True, block_size=64, topk_coarse=2)) > 0
    n = C.c_size_t()
    assert L.sparse_attn_tree_workspace_size(C.byref(params(num_queries=1025, capacity_tokens=4000)), C.byref(n)) == B.UNSUPPORTED
    assert L.sparse_attn_tree_workspace_size(C.byref(params()), None) == B.INVALID_ARG
    assert L.sparse_attn_tree_workspace_size(None, C.byref(n)) == B.INVALID_ARG


def commit(L, p=None, lens=FAKE, path=FAKE, stride=4, n=FAKE, kp=FAKE, vp=FAKE, bt=FAKE, lo=None, hi=None, new=FAKE + 64,
           ws=FAKE, size=256):
    p = params() if p is None else p
    return L.sparse_attn_commit_drafts(C.byref(p), lens, path, stride, n, kp, vp, bt, lo, hi, new, ws, size, None)


def test_commit_refusals(L):
    bad = [dict(path=None), dict(stride=-1), dict(n=None), dict(kp=None), dict(vp=None), dict(bt=None), dict(new=None),
           dict(ws=None), dict(size=255), dict(lo=FAKE), dict(hi=FAKE), dict(path=FAKE + 2), dict(kp=ODD), dict(vp=ODD),
           dict(new=FAKE), dict(new=FAKE + 4), dict(new=FAKE - 4), dict(lens=FAKE + 1), dict(n=FAKE + 1),
           dict(p=params(capacity_tokens=1004)), dict(lo=ODD, hi=FAKE)]
    for change in bad:
        assert commit(L, **change) == B.INVALID_ARG, change
    assert commit(L, p=params(num_queries=1025, capacity_tokens=4000)) == B.UNSUPPORTED
    assert commit(L, p=params(batch=0)) == B.OK


def test_binding_refuses_host_tensors_and_wrong_shapes():
    """The binding checks device, shape, dtype and layout before the library is called."""
    c = Case()
    p = c.params()
    table = c.block_table()
    k, v = c.pools()
    ws = torch.zeros(256, dtype=torch.uint8)
    rows = torch.zeros(4, c.hkv, c.dim, dtype=c.dtype)
    with pytest.raises(ValueError, match="CUDA"):
        B.sparse_attn_append_kv(p, None, rows, rows, None, None, k, v, table, ws)
    q = torch.zeros(c.batch, c.drafts, c.hq, c.dim, dtype=c.dtype)
    with pytest.raises(ValueError, match="CUDA"):
        B.sparse_attn_tree_decode(p, q, k, v, table, q.float(), ws)
    with pytest.raises(ValueError, match="CUDA"):
        B.sparse_attn_commit_drafts(p, torch.zeros(2, 3, dtype=torch.int32), table, k, v, table, table, ws)
