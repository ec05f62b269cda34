"""Refusals of the call behind an eviction, on the host before any launch (no GPU needed): the pointers here are never
dereferenced."""
import ctypes as C

import pytest

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.test_long_host import FAKE, ODD, params


@pytest.fixture(scope="module")
def L():
    build()
    return B.lib()


FAR = 1 << 24


def adopt(L, p=None, lens=FAKE, keep=200, keep_lens=None, sinks=4, recent=32, new=2 * FAKE, bt=FAR, nt=2 * FAR, width=7, w=FAKE,
          ws=FAKE, n=1 << 40):
    p = params() if p is None else p
    return L.sparse_attn_evict_adopt(C.byref(p), lens, keep, keep_lens, sinks, recent, new, bt, nt, width, w, ws, n, None)


def test_refusals(L):
    size = B.sparse_attn_evict_workspace_size(params(), 200)
    bad = [dict(lens=None), dict(new=None), dict(bt=None), dict(nt=None), dict(ws=None), dict(ws=ODD), dict(n=size - 1), dict(w=ODD),
           dict(lens=FAKE + 2), dict(new=2 * FAKE + 1), dict(bt=FAR + 2), dict(nt=2 * FAR + 1), dict(keep_lens=FAR // 2 + 1),
           dict(keep=0), dict(sinks=-1), dict(recent=-1), dict(sinks=170), dict(width=6), dict(width=0), dict(width=-1),
           dict(width=33), dict(new=FAKE), dict(new=FAKE + 4), dict(keep_lens=FAKE - 4), dict(nt=FAR + 32), dict(nt=FAR - 4),
           dict(new=FAR + 8), dict(lens=FAR + 8)]
    for change in bad:
        assert adopt(L, **change) == B.INVALID_ARG, change
    assert adopt(L, p=params(head_dim=96)) == B.UNSUPPORTED
    assert adopt(L, p=params(batch=1 << 26), keep=7, width=1, sinks=0, recent=0) == B.UNSUPPORTED
    assert adopt(L, p=params(batch=0)) == B.OK
