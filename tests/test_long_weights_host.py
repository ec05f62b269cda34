"""Refusals of the append that sets new tokens' weights, on the host before any launch (no GPU needed): the
pointers here are never dereferenced."""
import ctypes as C

import pytest

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.test_long_host import FAKE, ODD, params


@pytest.fixture(scope="module")
def L():
    build()
    return B.lib()


def append(L, rows=10, eps=1e-6, qw=FAKE, k=FAKE, w=FAKE, ws=FAKE, n=256):
    p = params()
    return L.sparse_attn_append_kv_weights(C.byref(p), rows, None, FAKE, FAKE, 3, FAKE, 128, 1, FAKE, qw, 0, FAKE, 128, eps,
                                           FAKE, 1024, k, 256, FAKE, 256, FAKE, FAKE, FAKE, FAKE, None, None, w, ws, n, None)


def test_refusals(L):
    for change in (dict(w=ODD), dict(w=FAKE + 1), dict(k=None), dict(eps=0.0), dict(rows=9), dict(ws=None), dict(n=255),
                   dict(qw=ODD)):
        assert append(L, **change) == B.INVALID_ARG, change
    assert append(L, rows=0, k=None, w=None) == B.OK
