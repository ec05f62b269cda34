"""The binding and the classes of the draft calls, without a GPU: what they ask of the library and on
which device."""
import contextlib
import ctypes as C

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300 import decoder
from query_guided_block_gb300.build import build

F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    B.lib()


def params(**over):
    kw = dict(batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, n_tokens=1000, block_size=32, num_pages=100,
              window_tokens=40, topk=4, num_queries=5, capacity_tokens=1005)
    kw.update(over)
    return B.make_params(**kw)


@pytest.mark.parametrize("kv", [BF, F32])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("block", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("queries", [1, 5])
@pytest.mark.parametrize("two_level", [False, True])
def test_selection_width_is_known_wherever_the_tree_call_takes_a_selection(kv, dim, block, queries, two_level):
    p = params(kv_dtype=kv, head_dim=dim, block_size=block, num_queries=queries, two_level=two_level, coarse_block=256,
               topk_coarse=2)
    size = C.c_size_t()
    assert B.lib().sparse_attn_tree_workspace_size(C.byref(p), C.byref(size)) == B.OK
    nb = -(-1000 // block)
    first = 960 // block
    width = min(4, first) + nb - first
    assert B.sparse_attn_sel_stride(p) == width
    assert B._shapes(p).sel == (2, 2, width)


def test_selection_width_of_bad_parameters_is_refused():
    for over in (dict(head_dim=96), dict(num_q_heads=6), dict(block_size=48), dict(topk=-1), dict(n_tokens=32 * 16384 + 1, capacity_tokens=0)):
        with pytest.raises(B.SparseAttnError):
            B.sparse_attn_sel_stride(params(**over))


def test_the_error_word_is_read_on_the_decoders_device(monkeypatch):
    """With another device current, the read must wait for the stream of the decoder's device."""
    asked = []

    class Stream:
        cuda_stream = 1234

    def current_stream(device=None):
        asked.append(("stream", None if device is None else torch.device(device)))
        return Stream()

    @contextlib.contextmanager
    def on(device):
        asked.append(("device", torch.device(device)))
        yield

    def read(ws, stream=None):
        asked.append(("read", stream))
        return 0

    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(decoder.B, "sparse_attn_get_device_error", read)
    dec = decoder.DraftDecoder.__new__(decoder.DraftDecoder)
    dec.device, dec.ws = torch.device("cuda", 3), None
    assert dec.device_error() == 0
    (first, device), *_, (last, stream) = asked
    assert (first, device) == ("device", torch.device("cuda", 3)) and last == "read"
    # the default of the read is the current stream of the current device, which is 3 by then
    assert stream is None or ("stream", torch.device("cuda", 3)) in asked
    asked.clear()
    assert dec.device_error(77) == 0 and asked[-1] == ("read", 77)


def test_commit_refuses_new_lengths_over_its_other_inputs():
    """Every KV head's CTA reads the path and its length while the first one writes the new length.
    (Refused on the host: nothing is launched.)"""
    p = params()
    at = 1 << 20
    lens, path, count, pools, new = at, at + 256, at + 512, at + 4096, at + 1024

    def commit(lens=lens, path=path, stride=4, count=count, new=new):
        return B.lib().sparse_attn_commit_drafts(C.byref(p), lens, path, stride, count, pools, pools, at, None, None, new,
                                                 at, 256, None)

    for over in (dict(new=lens), dict(new=lens + 4), dict(new=lens - 4), dict(new=path), dict(new=path + 28),
                 dict(new=path - 4), dict(new=count), dict(new=count + 4), dict(new=count - 4)):
        assert commit(**over) == B.INVALID_ARG, over
