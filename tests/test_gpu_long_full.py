"""Contexts longer than the length that a LongContextDecoder's parameters name: the pages reach further."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from query_guided_block_gb300.decoder import LongContextDecoder
from tests.long_reference import kept_tokens

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BATCH, HQ, HKV, D, BS, Q, KEEP = 5, 8, 2, 64, 16, 4, 32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def world(lens, n_tokens, capacity):
    g = torch.Generator().manual_seed(2)
    nb = -(-capacity // BS)
    pages = BATCH * (nb + KEEP // BS)
    order = torch.randperm(pages, generator=g).to(torch.int32).cuda()
    k, v = (torch.randn(pages, HKV, BS, D, generator=g).to(BF).cuda() for _ in range(2))
    p = B.make_params(BATCH, HQ, HKV, D, n_tokens, BS, pages, 0, 1, num_queries=Q, capacity_tokens=capacity)
    dec = LongContextDecoder(p, int32(lens), keep_tokens=KEEP)
    dec.weights.uniform_()
    return dec, k, v, order[: BATCH * nb].view(BATCH, nb).clone(), order[BATCH * nb:].view(BATCH, -1).contiguous()


@pytest.mark.parametrize("n_tokens, capacity", [(156, 160), (100, 160), (17000, 17020)])
def test_a_full_context_is_evicted(n_tokens, capacity):
    lens = [n_tokens, n_tokens + 1, capacity - 1, capacity, -1]
    dec, k, v, table, new = world(lens, n_tokens, capacity)
    weights, before, old = dec.weights.cpu(), k.clone(), table.clone()
    dec.evict(2, 8, k, v, table, new)
    assert dec.device_error() == 0 and dec.seq_lens.tolist() == [KEEP] * 4 + [-1]
    assert torch.equal(table[:4, : KEEP // BS], new[:4]) and torch.equal(table[4], old[4])
    for b, n in enumerate(lens[:4]):
        for h in range(HKV):
            keep = kept_tokens(weights[b, h].tolist(), n, KEEP, 2, 8)
            assert dec.kept_ids[b, h].tolist() == keep
            t, i = torch.tensor(keep, device="cuda"), torch.arange(KEEP, device="cuda")
            assert torch.equal(k[new[b].long()[i // BS], h, i % BS], before[old[b].long()[t // BS], h, t % BS])
    # and goes on
    q = torch.randn(BATCH, Q, HQ, D, device="cuda").to(BF)
    rows = [torch.randn(BATCH * Q, HKV, D, device="cuda").to(BF) for _ in range(2)]
    dec.append(None, *rows, None, None, k, v, table)
    dec.decode_weighed(q, k, v, table)
    assert dec.device_error() == 0


def test_a_context_that_no_attention_took_does_not_grow():
    """The attention leaves contexts past n_tokens alone; so does accept, until there are parameters for them."""
    dec, k, v, table, _ = world([10, 100, 101, -1, 0], 100, 160)
    q = torch.randn(BATCH, Q, HQ, D, device="cuda").to(BF)
    rows = [torch.randn(BATCH * Q, HKV, D, device="cuda").to(BF) for _ in range(2)]
    dec.append(None, *rows, None, None, k, v, table)
    dec.decode_weighed(q, k, v, table)
    assert dec.device_error() == B.ERR_LENGTH
    dec.accept()
    assert dec.seq_lens.tolist() == [14, 104, 101, -1, 4]
    dec.p = B.make_params(BATCH, HQ, HKV, D, 156, BS, dec.p.num_pages, 0, 1, num_queries=Q, capacity_tokens=160)
    dec.append(None, *rows, None, None, k, v, table)
    dec.decode_weighed(q, k, v, table)
    assert dec.device_error() == 0
    dec.accept()
    assert dec.seq_lens.tolist() == [18, 108, 105, -1, 8]


def test_lengths_past_the_pages_are_reported():
    dec, k, v, table, new = world([161, -2, 160, 20, 0], 156, 160)
    before = table.clone()
    dec.evict(2, 8, k, v, table, new)
    assert dec.device_error() == B.ERR_LENGTH
    assert dec.seq_lens.tolist() == [161, -2, KEEP, 20, 0]
    assert torch.equal(table[:2], before[:2]) and torch.equal(table[2:, :2], new[2:])
