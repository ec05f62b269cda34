"""Attention weights of tokens that come in where others were: behind an eviction, after rejected drafts, in
the slot of another request.  They start at zero, whatever the entries held."""
import math

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from query_guided_block_gb300.decoder import LongContextDecoder
from tests.draft_reference import U, Case, place
from tests.long_reference import kept_tokens

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BATCH, HQ, HKV, D, BS, Q, KEEP = 3, 8, 2, 64, 16, 4, 32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class World:
    def __init__(self, lens, capacity=160):
        self.g = torch.Generator().manual_seed(1)
        nb = capacity // BS
        pages = 3 * BATCH * nb
        self.free = torch.randperm(pages, generator=self.g).tolist()
        self.k = torch.randn(pages, HKV, BS, D, generator=self.g).to(BF).cuda()
        self.v = torch.randn(pages, HKV, BS, D, generator=self.g).to(BF).cuda()
        self.table = int32([[self.free.pop() for _ in range(nb)] for _ in range(BATCH)])
        p = B.make_params(BATCH, HQ, HKV, D, capacity - Q, BS, pages, 0, 1, num_queries=Q, capacity_tokens=capacity)
        self.dec = LongContextDecoder(p, int32(lens), keep_tokens=KEEP)

    def append(self, counts, norm):
        n = sum(counts)
        q, k, v = (torch.randn(n, h, D, generator=self.g).to(BF).cuda() for h in (HQ, HKV, HKV))
        cu = int32([0] + torch.tensor(counts).cumsum(0).tolist())
        out = torch.empty_like(q)
        args = (None, out, self.k, self.v, self.table, cu)
        if norm:
            w = torch.ones(D, device="cuda")
            self.dec.append_norm(q, k, v, w, w, 1e-6, *args)
        else:
            self.dec.append(q, k, v, *args)
        return out

    def queries(self):
        return torch.randn(BATCH, Q, HQ, D, generator=self.g).to(BF).cuda()

    def grown(self, b, h, q):
        """What a call of Q queries adds to the weights of the sequence's tokens, in 64 bits."""
        n = int(self.dec.seq_lens[b])
        t = torch.arange(n + Q)
        k = self.k[self.table[b].long().cpu()[t // BS], h, t % BS].double().cpu()
        sums = torch.zeros(n + Q, dtype=torch.float64)
        for i in range(Q):
            for head in range(h * HQ // HKV, (h + 1) * HQ // HKV):
                sums[: n + i + 1] += torch.softmax(k[: n + i + 1] @ q[b, i, head].double().cpu() / math.sqrt(D), 0)
        return sums


def check(w, q, before):
    """The weights after decode_weighed of q: those of `before` (a list of each sequence and head's sums) and what the
    call adds.  Scores of unit variance over 64 channels are below 64: 2^-18 of a weight (64 units 2^-23 of
    the score, exp2's 2^-21 and the total's), and a rounding of the sum."""
    got = w.dec.weights.double().cpu()
    for b in range(BATCH):
        for h in range(HKV):
            add = w.grown(b, h, q)
            old = torch.zeros_like(add)
            old[: len(before[b][h])] = before[b][h]
            assert ((got[b, h, : len(add)] - old - add).abs() <= 2.0 ** -18 * add + 2 * U * (old + add)).all(), (b, h)


@pytest.mark.parametrize("norm", [False, True])
def test_a_second_prompt_behind_an_eviction(norm):
    """The prompt of the next turn takes the indexes of evicted tokens; only its last tokens are weighed."""
    w = World([80, 70, 90])
    w.dec.weights.uniform_(1, 2)                                           # sums of a long first turn
    lens, old = w.dec.seq_lens.tolist(), w.dec.weights.cpu()
    new = int32([[w.free.pop() for _ in range(KEEP // BS)] for _ in range(BATCH)])
    w.dec.evict(2, 8, w.k, w.v, w.table, new)
    assert w.dec.seq_lens.tolist() == [KEEP] * BATCH
    assert (w.dec.weights[:, :, KEEP:] == 0).all()
    before = [[old[b, h, kept_tokens(old[b, h].tolist(), lens[b], KEEP, 2, 8)].double() for h in range(HKV)]
              for b in range(BATCH)]
    w.append([60, 33, Q], norm)
    w.dec.seq_lens.add_(int32([60 - Q, 33 - Q, 0]))
    q = w.queries()
    w.dec.decode_weighed(q, w.k, w.v, w.table)
    check(w, q, before)
    # and these sums, not those of tokens that are gone, say what the next eviction keeps
    w.dec.accept()
    weights, lens = w.dec.weights.cpu(), w.dec.seq_lens.tolist()
    w.dec.evict(2, 8, w.k, w.v, w.table, int32([[w.free.pop() for _ in range(KEEP // BS)] for _ in range(BATCH)]))
    for b in range(BATCH):
        for h in range(HKV):
            assert w.dec.kept_ids[b, h].tolist() == kept_tokens(weights[b, h].tolist(), lens[b], KEEP, 2, 8)
    assert w.dec.device_error() == 0


def test_a_sequence_left_alone_keeps_its_weights():
    w = World([80, 70, 20])
    w.dec.weights.uniform_(1, 2)
    old = w.dec.weights.clone()
    new = int32([[w.free.pop() for _ in range(KEEP // BS)] for _ in range(BATCH)])
    w.dec.evict(2, 8, w.k, w.v, w.table, new, keep_lens=int32([KEEP, -1, KEEP]))
    assert torch.equal(w.dec.weights[1], old[1])
    assert torch.equal(w.dec.weights[2, :, :20], old[2, :, :20]) and (w.dec.weights[2, :, 20:] == 0).all()


@pytest.mark.parametrize("norm", [False, True])
def test_a_slot_given_to_another_request(norm):
    w = World([80, 70, 90])
    w.dec.weights.uniform_(1, 2)
    old = w.dec.weights.double().cpu()
    w.dec.seq_lens.copy_(int32([80, 0, 90]))
    w.append([Q, 50, Q], norm)
    w.dec.seq_lens.add_(int32([0, 50 - Q, 0]))
    q = w.queries()
    w.dec.decode_weighed(q, w.k, w.v, w.table)
    check(w, q, [[old[0, h, :80] for h in range(HKV)], [old[1, h, :0] for h in range(HKV)], [old[2, h, :90] for h in range(HKV)]])


@pytest.mark.parametrize("how", ["rejected", "abandoned"])
def test_tokens_that_were_weighed_and_did_not_stay(how):
    """Drafts that a commit rejects, or that are never accepted: a prompt in their place starts at zero."""
    w = World([40, 30, 20])
    w.append([Q] * BATCH, False)
    w.dec.decode_weighed(w.queries(), w.k, w.v, w.table)
    if how == "rejected":
        path = int32([list(range(Q))] * BATCH)
        w.dec.commit(path, int32([1, 0, 2]), w.k, w.v, w.table)
    lens, old = w.dec.seq_lens.tolist(), w.dec.weights.double().cpu()
    assert lens == ([41, 30, 22] if how == "rejected" else [40, 30, 20])
    w.append([30, 30, 30], False)
    w.dec.seq_lens.add_(30 - Q)
    q = w.queries()
    w.dec.decode_weighed(q, w.k, w.v, w.table)
    check(w, q, [[old[b, h, :n] for h in range(HKV)] for b, n in enumerate(lens)])


APPENDS = {
    "one": dict(batch=1, counts=[1], lens=[300]),
    "ragged": dict(batch=5, counts=[200, 0, 1, 33, 65], lens=[0, 7, -1, 64, 31]),
    "heads": dict(batch=2, counts=[40, 90], lens=[100, 3], hq=16, hkv=16),
    "block_128": dict(batch=2, counts=[200, 128], lens=[100, 0], block=128),
    "fp32": dict(batch=2, counts=[70, 5], lens=[60, 1], dtype=torch.float32),
}


@pytest.mark.parametrize("kind", ["plain", "norm", "norm_heads"])
@pytest.mark.parametrize("name", APPENDS)
def test_the_append_sets_the_new_entries_alone(name, kind):
    """The new tokens' entries become 0, no other is touched, and the rest of the call is as without weights."""
    kw = dict(APPENDS[name])
    counts, lens, dtype = kw.pop("counts"), kw.pop("lens"), kw.pop("dtype", BF)
    c = Case(lens=tuple(lens), context=300, room=100, dim=64, dtype=dtype, kv=dtype, **kw)
    table, rows = c.block_table().cuda(), sum(counts)
    q, k, v = (c.normal(s, rows, h, c.dim).cuda() for s, h in (("q", c.hq), ("k", c.hkv), ("v", c.hkv)))
    heads = {"plain": None, "norm": (), "norm_heads": (1,)}[kind]
    qw, kw_ = (None, None) if heads is None else (torch.rand(*((h,) if heads else ()), c.dim, device="cuda") for h in (c.hq, c.hkv))
    cu = int32([0] + torch.tensor(counts).cumsum(0).tolist())
    made = []
    for weights in (None, torch.full((c.batch, c.hkv, c.nb_cap * c.block), float("nan"), device="cuda")):
        pools = [x.cuda() for x in c.pools(empty=0.0)]
        out, ws = torch.zeros_like(q), torch.zeros(256, dtype=torch.uint8, device="cuda")
        box = [torch.zeros(c.batch, c.hkv, c.nb_cap, c.dim, dtype=dtype, device="cuda") for _ in range(2)]
        B.sparse_attn_append_kv_norm(c.params(), q, k, v, qw, kw_, 1e-6, None, out, *pools, table, ws, cu, int32(lens),
                                     kmin=box[0], kmax=box[1], weights=weights)
        assert B.sparse_attn_get_device_error(ws) == 0
        made.append([out, *pools, *box])
    assert all(torch.equal(x, y) for x, y in zip(*made))
    for b, (n, m) in enumerate(zip(lens, counts)):
        set_ = torch.zeros(c.nb_cap * c.block, dtype=torch.bool, device="cuda")
        if n >= 0:
            set_[n:n + m] = True
        assert (weights[b][:, set_] == 0).all() and weights[b][:, ~set_].isnan().all()


def test_uniform_appends_and_bad_pages():
    """Without cu_rows and lengths; a token without a page has an entry all the same."""
    c = Case(batch=2, context=300, room=50)
    table = c.block_table()
    table[0, 9] = -1
    k, v = c.normal("k", 14, c.hkv, c.dim).cuda(), c.normal("v", 14, c.hkv, c.dim).cuda()
    pools = [x.cuda() for x in c.pools(empty=0.0)]
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    w = torch.ones(c.batch, c.hkv, c.nb_cap * c.block, device="cuda")
    B.sparse_attn_append_kv_norm(c.params(), None, k, v, None, None, 0.0, None, None, *pools, table.cuda(), ws, weights=w)
    assert B.sparse_attn_get_device_error(ws) == B.ERR_PAGE
    t = torch.arange(293, 300)
    assert (w[:, :, t] == 0).all() and w.sum() == w.numel() - c.batch * c.hkv * 7
    page, off = place(c, table, 1, t)
    assert torch.equal(pools[0].cpu()[page, :, off], k.cpu()[7:])
