"""The page table behind an eviction: what a sequence grows into afterwards, beside a sequence that shared its
first pages."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from query_guided_block_gb300.decoder import LongContextDecoder

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HQ, HKV, D, BS, Q, KEEP = 8, 2, 64, 16, 4, 32
CAPACITY, PREFIX = 160, 64


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class World:
    """Sequences 0 and 1 share a prefix of 64 tokens; 2 is by itself, 3 inactive."""

    def __init__(self):
        g = self.g = torch.Generator().manual_seed(4)
        nb, batch = CAPACITY // BS, 4
        pages = 12 * nb
        self.free = torch.randperm(pages, generator=g).tolist()
        self.k = torch.randn(pages, HKV, BS, D, generator=g).to(BF).cuda()
        self.v = torch.randn(pages, HKV, BS, D, generator=g).to(BF).cuda()
        table = [[self.free.pop() for _ in range(nb)] for _ in range(batch)]
        table[1][: PREFIX // BS] = table[0][: PREFIX // BS]
        table[3] = [table[2][5]] * nb                                      # nothing: its row may hold anything
        self.table = int32(table)
        p = B.make_params(batch, HQ, HKV, D, CAPACITY - Q, BS, pages, 0, 1, num_queries=Q, capacity_tokens=CAPACITY)
        self.dec = LongContextDecoder(p, int32([100, 90, 110, -1]), num_groups=2, keep_tokens=KEEP)
        self.dec.weights.uniform_()

    def new(self, n=KEEP // BS):
        return int32([[self.free.pop() for _ in range(n)] for _ in range(4)])

    def append(self, counts):
        n = sum(counts)
        k, v = (torch.randn(n, HKV, D, generator=self.g).to(BF).cuda() for _ in range(2))
        self.dec.append(None, k, v, None, None, self.k, self.v, self.table, int32([0] + torch.tensor(counts).cumsum(0).tolist()))

    def context(self, b, n):
        t = torch.arange(n, device="cuda")
        page = self.table[b].long()[t // BS]
        return self.k[page, :, t % BS].clone(), self.v[page, :, t % BS].clone()


def test_a_sequence_that_grows_behind_an_eviction_leaves_its_sibling_alone():
    w = World()
    before, new = w.table.clone(), w.new()
    sibling, q = w.context(1, 90), torch.randn(4, Q, HQ, D, generator=w.g).to(BF).cuda()
    w.dec.seq_lens.copy_(int32([100, 86, 110, -1]))                        # the last four as drafts
    alone = w.dec.decode(q, w.k, w.v, w.table).clone()
    w.dec.evict(2, 8, w.k, w.v, w.table, new, keep_lens=int32([KEEP, -1, -1, KEEP]))
    assert w.dec.seq_lens.tolist() == [KEEP, 86, 110, -1]
    # its own pages stay in its row, the shared ones do not
    want = before.clone()
    want[0, :2] = new[0]
    want[0, 2:PREFIX // BS] = -1
    assert torch.equal(w.table, want)
    w.append([20, 0, 0, 0])                                                # past the new pages
    assert w.dec.device_error() == B.ERR_PAGE
    assert all(torch.equal(x, y) for x, y in zip(w.context(1, 90), sibling))
    # with pages of its own it grows
    w.table[0, 2:PREFIX // BS] = int32([w.free.pop(), w.free.pop()])
    w.append([20, 0, 0, 0])
    assert w.dec.device_error() == 0
    assert all(torch.equal(x, y) for x, y in zip(w.context(1, 90), sibling))
    out = w.dec.decode(q, w.k, w.v, w.table)
    assert torch.equal(out[1], alone[1]) and w.dec.device_error() == 0


def test_both_of_a_prefix_move():
    """Both rows lose the shared pages; a sequence by itself keeps its own, whatever an inactive row holds."""
    w = World()
    before, new = w.table.clone(), w.new()
    w.dec.evict(2, 8, w.k, w.v, w.table, new)
    want = before.clone()
    want[:3, :2] = new[:3]
    want[:2, 2:PREFIX // BS] = -1
    assert torch.equal(w.table, want) and w.dec.seq_lens.tolist() == [KEEP, KEEP, KEEP, -1]
    w.append([4, 4, 40, 0])
    assert w.dec.device_error() == B.ERR_PAGE
    w.table[:2, 2:PREFIX // BS] = w.new()[:2]
    w.append([4, 4, 40, 0])
    assert w.dec.device_error() == 0


@pytest.mark.parametrize("width", [CAPACITY // BS, 5])
def test_rows_replaced_beyond_the_budget(width):
    """new_table may reach past the kept tokens, up to the whole row."""
    w = World()
    before, new = w.table.clone(), w.new(width)
    new[:, 4:] = -1
    kept = [w.context(b, n) for b, n in ((0, 100), (1, 90), (2, 110))]
    w.dec.evict(2, 8, w.k, w.v, w.table, new)
    want = before.clone()
    want[:3, :width] = new[:3]
    assert torch.equal(w.table, want)
    for b in range(3):
        k, v = w.context(b, KEEP)
        for h in range(HKV):
            ids = w.dec.kept_ids[b, h].long()
            assert torch.equal(k[:, h], kept[b][0][ids, h]) and torch.equal(v[:, h], kept[b][1][ids, h])
    w.append([30, 30, 30, 0])
    assert w.dec.device_error() == 0
    with pytest.raises(ValueError, match="block_table has 10"):
        w.dec.evict(2, 8, w.k, w.v, w.table, int32([[0] * 11] * 4))
    with pytest.raises(ValueError, match="new_table"):
        w.dec.evict(2, 8, w.k, w.v, w.table, int32([[0]] * 4))


def test_captured_evictions():
    """The table after a replay is that of a call."""
    rows = []
    for captured in (False, True):
        w = World()
        start = [x.clone() for x in (w.table, w.dec.seq_lens, w.dec.weights.fill_(0.5))]
        new, wide = w.new(), w.new(5)
        for table in (new, wide):
            run = lambda: w.dec.evict(2, 8, w.k, w.v, w.table, table)
            if captured:
                run()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    run()
                for x, y in zip((w.table, w.dec.seq_lens, w.dec.weights), start):
                    x.copy_(y)
                run = graph.replay
            else:
                for x, y in zip((w.table, w.dec.seq_lens, w.dec.weights), start):
                    x.copy_(y)
            run()
            rows.append((w.table.clone(), w.dec.seq_lens.clone(), w.dec.kept_ids.clone(), w.dec.weights.clone()))
        assert w.dec.device_error() == 0
    for a, b in zip(rows[:2], rows[2:]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
