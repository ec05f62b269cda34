"""Two LongContextDecoders at work at the same time on two streams: what either computes by itself."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from query_guided_block_gb300.decoder import LongContextDecoder

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BATCH, HQ, HKV, D, BS, KEEP, STEPS = 4, 32, 8, 64, 32, 512, 4
CAPACITY = 4096


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class World:
    """Contexts of about 3000 tokens; every buffer that a step uses is the world's own."""

    def __init__(self, seed, drafts, stream):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(BF)
        nb, self.Q, self.stream = CAPACITY // BS, drafts, stream
        pages = BATCH * (nb + KEEP // BS + 2)                  # room to grow behind the budget, too
        self.k, self.v = normal(pages, HKV, BS, D), normal(pages, HKV, BS, D)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.table, self.new = order[: BATCH * nb].view(BATCH, nb).clone(), order[BATCH * nb:].view(BATCH, -1).contiguous()
        p = B.make_params(BATCH, HQ, HKV, D, CAPACITY - drafts, BS, pages, 0, 1, num_queries=drafts, capacity_tokens=CAPACITY)
        self.dec = LongContextDecoder(p, int32([3000, 2000, 2900, 3001]), num_groups=2, keep_tokens=KEEP)
        self.rows = [normal(BATCH * drafts, h, D) for h in (HQ, HKV, HKV)]
        self.weight, self.q = torch.ones(D, device="cuda"), torch.empty(BATCH * drafts, HQ, D, dtype=BF, device="cuda")
        self.freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).cuda()
        self.cuts, self.prefix, self.shared = int32([0, 2, 4]), int32([0, 2048]), int32([0, 2048])
        self.table[3, : 2048 // BS] = self.table[2, : 2048 // BS]
        self.outs = torch.zeros(STEPS, 2, BATCH, drafts, HQ, D, device="cuda")
        self.state = (self.dec.seq_lens, self.dec.weights, self.k, self.v, self.table, self.dec.kept_ids, self.outs)
        self.start = [x.clone() for x in self.state]

    def reset(self):
        for x, y in zip(self.state, self.start):
            x.copy_(y)
        self.prefix.copy_(self.shared)

    def step(self, i):
        s, d = self.stream, self.dec
        d.append_norm(*self.rows, self.weight, self.weight, 1e-6, self.freq, self.q, self.k, self.v, self.table, stream=s)
        q = self.q.view(BATCH, self.Q, HQ, D)
        with torch.cuda.stream(s):
            self.outs[i, 0].copy_(d.decode_shared(q, self.k, self.v, self.table, self.cuts, self.prefix, stream=s))
            self.outs[i, 1].copy_(d.decode_weighed(q, self.k, self.v, self.table, stream=s))
        d.accept(stream=s)
        if i == 1:
            d.evict(4, 64, self.k, self.v, self.table, self.new, stream=s)
            with torch.cuda.stream(s):
                self.prefix.zero_()

    def result(self):
        return [x.clone() for x in self.state]


@pytest.fixture(scope="module")
def worlds():
    """One of a token a step, one of windows of 16 (tensor cores); and what each computes by itself."""
    made = [World(1, 1, torch.cuda.Stream()), World(2, 16, torch.cuda.Stream())]
    alone = []
    for w in made:
        torch.cuda.synchronize()
        for i in range(STEPS):
            w.step(i)
            torch.cuda.synchronize()
        alone.append(w.result())
        assert w.dec.device_error() == 0 and w.dec.seq_lens.tolist() == [KEEP + 2 * w.Q] * BATCH
        w.reset()
    torch.cuda.synchronize()
    return made, alone


def same(made, alone):
    for w, want in zip(made, alone):
        assert all(torch.equal(x, y) for x, y in zip(w.state, want))
        assert w.dec.device_error() == 0


def test_calls_in_turn(worlds):
    """Step by step, a call for one stream and the next for the other."""
    made, alone = worlds
    for _ in range(3):
        for i in range(STEPS):
            for w in made:
                w.step(i)
        torch.cuda.synchronize()
        same(made, alone)
        for w in made:
            w.reset()
        torch.cuda.synchronize()


def test_graphs_at_once(worlds):
    """All steps in a graph a world, both replayed behind a common event, several times over."""
    made, alone = worlds
    graphs = []
    for w in made:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=w.stream):
            w.reset()
            for i in range(STEPS):
                w.step(i)
        graphs.append(graph)
    for _ in range(5):
        go = torch.cuda.Event()
        go.record()
        for w, graph in zip(made, graphs):
            w.stream.wait_event(go)
            with torch.cuda.stream(w.stream):
                graph.replay()
        torch.cuda.synchronize()
        same(made, alone)
    for w in made:
        w.reset()
    torch.cuda.synchronize()
