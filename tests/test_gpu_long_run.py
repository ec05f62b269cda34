"""The long-context calls together, as a serving loop makes them: prompts with norms and several position axes
into the cache, weighed attention, eviction, more steps behind it; shared prefixes; captured steps."""
import math

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from query_guided_block_gb300.decoder import LongContextDecoder
from tests.draft_reference import U
from tests.long_reference import kept_tokens

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
BATCH, HQ, HKV, D, BS, Q, KEEP, SINKS, RECENT = 3, 8, 2, 64, 16, 4, 32, 2, 8
LENS = [70, 45, 90]


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class World:
    """A batch in a pool with pages to spare."""

    def __init__(self, seed=0, lens=LENS, groups=0, capacity=128):
        self.g = torch.Generator().manual_seed(seed)
        self.nb = capacity // BS
        pages = 4 * BATCH * self.nb
        self.free = torch.randperm(pages, generator=self.g).tolist()
        self.k = torch.zeros(pages, HKV, BS, D, dtype=BF, device="cuda")
        self.v = torch.zeros_like(self.k)
        self.table = self.pages(self.nb)
        p = B.make_params(BATCH, HQ, HKV, D, capacity - Q, BS, pages, 0, 1, num_queries=Q, capacity_tokens=capacity)
        self.dec = LongContextDecoder(p, int32(lens), num_groups=groups, keep_tokens=KEEP)
        self.qw, self.kw = (1 + 0.2 * torch.randn(D, generator=self.g)).cuda(), (1 + 0.2 * torch.randn(D, generator=self.g)).cuda()
        self.freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).cuda()
        self.axis = (torch.arange(D // 2) * 3 // (D // 2)).to(torch.int32).cuda()

    def pages(self, n):
        return int32([[self.free.pop() for _ in range(n)] for _ in range(BATCH)])

    def rows(self, n):
        x = torch.randn(n, (HQ + 2 * HKV) * D, generator=self.g).to(BF).cuda()
        return [y.unflatten(1, (-1, D)) for y in x.split([HQ * D, HKV * D, HKV * D], 1)]

    def append(self, counts, positions, rows=None, stream=None):
        """Rows of each sequence at these places in time, rows and columns of images beside it; the rotated queries."""
        q, k, v = self.rows(sum(counts)) if rows is None else rows
        cu = int32([0] + torch.tensor(counts).cumsum(0).tolist())
        out = torch.empty(q.shape, dtype=BF, device="cuda")
        self.dec.append_norm(q, k, v, self.qw, self.kw, 1e-6, self.freq, out, self.k, self.v, self.table, cu_rows=cu,
                             positions=positions, axis_of=self.axis, stream=stream)
        return out

    def token(self, b, h, t):
        page = int(self.table[b, t // BS])
        return self.k[page, h, t % BS].double().cpu(), self.v[page, h, t % BS].double().cpu()


def positions(starts, counts):
    t = torch.cat([torch.arange(s, s + n) for s, n in zip(starts, counts)])
    return torch.stack([t, t // 7, t % 7]).to(torch.int32).cuda()


def check_step(w, ctx, q, out, before):
    """Attention over the lists of (key, value) and the weights' growth, in 64 bits.  Few tokens and unit
    variance: scores are below 64, so 2^-18 covers a weight's error (64 units 2^-23 of score, exp2's 2^-21), and with
    values below 8 an output is within 2^-14."""
    got, weights = out.double().cpu(), w.dec.weights.double().cpu()
    for b in range(BATCH):
        for h in range(HKV):
            k, v = (torch.stack(x) for x in zip(*ctx[b][h]))
            n = len(ctx[b][h]) - Q
            grown = torch.zeros(n + Q, dtype=torch.float64)
            for i in range(Q):
                for g in range(HQ // HKV):
                    head = h * (HQ // HKV) + g
                    s = k[: n + i + 1] @ q[b, i, head].double().cpu() / math.sqrt(D)
                    p = torch.softmax(s, 0)
                    grown[: n + i + 1] += p
                    assert (got[b, i, head] - p @ v[: n + i + 1]).abs().max() < 2.0 ** -14
            old = torch.cat([before[b, h, :n], torch.zeros(Q, dtype=torch.float64)])
            assert ((weights[b, h, : n + Q] - old - grown).abs() <= 2.0 ** -18 * grown + 2 * U * (old + grown)).all()


def test_a_serving_loop():
    w = World(lens=[0, 0, 0])
    w.append([n - Q for n in LENS], positions([0, 0, 0], [n - Q for n in LENS]))
    w.dec.seq_lens.copy_(int32([n - Q for n in LENS]))
    ctx = [[[w.token(b, h, t) for t in range(LENS[b] - Q)] for h in range(HKV)] for b in range(BATCH)]
    now = [n - Q for n in LENS]                                            # positions in time, whatever is evicted
    for turn in range(5):
        before = w.dec.weights.double().cpu()
        lens = w.dec.seq_lens.tolist()
        q = w.append([Q] * BATCH, positions(now, [Q] * BATCH)).view(BATCH, Q, HQ, D)
        now = [n + Q for n in now]
        for b in range(BATCH):
            for h in range(HKV):
                ctx[b][h] += [w.token(b, h, t) for t in range(lens[b], lens[b] + Q)]
        out = w.dec.decode_weighed(q, w.k, w.v, w.table)
        check_step(w, ctx, q, out, before)
        w.dec.accept()
        if turn in (0, 3):                                                 # down to the budget
            weights, lens = w.dec.weights.cpu(), w.dec.seq_lens.tolist()
            w.dec.evict(SINKS, RECENT, w.k, w.v, w.table, w.pages(-(-KEEP // BS)))
            assert w.dec.seq_lens.tolist() == [min(n, KEEP) for n in lens]
            for b in range(BATCH):
                for h in range(HKV):
                    keep = kept_tokens(weights[b, h].tolist(), lens[b], KEEP, SINKS, RECENT)
                    ctx[b][h] = [ctx[b][h][t] for t in keep]
                    for i, t in enumerate(keep):
                        k, v = w.token(b, h, i)
                        assert torch.equal(k, ctx[b][h][i][0]) and torch.equal(v, ctx[b][h][i][1])
                    assert torch.equal(w.dec.weights[b, h, : len(keep)].cpu(), weights[b, h, keep])
    assert w.dec.device_error() == 0


def test_sequences_left_alone_keep_their_pages():
    w = World()
    w.dec.weights.uniform_()
    before, new = w.table.clone(), w.pages(2)
    w.dec.evict(SINKS, RECENT, w.k, w.v, w.table, new, keep_lens=int32([20, -1, 32]))
    assert w.dec.seq_lens.tolist() == [20, LENS[1], 32]
    assert torch.equal(w.table[1], before[1]) and torch.equal(w.table[0, :2], new[0]) and torch.equal(w.table[:, 2:], before[:, 2:])


def test_shared_prefix_is_the_same_attention():
    """The sequences of a batch that was sampled from one prompt: with the prefix shared, and each by itself."""
    w = World(lens=[0, 0, 0], groups=2)
    prefix, part = 40, [9, 20, 3]
    w.table[1:, : prefix // BS] = w.table[0, : prefix // BS]
    q0, k0, v0 = w.rows(prefix)
    copies = [torch.cat([x] * BATCH) for x in (q0, k0, v0)]                # each writes the same rows, shared pages too
    for b in range(BATCH):
        w.dec.seq_lens.copy_(int32([0 if x == b else -1 for x in range(BATCH)]))
        w.append([prefix] * BATCH, positions([0] * BATCH, [prefix] * BATCH), rows=copies)
    w.dec.seq_lens.fill_(prefix)
    w.append(part, positions([prefix] * BATCH, part))
    w.dec.seq_lens.copy_(int32([prefix + n for n in part]))
    q = w.append([Q] * BATCH, positions([prefix + n for n in part], [Q] * BATCH)).view(BATCH, Q, HQ, D)
    alone = w.dec.decode(q, w.k, w.v, w.table).clone()
    for cuts, lens in (([0, 3], [prefix]), ([0, 2, 3], [32, 40])):
        out = w.dec.decode_shared(q, w.k, w.v, w.table, int32(cuts), int32(lens))
        # two fp32 computations: each within the error of check_step
        assert (out - alone).abs().max() < 2.0 ** -13
    with pytest.raises(ValueError, match="room for 2"):
        w.dec.decode_shared(q, w.k, w.v, w.table, int32([0, 1, 2, 3]), int32([0, 0, 0]))
    assert w.dec.device_error() == 0


@pytest.mark.parametrize("side", [False, True])
def test_captured_steps_replay_as_the_contexts_grow(side):
    """Append, weighed attention and the lengths' growth in one graph, eviction in another, on one workspace: the
    same bits as step by step."""
    worlds = [World(seed=3), World(seed=3)]
    rows = worlds[0].rows(Q * BATCH)
    pos = positions(LENS, [Q] * BATCH)
    new = worlds[0].pages(2)
    for w in worlds:
        w.dec.seq_lens.copy_(int32(LENS))
        w.dec.weights.uniform_(generator=torch.Generator(device="cuda").manual_seed(5))
        w.k.normal_(generator=torch.Generator(device="cuda").manual_seed(6))
        w.v.normal_(generator=torch.Generator(device="cuda").manual_seed(7))
    outs = []

    def step(w, stream=None):
        q = w.append([Q] * BATCH, pos, rows=rows, stream=stream)
        out = w.dec.decode_weighed(q.view(BATCH, Q, HQ, D), w.k, w.v, w.table, stream=stream)
        w.dec.accept(stream=stream)
        return out

    a, b = worlds
    for _ in range(3):
        outs.append(step(a).clone())
    a.dec.evict(SINKS, RECENT, a.k, a.v, a.table, new)
    outs.append(step(a).clone())

    start = [x.clone() for x in (b.dec.seq_lens, b.dec.weights, b.k, b.v, b.table)]
    cu = int32([Q * i for i in range(BATCH + 1)])
    q_out = torch.empty(Q * BATCH, HQ, D, dtype=BF, device="cuda")

    def captured_step():
        b.dec.append_norm(*rows, b.qw, b.kw, 1e-6, b.freq, q_out, b.k, b.v, b.table, cu_rows=cu, positions=pos, axis_of=b.axis)
        b.dec.decode_weighed(q_out.view(BATCH, Q, HQ, D), b.k, b.v, b.table)
        b.dec.accept()

    stream = torch.cuda.Stream() if side else torch.cuda.current_stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        captured_step()                                                    # before the capture: kernels are set up
        b.dec.evict(SINKS, RECENT, b.k, b.v, b.table, new)
        torch.cuda.synchronize()
        one, two = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(one):
            captured_step()
        with torch.cuda.graph(two):
            b.dec.evict(SINKS, RECENT, b.k, b.v, b.table, new)
        for x, y in zip((b.dec.seq_lens, b.dec.weights, b.k, b.v, b.table), start):
            x.copy_(y)
        for i in range(3):
            one.replay()
            assert torch.equal(b.dec.out, outs[i]), i
        two.replay()
        one.replay()
        assert torch.equal(b.dec.out, outs[3])
    torch.cuda.synchronize()
    assert torch.equal(a.dec.weights, b.dec.weights) and torch.equal(a.dec.seq_lens, b.dec.seq_lens)
    assert torch.equal(a.k, b.k) and torch.equal(a.table, b.table) and torch.equal(a.dec.kept_ids, b.dec.kept_ids)
    assert a.dec.device_error() == 0 and b.dec.device_error() == 0


def test_two_streams_at_once():
    """Two caches, each with a workspace of its own, on two streams: the bits of one after the other."""
    def work(w, rows, pos, new, stream):
        outs = []
        for _ in range(6):
            q = w.append([Q] * BATCH, pos, rows=rows, stream=stream).view(BATCH, Q, HQ, D)
            with torch.cuda.stream(stream):
                outs.append(w.dec.decode_weighed(q, w.k, w.v, w.table, stream=stream).clone())
                outs.append(w.dec.decode_shared(q, w.k, w.v, w.table, cuts, prefix, stream=stream).clone())
        w.dec.evict(SINKS, RECENT, w.k, w.v, w.table, new, stream=stream)
        return outs

    cuts, prefix = int32([0, 1, 2, 3]), int32([40, 45, 3])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for together in (False, True):
        worlds = [World(seed=11, groups=3), World(seed=12, groups=3)]
        made = []
        for w in worlds:
            w.k.normal_(generator=torch.Generator(device="cuda").manual_seed(8))
            w.v.normal_(generator=torch.Generator(device="cuda").manual_seed(9))
            made.append((w, w.rows(Q * BATCH), positions(LENS, [Q] * BATCH), w.pages(2)))
        torch.cuda.synchronize()
        outs = []
        for m, s in zip(made, streams if together else [streams[0]] * 2):
            outs.append(work(*m, s))
            if not together:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        got.append([x for o in outs for x in o] + [y for w in worlds for y in (w.dec.weights, w.k, w.v, w.dec.kept_ids, w.table)])
        assert all(w.dec.device_error() == 0 for w in worlds)
    assert all(torch.equal(x, y) for x, y in zip(*got))
