"""Weighed attention where its launches change: many output rows, either side of where scores are kept, one
workspace for both; against 64 bits."""
import math

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, U
from tests.test_gpu_weigh import run

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Batch:
    """Sequences over pages that they share (nothing writes them), too many for the page-by-page reference."""

    def __init__(self, lens, capacity, hq, hkv, drafts, dim=64, block=32, pages=300, dtype=BF, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.capacity, self.hq, self.hkv, self.drafts, self.dim, self.block = lens, capacity, hq, hkv, drafts, dim, block
        self.dtype, self.pages, self.nb_cap = dtype, pages, -(-capacity // block)
        self.k, self.v = (torch.randn(pages, hkv, block, dim, generator=g, device="cuda").to(dtype) for _ in range(2))
        self.table = torch.randint(0, pages, (len(lens), self.nb_cap), generator=g, device="cuda").to(torch.int32)
        self.q = torch.randn(len(lens), drafts, hq, dim, generator=g, device="cuda").to(dtype)
        self.before = torch.rand(len(lens), hkv, self.nb_cap * block, generator=g, device="cuda")

    def params(self, **over):
        kw = dict(kv_dtype=self.dtype, q_dtype=self.dtype, num_queries=self.drafts, capacity_tokens=self.capacity)
        kw.update(over)
        n = kw.pop("n_tokens", max(self.lens))
        return B.make_params(len(self.lens), self.hq, self.hkv, self.dim, n, self.block, self.pages, 0, 1, **kw)

    def call(self, p, ws):
        out, w = torch.full(self.q.shape, 5.0, device="cuda"), self.before.clone()
        B.sparse_attn_weigh_decode(p, self.q, self.k, self.v, self.table, w, out, ws, seq_lens=int32(self.lens))
        assert B.sparse_attn_get_device_error(ws) == 0
        return out, w

    def check(self, out, w, seqs):
        """Sequences `seqs` of a result against 64 bits, all at once, within the bounds that
        long_reference.attention_exact derives."""
        Q, G, scale = self.drafts, self.hq // self.hkv, 1 / math.sqrt(self.dim)
        n = torch.tensor([self.lens[b] for b in seqs], device="cuda")
        T = int(n.max()) + Q
        t = torch.arange(T, device="cuda")
        pages = self.table[seqs].long()[:, t // self.block]
        k, v = (x[pages, :, t % self.block].double().transpose(1, 2) for x in (self.k, self.v))       # [S, Hkv, T, D]
        q = self.q[seqs].double().view(len(seqs), Q, self.hkv, G, self.dim).transpose(1, 2).flatten(2, 3)
        s = q @ k.transpose(-1, -2) * scale
        last = n[:, None] + torch.arange(Q, device="cuda").repeat_interleave(G)                       # [S, R]
        seen = (t <= last[..., None])[:, None]
        p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
        held = 2.0 ** -21 if self.dtype == BF else 4 * 2.0 ** -21
        err = ((self.dim / 8 + 2) * 2 ** -22 + 2 ** -21) * (q.abs() @ k.abs().transpose(-1, -2)) * scale + s.abs() * 2 * U + held
        m = (last + 1)[:, None].double()
        total = (p * err).sum(-1) + (m / 4 + 64) * U
        exact, mag = p @ v, p @ v.abs()
        bound = (p * err) @ v.abs() + (total + (m / 32 + 64) * 2 ** -22)[..., None] * mag + 1e-30
        got = out[seqs].double().view(len(seqs), Q, self.hkv, G, self.dim).transpose(1, 2).flatten(2, 3)
        assert ((got - exact).abs() <= bound).all(), ((got - exact).abs() / bound).max()
        sums, R = p.sum(2), Q * G
        old = torch.where(t < n[:, None, None], self.before[seqs][:, :, :T].double(), torch.zeros((), device="cuda").double())
        limit = (p * (err + total[..., None])).sum(2) + (R + 2) * U * sums + U * (old + sums) + R * 2.0 ** -126
        behind = t >= (n + Q)[:, None, None]
        got = w[seqs][:, :, :T].double()
        assert ((got - old - sums).abs() <= limit)[~behind.expand_as(got)].all()
        assert torch.equal(w[seqs][:, :, T:], self.before[seqs][:, :, T:])
        assert torch.equal(w[seqs][:, :, :T][behind.expand_as(got)], self.before[seqs][:, :, :T][behind.expand_as(got)])


def fresh(size):
    ws = torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")
    B.sparse_attn_workspace_init(ws[:256])
    return ws


# 152 SMs: from 9728 output rows on a join of its own, from 38912 on one that looks eight rows' shares up at once
MANY = {
    "join_apart": dict(lens=[(7 * i) % 40 for i in range(420)], hq=32, hkv=8, drafts=1),
    "join_many": dict(lens=[(7 * i) % 40 for i in range(1300)], hq=32, hkv=8, drafts=1),
    "join_many_8_rows": dict(lens=[(7 * i) % 40 for i in range(700)], hq=32, hkv=8, drafts=2),
    "join_many_fp32": dict(lens=[(7 * i) % 40 for i in range(1300)], hq=32, hkv=8, drafts=1, dtype=F32),
    "join_many_tensor": dict(lens=[(7 * i) % 40 for i in range(70)], hq=32, hkv=8, drafts=20),
    "join_many_rows_28": dict(lens=[(7 * i) % 40 for i in range(200)], hq=32, hkv=8, drafts=7),
    "join_many_dim_128": dict(lens=[(7 * i) % 40 for i in range(1300)], hq=32, hkv=8, drafts=1, dim=128),
}


@pytest.mark.parametrize("long", [0, 900])
@pytest.mark.parametrize("name", MANY)
def test_many_output_rows(name, long):
    """Short contexts, whose rows the attention finishes, alone or with a few long ones in several parts."""
    kw = dict(MANY[name])
    lens = list(kw.pop("lens"))
    places = [3, 64, len(lens) - 1] if long else []
    for i, b in enumerate(places):
        lens[b] = long - 100 * i
    x = Batch(lens, max(lens) + kw["drafts"], **kw)
    out, w = x.call(x.params(), fresh(B.sparse_attn_weigh_workspace_size(x.params())))
    if places:
        x.check(out, w, places)
    rest = [b for b in range(len(lens)) if b not in places]
    for i in range(0, len(rest), 200):
        x.check(out, w, rest[i:i + 200])


def test_one_workspace_either_side_of_the_kept_scores():
    """36 rows x 32 units make 96 tiles of 16 rows for each 64 tokens: up to 384 tokens (608 tiles) scores are kept, beyond
    they are computed again.  A workspace of the capacity serves both, and nothing behind it is touched."""
    x = Batch([375, 300, 17, 0], 1000, hq=32, hkv=8, drafts=9)
    size = B.sparse_attn_weigh_workspace_size(x.params())
    assert size < 100 << 20
    room = torch.full((size + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    ws = room[:size]
    B.sparse_attn_workspace_init(ws[:256])
    for n in (375, 376, 991, 384, 311, 375):
        x.lens[0] = n
        out, w = x.call(x.params(n_tokens=n), ws)
        x.check(out, w, [0, 1, 2, 3])
        assert (room[size:] == 0xAB).all()
    assert B.sparse_attn_weigh_workspace_size(x.params(n_tokens=311, capacity_tokens=320)) <= size


def test_one_workspace_either_side_of_256_megabytes():
    """32 rows x 72 units are 9216 bytes of scores a token: 256 MB up to 29127 tokens, whole tiles of 64 up to 29120."""
    x = Batch([0] * 9, 30008, hq=32, hkv=8, drafts=8, block=128, pages=235 * 9)
    size = B.sparse_attn_weigh_workspace_size(x.params(n_tokens=30000))
    room = torch.full((size + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    ws = room[:size]
    B.sparse_attn_workspace_init(ws[:256])
    for tokens in (29120, 29121, 2000):
        n = tokens - 8
        x.lens = [n, 5, 0, n, 300, 70, 0, 1000, n - 1]
        p = x.params(n_tokens=n)
        assert B.sparse_attn_weigh_workspace_size(x.params(n_tokens=n, capacity_tokens=tokens)) <= size
        out, w = x.call(p, ws)
        for b in (0, 4, 8):
            x.check(out, w, [b])
        assert (room[size:] == 0xAB).all()


# more than 32 query rows and more than 608 tiles: the tensor-core kernels
TENSOR = {
    "rows_36": Case(batch=4, drafts=9, hq=32, hkv=8, lens=(700, 650, 640, 701), context=701, block=64),
    "rows_40": Case(batch=4, drafts=10, hq=32, hkv=8, lens=(700, 0, 640, 1), context=700),
    "units": Case(batch=40, drafts=9, hq=32, hkv=8, lens=tuple(3 * i for i in range(40)), context=130, block=32),
}


@pytest.mark.parametrize("scale", [0.0, 0.02, 3.0, 1e4])
@pytest.mark.parametrize("name", TENSOR)
def test_tensor_cores_against_64_bits(name, scale):
    run(TENSOR[name], old=0.1, scale=scale)


def test_pages_out_of_range_weigh_nothing_on_the_tensor_cores():
    c = TENSOR["rows_40"]
    table = c.block_table()
    pools = [x.cuda() for x in c.fill(c.pools(empty=0.0), table)]
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim).cuda()
    p = c.params()
    table[0, 1], table[2, 0] = c.pages, -1
    ws = fresh(B.sparse_attn_weigh_workspace_size(p))
    out = torch.zeros(c.batch, c.drafts, c.hq, c.dim, device="cuda")
    w = torch.zeros(c.batch, c.hkv, c.nb_cap * c.block, device="cuda")
    B.sparse_attn_weigh_decode(p, q, *pools, table.cuda(), w, out, ws, seq_lens=int32(c.all_lens))
    assert B.sparse_attn_get_device_error(ws) == B.ERR_PAGE
    assert (w[0, :, c.block:2 * c.block] == 0).all() and (w[2, :, :c.block] == 0).all() and (w[0, :, :c.block] > 0).all()
    assert out.isfinite().all() and w.isfinite().all()
