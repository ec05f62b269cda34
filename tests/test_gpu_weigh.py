"""Attention that adds up the weight of every cached token, against 64 bits."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case
from tests.long_reference import attention_exact

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def workspace(size):
    ws = torch.full((size,), 0xAB, dtype=torch.uint8, device="cuda")       # only the header is zeroed
    B.sparse_attn_workspace_init(ws[:256])
    return ws


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(c, old=0.0, scale=0.0, lens_null=False):
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    p = c.params(softmax_scale=scale)
    ws = workspace(B.sparse_attn_weigh_workspace_size(p))
    before = old * torch.rand(c.batch, c.hkv, c.nb_cap * c.block, generator=c.gen("w"))
    for b, n in enumerate(c.all_lens):
        before[b, :, max(0, n):] = float("nan")                            # nothing is read there
    out = torch.full((c.batch, c.drafts, c.hq, c.dim), 5.0, device="cuda")
    w = before.cuda()
    gpu = (q.cuda(), pools[0].cuda(), pools[1].cuda(), table.cuda())
    lens = None if lens_null else int32(c.all_lens)
    B.sparse_attn_weigh_decode(p, *gpu, w, out, ws, seq_lens=lens)
    assert B.sparse_attn_get_device_error(ws) == 0
    exact, bound, w_exact, w_bound = attention_exact(c, q, pools, table, scale=scale or None, weights=before)
    got, got_w = out.cpu().double(), w.cpu().double()
    for b, n in enumerate(c.all_lens):
        if n < 0:
            assert (got[b] == 5.0).all() and got_w[b].isnan().all()
            continue
        err = (got[b] - exact[b]).abs()
        assert (err <= bound[b]).all(), f"sequence {b}: {err.max():.3g}, {(err / bound[b]).max():.3g} of the bound"
        m = n + c.drafts
        err = (got_w[b, :, :m] - w_exact[b, :, :m]).abs()
        assert (err <= w_bound[b, :, :m]).all(), f"weights of {b}: {err.max():.3g}, {(err / w_bound[b, :, :m]).max():.3g}"
        assert got_w[b, :, m:].isnan().all()                               # behind the new tokens: as it was
    again, w2 = torch.full_like(out, 5.0), before.cuda()
    B.sparse_attn_weigh_decode(p, *gpu, w2, again, ws, seq_lens=lens)
    assert torch.equal(out, again) and torch.equal(w.nan_to_num(-1.0), w2.nan_to_num(-1.0))
    return out, w


CASES = {
    "one_token": Case(batch=1, drafts=1, lens=(300,)),
    "first_token": Case(batch=2, drafts=1, lens=(0, 1)),
    "batch": Case(batch=5, drafts=1, lens=(300, 0, -1, 33, 64)),
    "odd_block_ends": Case(batch=3, drafts=1, lens=(63, 64, 65), block=8),
    "window": Case(batch=3, drafts=33, lens=(300, 0, 65)),
    "prompt": Case(batch=2, drafts=90, lens=(0, 10), hq=16, hkv=2),
    "block_128": Case(batch=2, drafts=3, lens=(300, 129), block=128),
    "dim_64": Case(batch=2, drafts=3, lens=(300, 129), dim=64, block=16),
    "dim_64_rows": Case(batch=2, drafts=40, lens=(300, 129), dim=64, block=16),
    "heads": Case(batch=2, drafts=1, lens=(300, 129), hq=8, hkv=8),
    "group_of_8": Case(batch=2, drafts=5, lens=(300, 129), hq=8, hkv=1),
    "one_head": Case(batch=2, drafts=1, lens=(300, 129), hq=1, hkv=1),
    "fp32": Case(batch=2, drafts=1, lens=(300, 129), dtype=F32, kv=F32),
    "fp32_rows": Case(batch=2, drafts=20, lens=(300, 129), dtype=F32, kv=F32, dim=64),
    "fp32_queries": Case(batch=2, drafts=1, lens=(300, 129), dtype=F32),
    "fp32_queries_rows": Case(batch=2, drafts=20, lens=(300, 129), dtype=F32),
    "bf16_queries_fp32_cache": Case(batch=2, drafts=2, lens=(300, 129), kv=F32, dim=64),
    "long": Case(batch=2, drafts=1, lens=(9000, 6001), context=9000, block=64, hq=4, hkv=1),
    "long_window": Case(batch=2, drafts=32, lens=(3000, 2001), context=3500, block=64, hq=4, hkv=1),
    "many_units": Case(batch=50, drafts=1, lens=tuple(7 * i for i in range(50)), context=400, hq=16, hkv=8, dim=64),
}

# many tiles, with more than 32 query rows for the tensor-core kernels
TENSOR = {
    "rows_20": Case(batch=4, drafts=5, hq=32, hkv=8, lens=(700, 650, 640, 701), context=701, block=64),
    "rows_32": Case(batch=4, drafts=8, hq=32, hkv=8, lens=(700, 0, 640, 1), context=700),
    "rows_128": Case(batch=2, drafts=32, hq=32, hkv=8, lens=(400, 383), context=400, block=128),
    "rows_264": Case(batch=3, drafts=33, hq=16, hkv=2, lens=(400, 127, 128), context=400, block=64),
    "rows_560": Case(batch=4, drafts=70, hq=8, hkv=1, lens=(400, -1, 3, 256), context=400, block=16),
    "dim_64": Case(batch=4, drafts=9, hq=32, hkv=8, lens=(700, 650, 640, 701), context=701, dim=64, block=8),
    "dim_64_rows_160": Case(batch=4, drafts=20, hq=32, hkv=4, lens=(400, 383, 0, 200), context=400, dim=64, block=128),
    "units": Case(batch=40, drafts=5, hq=32, hkv=8, lens=tuple(3 * i for i in range(40)), context=130, block=32),
}


@pytest.mark.parametrize("name", CASES)
def test_against_64_bits(name):
    run(CASES[name])


@pytest.mark.parametrize("name", TENSOR)
def test_many_rows_against_64_bits(name):
    run(TENSOR[name], old=0.1)


def test_one_workspace_as_the_context_grows():
    """Its size, of the capacity, serves every length: short contexts keep their scores, long ones do not."""
    for n in (10, 300, 700, 1500):
        c = Case(batch=4, drafts=8, hq=32, hkv=8, context=n, room=1600 - n)
        small = B.sparse_attn_weigh_workspace_size(c.params(capacity_tokens=n + 8))
        assert small <= B.sparse_attn_weigh_workspace_size(c.params())
    run(Case(batch=4, drafts=8, hq=32, hkv=8, context=250, room=1000))


def test_weights_add_up():
    """Every row gives one, and what was there before stays in."""
    c = CASES["window"]
    _, w = run(c)
    for b, n in enumerate(c.all_lens):
        total = w[b, :, : n + c.drafts].double().sum(-1).cpu()
        assert ((total - c.drafts * c.hq // c.hkv).abs() < 1e-3).all()
    run(c, old=3.0)


def test_every_length_the_same():
    run(Case(batch=3, drafts=2, context=200), lens_null=True)


@pytest.mark.parametrize("scale", [0.02, 3.0, 1e4])
@pytest.mark.parametrize("name", ["batch", "window", "rows_20", "rows_128"])
def test_scales(name, scale):
    run({**CASES, **TENSOR}[name], scale=scale)


@pytest.mark.parametrize("name", ["window", "rows_32", "rows_264"])
def test_pages_out_of_range_are_reported_and_weigh_nothing(name):
    c = {**CASES, **TENSOR}[name]
    table = c.block_table()
    pools = [x.cuda() for x in c.fill(c.pools(empty=0.0), table)]
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim).cuda()
    p = c.params()
    table[0, 1], table[2, 0] = c.pages, -1
    ws = workspace(B.sparse_attn_weigh_workspace_size(p))
    out = torch.zeros(c.batch, c.drafts, c.hq, c.dim, device="cuda")
    w = torch.zeros(c.batch, c.hkv, c.nb_cap * c.block, device="cuda")
    B.sparse_attn_weigh_decode(p, q, *pools, table.cuda(), w, out, ws, seq_lens=int32(c.all_lens))
    assert B.sparse_attn_get_device_error(ws) == B.ERR_PAGE
    assert (w[0, :, c.block:2 * c.block] == 0).all() and (w[2, :, :c.block] == 0).all() and (w[0, :, :c.block] > 0).all()
    assert out.isfinite().all() and w.isfinite().all()


def test_bad_lengths_are_reported():
    c = Case(batch=3, drafts=1, lens=(150, 131, 170), context=170)
    table = c.block_table()
    pools = [x.cuda() for x in c.fill(c.pools(empty=0.0), table)]
    q = c.normal("q", 3, 1, c.hq, c.dim).cuda()
    p = c.params()
    ws = workspace(B.sparse_attn_weigh_workspace_size(p))
    out, w = torch.full((3, 1, c.hq, c.dim), 5.0, device="cuda"), torch.zeros(3, c.hkv, c.nb_cap * c.block, device="cuda")
    B.sparse_attn_weigh_decode(p, q, *pools, table.cuda(), w, out, ws, seq_lens=int32([150, 171, -7]))
    assert B.sparse_attn_get_device_error(ws) == B.ERR_LENGTH
    assert (out[1:] == 5.0).all() and (w[1:] == 0).all() and (w[0] != 0).any()


def test_long_contexts_of_some_rows_keep_no_scores():
    """32 rows over so many tokens that their scores would be over 256 MB are computed again; the rows' weights add up
    to one, and sampled units agree with 64 bits."""
    c = Case(batch=9, drafts=8, hq=32, hkv=8, context=33001, block=128)
    p = c.params(num_pages=c.batch * c.nb_cap)
    size = B.sparse_attn_weigh_workspace_size(p)
    assert 256 << 20 < size < 400 << 20
    assert size >= B.sparse_attn_weigh_workspace_size(c.params(n_tokens=2000, capacity_tokens=2008))
    g = torch.Generator(device="cuda").manual_seed(1)
    pools = [torch.randn(c.batch * c.nb_cap, c.hkv, c.block, c.dim, generator=g, device="cuda", dtype=BF) for _ in range(2)]
    table = torch.randperm(c.batch * c.nb_cap, generator=g, device="cuda").to(torch.int32).view(c.batch, -1)
    q = torch.randn(c.batch, c.drafts, c.hq, c.dim, generator=g, device="cuda", dtype=BF)
    ws = workspace(size)
    w, out = torch.zeros(c.batch, c.hkv, c.nb_cap * c.block, device="cuda"), torch.empty(q.shape, device="cuda")
    B.sparse_attn_weigh_decode(p, q, *pools, table, w, out, ws)
    assert B.sparse_attn_get_device_error(ws) == 0
    assert ((w.double().sum(-1) - 32).abs() < 1e-3).all()
    n = c.context + c.drafts
    for b, h in ((0, 0), (4, 7), (8, 3)):
        k, v = (x[table[b].long(), h].reshape(-1, c.dim)[:n].double() for x in pools)
        s = q[b, :, 4 * h:4 * h + 4].double() @ k.t() * c.dim ** -0.5                    # [Q, G, tokens]
        late = torch.arange(n, device="cuda") > c.context + torch.arange(c.drafts, device="cuda")[:, None]
        prob = torch.softmax(s.masked_fill(late[:, None], -float("inf")), -1)
        # score errors of 2^-18 (chains of 8 steps of magnitudes up to 40), twice, and the totals' chain
        assert ((w[b, h, :n].double() - prob.sum((0, 1))).abs() <= 2.0 ** -15 * prob.sum((0, 1))).all()
        err = (out[b, :, 4 * h:4 * h + 4].double() - prob @ v).abs()
        assert (err <= 2.0 ** -15 * (prob @ v.abs())).all()
