"""Eviction by accumulated weight: kept tokens, their rows, weights and box bit for bit."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, place
from tests.long_reference import kept_tokens

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


def weights_of(c, kind):
    w = torch.randn(c.batch, c.hkv, c.nb_cap * c.block, generator=c.gen("w")).mul(2).exp()
    if kind == "ties":
        w = torch.randint(0, 3, w.shape, generator=c.gen("w")).float()
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "signs":                                                  # zeros of both signs, negatives, infinities
        pick = torch.randint(0, 6, w.shape, generator=c.gen("w"))
        w = torch.tensor([0.0, -0.0, -1.5, 2.0, float("inf"), 1e-42])[pick]
    elif kind == "close":                                                  # keys that differ in the last bits
        w = (torch.randint(0, 50, w.shape, generator=c.gen("w")) + torch.tensor(1.0).view(torch.int32)).int().view(F32)
    elif kind == "rising":
        w = torch.arange(w.shape[-1]).float().expand_as(w).contiguous()
    return w


def run(c, keep, sinks=0, recent=0, keep_lens=None, kind="spread", box=True, lens_null=False):
    table = c.block_table()
    blocks = -(-keep // c.block)
    k_pool, v_pool = c.fill(c.pools(empty=0.5), table)
    extra = torch.full((c.batch * blocks, *k_pool.shape[1:]), 0.75, dtype=c.kv)
    k_pool, v_pool = torch.cat([k_pool, extra]), torch.cat([v_pool, extra])
    new_table = (torch.randperm(c.batch * blocks, generator=c.gen("new")) + c.pages).view(c.batch, blocks).to(torch.int32)
    p = c.params(num_pages=c.pages + c.batch * blocks)
    before = weights_of(c, kind)
    kmin = torch.full((c.batch, c.hkv, c.nb_cap, c.dim), 7.0, dtype=c.kv)
    kmax = torch.full_like(kmin, -7.0)
    ids = torch.full((c.batch, c.hkv, keep), -9, dtype=torch.int32)
    ws = workspace(B.sparse_attn_evict_workspace_size(p, keep))
    w, gk, gv, lo, hi, gids = (x.cuda() for x in (before, k_pool, v_pool, kmin, kmax, ids))
    new_lens = int32([-3] * c.batch)
    B.sparse_attn_evict_tokens(p, keep, sinks, recent, w, gk, gv, table.cuda(), new_table.cuda(), gids, new_lens, ws,
                               seq_lens=None if lens_null else int32(c.all_lens),
                               keep_lens=None if keep_lens is None else int32(keep_lens),
                               kmin=lo if box else None, kmax=hi if box else None)
    assert B.sparse_attn_get_device_error(ws) == 0
    want_w, lens = before.clone(), []
    for b, n in enumerate(c.all_lens):
        k = keep if keep_lens is None else keep_lens[b]
        if n < 0 or k < 0:
            lens.append(n)
            continue
        lens.append(min(n, k))
        for h in range(c.hkv):
            t = torch.tensor(kept_tokens(before[b, h].tolist(), n, k, sinks, recent), dtype=torch.long)
            m = len(t)
            assert m == min(n, k)
            i = torch.arange(m)
            sp, so = place(c, table, b, t)
            dp = new_table[b].long()[i // c.block]
            for pool in (k_pool, v_pool):
                pool[dp, h, i % c.block] = pool[sp, h, so]
            want_w[b, h, :m] = before[b, h, t]
            ids[b, h, :m] = t.to(torch.int32)
            for j in range(-(-m // c.block)) if box else ():
                rows = k_pool[dp[j * c.block], h, : min(c.block, m - j * c.block)]
                kmin[b, h, j], kmax[b, h, j] = rows.amin(0), rows.amax(0)
    assert new_lens.tolist() == lens
    assert torch.equal(gids.cpu(), ids)
    assert torch.equal(gk.cpu(), k_pool) and torch.equal(gv.cpu(), v_pool)
    assert torch.equal(w.cpu(), want_w)
    assert torch.equal(lo.cpu(), kmin) and torch.equal(hi.cpu(), kmax)


CASES = {
    "one": (Case(batch=1, lens=(300,)), 100, dict(sinks=4, recent=20)),
    "keep_one": (Case(batch=1, lens=(300,)), 1, {}),
    "drop_one": (Case(batch=2, lens=(300, 300)), 299, dict(sinks=4, recent=20)),
    "all_fit": (Case(batch=3, lens=(300, 0, 1)), 300, dict(sinks=4, recent=20)),
    "ragged": (Case(batch=5, lens=(300, 0, 101, 100, 99)), 100, dict(sinks=1)),
    "inactive": (Case(batch=4, lens=(300, -1, 101, 250)), 100, dict(keep_lens=[50, 100, -1, 0])),
    "budgets": (Case(batch=4, lens=(300, 200, 101, 250)), 128, dict(keep_lens=[128, 24, 101, 25], sinks=4, recent=20)),
    "only_sinks_and_recent": (Case(batch=2, lens=(300, 200)), 24, dict(sinks=4, recent=20)),
    "ties": (Case(batch=3, lens=(300, 299, 150)), 77, dict(kind="ties", sinks=2, recent=9)),
    "equal": (Case(batch=2, lens=(300, 299)), 77, dict(kind="equal", recent=9)),
    "signs": (Case(batch=3, lens=(300, 299, 150)), 120, dict(kind="signs", sinks=2, recent=9)),
    "close": (Case(batch=3, lens=(300, 299, 150)), 77, dict(kind="close")),
    "rising": (Case(batch=2, lens=(300, 299)), 77, dict(kind="rising", sinks=3)),
    "block_8": (Case(batch=2, lens=(300, 299), block=8), 77, dict(sinks=3)),
    "block_128": (Case(batch=2, lens=(700, 299), context=700, block=128), 277, dict(sinks=3)),
    "dim_64": (Case(batch=2, lens=(300, 299), dim=64, block=16), 77, dict(sinks=3)),
    "fp32": (Case(batch=2, lens=(300, 299), dtype=F32, kv=F32), 130, dict(sinks=3)),
    "fp32_block_128": (Case(batch=2, lens=(300, 299), dtype=F32, kv=F32, block=128), 130, dict(sinks=3)),
    "fp32_block_64": (Case(batch=2, lens=(300, 299), dtype=F32, kv=F32, block=64), 130, dict(sinks=3)),
    "long_rows_of_runs": (Case(batch=3, lens=(4000, 3900, 4000), context=4000, hq=16, hkv=16, dim=64, block=64), 3500, {}),
    "fp32_64_block_128": (Case(batch=2, lens=(300, 299), dtype=F32, kv=F32, dim=64, block=128), 130, dict(sinks=3)),
    "no_box": (Case(batch=2, lens=(300, 299)), 77, dict(box=False)),
    "heads": (Case(batch=3, lens=(300, 299, 280), hq=8, hkv=8, dim=64), 77, {}),
    "one_cta": (Case(batch=1, lens=(5001,), context=5001, hq=1, hkv=1, dim=64), 1500, dict(sinks=4, recent=64)),
    "two_ctas": (Case(batch=60, lens=(17001,) + (-1,) * 59, context=17001, hq=1, hkv=1, dim=64, block=128), 1500,
                 dict(sinks=4, recent=64)),
    "four_ctas": (Case(batch=1, lens=(17001,), context=17001, hq=1, hkv=1, dim=64, block=64), 1500, dict(kind="ties")),
    "eight_ctas": (Case(batch=1, lens=(40001,), context=40001, hq=1, hkv=1, dim=64, block=64), 5000, dict(kind="ties")),
    "eight_ctas_short": (Case(batch=2, lens=(40000, 700), context=40001, hq=1, hkv=1, dim=64, block=64), 500, {}),
    "many_units": (Case(batch=90, lens=tuple(200 + 3 * i for i in range(90)), context=500, hq=2, hkv=2, dim=64), 150, {}),
}


@pytest.mark.parametrize("name", CASES)
def test_against_sorting(name):
    c, keep, kw = CASES[name]
    run(c, keep, **kw)


def test_every_length_the_same():
    run(Case(batch=3, context=200), 60, recent=5, lens_null=True)


@pytest.mark.parametrize("kind", ["spread", "ties"])
def test_keys_past_shared_memory(kind):
    """More weights than a CTA keeps at hand, with a unit for every SM."""
    units, n, keep = 160, 60001, 300
    g = torch.Generator(device="cuda").manual_seed(5)
    p = B.make_params(1, units, units, 64, n, 128, 600, 0, 1)
    nb = -(-n // 128)
    w = torch.rand(1, units, nb * 128, generator=g, device="cuda")
    if kind == "ties":
        w = (w * 5).floor()
    pools = [torch.zeros(600, units, 128, 64, dtype=BF, device="cuda") for _ in range(2)]
    table = torch.arange(nb, dtype=torch.int32, device="cuda").view(1, -1)
    new = torch.arange(nb, nb + 3, dtype=torch.int32, device="cuda").view(1, -1)
    ids, lens = torch.zeros(1, units, keep, dtype=torch.int32, device="cuda"), int32([0])
    ws = workspace(B.sparse_attn_evict_workspace_size(p, keep))
    want = w[:, :, :n].argsort(dim=-1, descending=True, stable=True)[..., :keep].sort(dim=-1).values
    B.sparse_attn_evict_tokens(p, keep, 0, 0, w, *pools, table, new, ids, lens, ws)
    assert B.sparse_attn_get_device_error(ws) == 0 and lens.tolist() == [keep]
    assert torch.equal(ids.long(), want)


def small():
    c = Case(batch=2, lens=(300, 299))
    table = c.block_table()
    pools = [torch.zeros(c.pages + 8, c.hkv, c.block, c.dim, dtype=BF, device="cuda") for _ in range(2)]
    new = torch.arange(c.pages, c.pages + 8, dtype=torch.int32).view(2, 4)
    return c, c.params(num_pages=c.pages + 8), table, pools, new


def call(c, p, table, pools, new, lens=None, keep_lens=None):
    w = weights_of(c, "spread").cuda()
    ids, new_lens = torch.full((2, c.hkv, 100), -9, dtype=torch.int32, device="cuda"), int32([0, 0])
    ws = workspace(B.sparse_attn_evict_workspace_size(p, 100))
    B.sparse_attn_evict_tokens(p, 100, 4, 20, w, *pools, table.cuda(), new.cuda(), ids, new_lens, ws,
                               seq_lens=int32(c.all_lens if lens is None else lens),
                               keep_lens=None if keep_lens is None else int32(keep_lens))
    return B.sparse_attn_get_device_error(ws), ids, new_lens.tolist()


def test_bad_pages_are_reported():
    c, p, table, pools, new = small()
    for which, value in (("table", -1), ("table", c.pages + 8), ("new", -1), ("new", 2**31 - 1)):
        t, n = table.clone(), new.clone()
        (t if which == "table" else n)[1, 0] = value
        flags, _, lens = call(c, p, t, pools, n)
        assert flags == B.ERR_PAGE and lens == [100, 100]


def test_rows_of_good_pages_move_past_a_bad_one():
    c, p, table, pools, new = small()
    host = [torch.randn(x.shape, generator=c.gen("rows")).to(BF) for x in pools]
    pools = [x.cuda() for x in host]
    bad = table.clone()
    bad[0, 2], bad[1, 0] = c.pages + 100, -5
    flags, ids, lens = call(c, p, bad, pools, new)
    assert flags == B.ERR_PAGE and lens == [100, 100]
    for b in range(2):
        for h in range(c.hkv):
            t = ids[b, h].cpu().long()
            good = (bad[b].long()[t // c.block] >= 0) & (bad[b].long()[t // c.block] < c.pages)
            assert good.any() and not good.all()
            i = torch.arange(100)
            for pool, before in zip(pools, host):
                want = before[bad[b].long()[t[good] // c.block], h, t[good] % c.block]
                assert torch.equal(pool.cpu()[new[b].long()[i[good] // c.block], h, i[good] % c.block], want)
                old = before[new[b].long()[i[~good] // c.block], h, i[~good] % c.block]
                assert torch.equal(pool.cpu()[new[b].long()[i[~good] // c.block], h, i[~good] % c.block], old)


def test_bad_lengths_are_reported_and_leave_the_sequence_alone():
    c, p, table, pools, new = small()
    for lens, keep_lens in (((301, 299), None), ((-2, 299), None), ((300, 299), [23, 100]), ((300, 299), [101, 100]),
                            ((300, 299), [-5, 100])):
        flags, ids, got = call(c, p, table, pools, new, lens, keep_lens)
        assert flags == B.ERR_LENGTH and got == [lens[0], 100] and (ids[0] == -9).all()
