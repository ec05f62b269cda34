"""Attention of a batch whose groups of sequences share prefixes, against 64 bits."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, pack_mask, place, random_tree
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


def share(c, table, pools, cuts, prefixes):
    """Whole blocks of a prefix become the first holder's pages, the block that it ends in a copy."""
    table = table.clone()
    for g, n in enumerate(prefixes):
        members = [b for b in range(cuts[g], cuts[g + 1]) if c.all_lens[b] >= n]
        for b in members[1:]:
            whole = n // c.block
            table[b, :whole] = table[members[0], :whole]
            if n % c.block:
                src, dst = table[members[0], whole], table[b, whole]
                for pool in pools:
                    pool[dst, :, : n % c.block] = pool[src, :, : n % c.block]
    return table


def run(c, cuts, prefixes, see=None, scale=0.0, lens_null=False):
    own_table = c.block_table()
    pools = c.fill(c.pools(), own_table)
    table = share(c, own_table, pools, cuts, prefixes)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    p = c.params(softmax_scale=scale)
    ws = workspace(B.sparse_attn_shared_workspace_size(p, len(prefixes)))
    out = torch.full((c.batch, c.drafts, c.hq, c.dim), 5.0, device="cuda")
    args = (p, q.cuda(), pools[0].cuda(), pools[1].cuda(), table.cuda(), int32(cuts), int32(prefixes))
    kw = dict(seq_lens=None if lens_null else int32(c.all_lens), tree_mask=None if see is None else pack_mask(see).cuda())
    B.sparse_attn_shared_decode(*args, out, ws, **kw)
    assert B.sparse_attn_get_device_error(ws) == 0
    exact, bound, _, _ = attention_exact(c, q, pools, table, see, scale=scale or None)
    got = out.cpu().double()
    for b, n in enumerate(c.all_lens):
        if n < 0:
            assert (got[b] == 5.0).all()
        else:
            err = (got[b] - exact[b]).abs()
            assert (err <= bound[b]).all(), f"sequence {b}: {err.max():.3g}, {(err / bound[b]).max():.3g} of the bound"
    again = torch.full_like(out, 5.0)                                      # the same bits on the used workspace
    B.sparse_attn_shared_decode(*args, again, ws, **kw)
    assert torch.equal(out, again)
    return out


CASES = {
    "samples": (Case(batch=4, drafts=1, lens=(150, 131, 170, 140), context=170), [0, 4], [130]),
    "one_sequence": (Case(batch=1, drafts=1, lens=(150,), context=150), [0, 1], [70]),
    "nothing_shared": (Case(batch=3, drafts=2, lens=(150, 0, 40), context=150), [0, 3], [0]),
    "nothing_else": (Case(batch=3, drafts=1, lens=(128, 128, 128), context=128), [0, 3], [128]),
    "one_shared_token": (Case(batch=3, drafts=3, lens=(150, 1, 40), context=150), [0, 3], [1]),
    "groups": (Case(batch=7, drafts=2, lens=(150, 131, 70, 90, 64, 300, 200), context=300), [0, 2, 5, 6, 7],
               [130, 64, 299, 0]),
    "empty_groups_and_loners": (Case(batch=6, drafts=1, lens=(50, 131, 70, 90, 64, 30), context=300), [1, 1, 4, 4, 5],
                                [17, 64, 200, 33]),
    "inactive": (Case(batch=6, drafts=1, lens=(-1, 131, 70, -1, 64, -1), context=300), [0, 3, 5, 6], [64, 40, 99]),
    "many_members": (Case(batch=40, drafts=1, lens=tuple(200 + 3 * i for i in range(40)), context=330, hq=16, hkv=2),
                     [0, 33, 40], [200, 299]),
    "drafts": (Case(batch=5, drafts=9, lens=(250, 231, 270, 90, 64), context=300), [0, 3, 5], [222, 64]),
    "wide": (Case(batch=3, drafts=70, lens=(250, 231, 270), context=300, hq=4, hkv=1), [0, 3], [222]),
    "block_8": (Case(batch=4, drafts=3, lens=(150, 131, 170, 140), context=170, block=8), [0, 4], [131]),
    "block_128": (Case(batch=4, drafts=3, lens=(550, 531, 570, 640), context=640, block=128), [0, 2, 4], [400, 513]),
    "dim_64": (Case(batch=4, drafts=3, lens=(550, 531, 570, 640), context=640, dim=64, block=16), [0, 2, 4], [400, 513]),
    "heads": (Case(batch=4, drafts=1, lens=(550, 531, 570, 640), context=640, hq=8, hkv=8), [0, 4], [512]),
    "one_head": (Case(batch=4, drafts=1, lens=(550, 531, 570, 640), context=640, hq=1, hkv=1), [0, 4], [512]),
    "fp32": (Case(batch=5, drafts=2, lens=(250, 231, 270, 90, 64), context=300, dtype=F32, kv=F32), [0, 3, 5], [222, 64]),
    "fp32_64": (Case(batch=9, drafts=5, lens=(250, 231, 270, 90, 64, 70, 80, 90, 99), context=300, dtype=F32, kv=F32, dim=64),
                [0, 3, 9], [222, 64]),
    "fp32_queries": (Case(batch=9, drafts=2, lens=(250, 231, 270, 90, 64, 70, 80, 90, 99), context=300, dtype=F32),
                     [0, 3, 9], [222, 64]),
    "fp32_queries_64": (Case(batch=3, drafts=1, lens=(250, 231, 270), context=300, dtype=F32, dim=64), [0, 3], [222]),
    "bf16_queries_fp32_cache": (Case(batch=3, drafts=1, lens=(250, 231, 270), context=300, kv=F32, dim=64), [0, 3], [222]),
    "long": (Case(batch=12, drafts=1, lens=tuple(5000 + 37 * i for i in range(12)), context=5500, block=64), [0, 12], [4999]),
    "long_small_rows": (Case(batch=2, drafts=1, lens=(9000, 8000), context=9000, block=64, hq=2), [0, 2], [7990]),
}


def big(batch, **kw):
    """Enough tiles for the tensor-core kernel."""
    lens = tuple(2500 + 3 * (i % 30) for i in range(batch))
    return Case(**{**dict(batch=batch, drafts=1, lens=lens, context=2600, hq=32, hkv=8, block=64), **kw})


TENSOR = {
    "rows_20": (big(5), [0, 5], [2500]),
    "rows_32": (big(8), [0, 8], [2499]),
    "rows_64": (big(16), [0, 16], [2433]),
    "rows_132": (big(33), [0, 33], [2500]),
    "rows_64_dim_64": (big(8, hkv=4, dim=64), [0, 8], [2300]),
    "rows_80_dim_64_block_16": (big(20, dim=64, block=16), [0, 20], [2391]),
    "rows_24_dim_64_block_8": (big(6, dim=64, block=8), [0, 6], [2391]),
    "rows_36_block_128": (big(9, block=128), [0, 9], [2391]),
    "groups": (big(40), [0, 20, 21, 39], [2500, 77, 1000]),
    "groups_of_one": (big(40, hkv=8, hq=64, drafts=3), list(range(41)), [2300 - 50 * i for i in range(40)]),
    "own_rows_36": (big(5, drafts=9), [0, 5], [1200]),
    "own_rows_72": (big(5, drafts=18, hq=16, hkv=4), [0, 3, 5], [200, 2480]),
    "own_rows_160_dim_64": (big(5, drafts=40, hq=16, hkv=4, dim=64, block=32), [0, 3, 5], [200, 2480]),
    "inactive": (big(12, lens=(-1, 2500, 2510, -1) * 3), [0, 9, 12], [2500, 100]),
}


@pytest.mark.parametrize("name", CASES)
def test_against_64_bits(name):
    run(*CASES[name])


@pytest.mark.parametrize("name", TENSOR)
def test_tensor_cores_against_64_bits(name):
    run(*TENSOR[name])


@pytest.mark.parametrize("name", ["own_rows_36", "own_rows_72", "own_rows_160_dim_64", "groups_of_one"])
def test_tensor_core_trees(name):
    c, cuts, prefixes = TENSOR[name]
    see = random_tree(c)
    see[:, 0, :] = False
    run(c, cuts, prefixes, see)


@pytest.mark.parametrize("name", ["samples", "rows_32", "rows_64", "rows_132", "own_rows_36"])
@pytest.mark.parametrize("scale", [2.0 ** 20, 2.0 ** 26, 1.9 * 2.0 ** 27, 2.0 ** 40])
def test_large_scores(name, scale):
    """Whole-numbered scores, exact in every order: softmax over them times a large factor is the mean of the
    values at the largest one, whichever launch has met it.  The mean of n values: n additions of U of the sum of
    their magnitudes and a division, or with weights equal but for exp2's 2^-21, that."""
    c, cuts, prefixes = {**CASES, **TENSOR}[name]
    own_table = c.block_table()
    pools = c.fill(c.pools(), own_table)
    g = c.gen("whole")
    pools = (torch.where(pools[0].isnan(), pools[0], torch.randint(-1, 2, pools[0].shape, generator=g).to(c.kv)), pools[1])
    table = share(c, own_table, pools, cuts, prefixes)
    q = torch.randint(-1, 2, (c.batch, c.drafts, c.hq, c.dim), generator=g).to(c.dtype)
    p = c.params(softmax_scale=scale)
    ws = workspace(B.sparse_attn_shared_workspace_size(p, len(prefixes)))
    out = torch.empty(c.batch, c.drafts, c.hq, c.dim, device="cuda")
    B.sparse_attn_shared_decode(p, q.cuda(), pools[0].cuda(), pools[1].cuda(), table.cuda(), int32(cuts), int32(prefixes), out,
                                ws, seq_lens=int32(c.all_lens))
    got = out.cpu().double()
    for b, n in enumerate(c.all_lens):
        for i in range(c.drafts):
            t = torch.arange(n + i + 1)
            page, off = place(c, table, b, t)
            for h in range(c.hq):
                kvh = h // (c.hq // c.hkv)
                score = pools[0][page, kvh, off].double() @ q[b, i, h].double()
                v = pools[1][page, kvh, off].double()[score == score.max()]
                bound = (len(v) * 2.0 ** -24 + 2.0 ** -20) * v.abs().mean(0)
                assert ((got[b, i, h] - v.mean(0)).abs() <= bound).all(), (b, i, h)


@pytest.mark.parametrize("name", ["drafts", "groups", "wide", "fp32_64", "dim_64"])
def test_trees(name):
    c, cuts, prefixes = CASES[name]
    see = random_tree(c)
    see[:, 0, :] = False                                                   # a draft that sees the context alone
    run(c, cuts, prefixes, see)


def test_every_length_the_same():
    run(Case(batch=3, drafts=2, context=200), [0, 3], [160], lens_null=True)


def test_rows_that_see_nothing_are_zero():
    c = Case(batch=2, drafts=3, lens=(0, 40), context=40)
    see = torch.zeros(2, 3, 3, dtype=torch.bool)
    out = run(c, [0, 2], [0], see)
    assert (out[0] == 0).all() and (out[1] != 0).any()


@pytest.mark.parametrize("scale", [0.02, 3.0, 1e4])
def test_scales(scale):
    run(*CASES["groups"], scale=scale)


def test_drafts_that_hold_anything_reach_only_those_that_see_them():
    c, cuts, prefixes = CASES["drafts"]
    own_table = c.block_table()
    pools = c.fill(c.pools(), own_table)
    table = share(c, own_table, pools, cuts, prefixes)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    see = random_tree(c)
    see[:, :, 4] = False
    see[:, 4, 4] = True                                                    # a leaf
    for b, n in enumerate(c.all_lens):
        pg, off = place(c, table, b, torch.tensor([n + 4]))
        pools[0][pg, :, off], pools[1][pg, :, off] = float("nan"), float("inf")
    p = c.params()
    ws = workspace(B.sparse_attn_shared_workspace_size(p, len(prefixes)))
    out = torch.empty(c.batch, c.drafts, c.hq, c.dim, device="cuda")
    B.sparse_attn_shared_decode(p, q.cuda(), pools[0].cuda(), pools[1].cuda(), table.cuda(), int32(cuts), int32(prefixes), out,
                                ws, seq_lens=int32(c.all_lens), tree_mask=pack_mask(see).cuda())
    clean = see.clone()
    clean[:, 4, 4] = False
    exact, bound, _, _ = attention_exact(c, q, pools, table, clean)
    got = out.cpu().double()
    others = [i for i in range(c.drafts) if i != 4]
    assert ((got - exact).abs() <= bound)[:, others].all()
    assert got[:, 4].isnan().all()


def errors_of(c, cuts, prefixes, lens=None):
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    table = share(c, table, pools, [0, c.batch], [min(c.all_lens)])
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim).cuda()
    p = c.params()
    ws = workspace(B.sparse_attn_shared_workspace_size(p, len(prefixes)))
    out = torch.full((c.batch, c.drafts, c.hq, c.dim), 5.0, device="cuda")
    B.sparse_attn_shared_decode(p, q, pools[0].cuda(), pools[1].cuda(), table.cuda(), int32(cuts), int32(prefixes), out, ws,
                                seq_lens=int32(c.all_lens if lens is None else lens))
    return B.sparse_attn_get_device_error(ws), out


def test_bad_lengths_and_groups_are_reported():
    c = Case(batch=4, drafts=1, lens=(150, 131, 170, 140), context=170)
    flags, out = errors_of(c, [0, 4], [140])                               # more than the second one holds
    assert flags == B.ERR_LENGTH and (out[1] == 5.0).all() and (out[[0, 2, 3]] != 5.0).all()
    for cuts, prefixes, lens in (([0, 4], [-1], None), ([0, 4], [171], None), ([0, 5], [20], None), ([-2, 4], [20], None),
                                 ([0, 3, 2], [20, 20], None), ([0, 4], [20], [150, 171, 160, 140]),
                                 ([0, 4], [20], [150, -7, 160, 140])):
        assert errors_of(c, cuts, prefixes, lens)[0] == B.ERR_LENGTH, (cuts, prefixes, lens)


def test_pages_out_of_range_are_reported():
    c = Case(batch=2, drafts=1, lens=(150, 131), context=170)
    table = c.block_table()
    pools = [x.cuda() for x in c.fill(c.pools(empty=0.0), table)]
    q = c.normal("q", 2, 1, c.hq, c.dim).cuda()
    p = c.params()
    for at, value in ((1, -1), (1, c.pages), (4, c.pages + 7), (4, 2**31 - 1)):
        bad = table.clone()
        bad[0, at] = value
        ws = workspace(B.sparse_attn_shared_workspace_size(p, 1))
        out = torch.empty(2, 1, c.hq, c.dim, device="cuda")
        B.sparse_attn_shared_decode(p, q, *pools, bad.cuda(), int32([0, 2]), int32([96]), out, ws, seq_lens=int32(c.all_lens))
        assert B.sparse_attn_get_device_error(ws) == B.ERR_PAGE
