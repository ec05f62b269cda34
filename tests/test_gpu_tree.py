"""Draft-tree attention through the C ABI against 64-bit attention.  Pools hold NaN wherever no
query may look, so a read out of place shows."""
import dataclasses

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, chain_mask, pack_mask, place, random_tree, tree_exact

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def workspace(p):
    ws = torch.empty(B.sparse_attn_tree_workspace_size(p), dtype=torch.uint8, device="cuda")
    B.sparse_attn_workspace_init(ws)
    return ws


def call(c, q, pools, table, see=None, sel=None, lens="own", ws=None, out=None, p=None, stream=None):
    p = c.params() if p is None else p
    ws = workspace(p) if ws is None else ws
    out = torch.full((c.batch, c.drafts, c.hq, c.dim), 5.0, dtype=F32, device="cuda") if out is None else out
    sl = torch.tensor(c.all_lens, dtype=torch.int32, device="cuda") if lens == "own" else lens
    ids, cnt = (None, None) if sel is None else (x.cuda() for x in sel)
    B.sparse_attn_tree_decode(p, q.cuda(), pools[0].cuda(), pools[1].cuda(), table.cuda(), out, ws, seq_lens=sl,
                              sel_ids=ids, sel_count=cnt, tree_mask=None if see is None else pack_mask(see).cuda(),
                              stream=stream)
    return out, ws


def check(c, out, exact, bound):
    for b, n in enumerate(c.all_lens):
        if n < 0:
            assert (out[b] == 5.0).all(), "an inactive sequence's rows were written"
            continue
        err = (out[b].cpu().double() - exact[b]).abs()
        assert (err <= bound[b]).all(), f"sequence {b}: off by {float((err / bound[b]).max()):.3g} times the bound"


def selection(c, width=None):
    """Random ascending selections of each unit's context blocks, counts from 0 up."""
    g = c.gen("sel")
    nb = -(-c.context // c.block)
    width = min(c.topk, nb) if width is None else width
    ids = torch.zeros(c.batch, c.hkv, max(1, width), dtype=torch.int32)
    cnt = torch.zeros(c.batch, c.hkv, dtype=torch.int32)
    for b, n in enumerate(c.all_lens):
        have = -(-max(n, 0) // c.block)
        for h in range(c.hkv):
            k = min(have, width - (b + h) % 3 if width > 2 else width)
            ids[b, h, :k] = torch.randperm(have, generator=g)[:k].sort().values.to(torch.int32)
            cnt[b, h] = k
    return ids, cnt


CASES = {
    "one_token": Case(batch=1, drafts=1, lens=(300,)),
    "one_token_alone": Case(batch=1, drafts=1, lens=(0,)),
    "one_row": Case(batch=1, hq=1, hkv=1, drafts=1, context=1, block=8),
    "few_rows": Case(drafts=3, lens=(300, 17)),
    "block_ends": Case(batch=6, drafts=5, block=32, lens=(32, 31, 27, 64, 0, 300)),
    "two_row_tiles": Case(drafts=40, lens=(300, 5), hq=16),
    "g8": Case(drafts=16, hq=16, hkv=2, lens=(250, 300)),
    "g1_d64": Case(drafts=33, hq=2, hkv=2, dim=64, block=64, lens=(129, 300)),
    "wide_masks": Case(drafts=100, hq=2, hkv=1, dim=64, block=16, lens=(299, 30)),
    "wide_g4": Case(drafts=70, hq=4, hkv=1, block=16, lens=(299, 30)),
    "bs8": Case(drafts=9, block=8, lens=(300, 61)),
    "bs128_d64": Case(drafts=9, block=128, dim=64, context=700, lens=(700, 129)),
    "longer": Case(batch=3, drafts=12, context=5000, block=64, lens=(5000, 1237, 64)),
    "many_parts": Case(batch=1, hq=4, hkv=1, drafts=17, context=40000, block=128),
    "many_entries": Case(batch=1, hq=4, hkv=1, dim=64, drafts=4, context=20000, block=8),
    "inactive": Case(batch=4, drafts=6, lens=(-1, 100, -1, 300)),
    "many_units": Case(batch=150, hq=4, hkv=2, dim=64, drafts=2, context=40, block=16, lens=tuple(i % 41 for i in range(150))),
    "fp32": Case(drafts=7, dtype=F32, kv=F32, lens=(300, 5)),
    "fp32_d64": Case(drafts=21, dim=64, hq=4, hkv=4, block=64, dtype=F32, kv=F32, lens=(300, 1)),
    "fp32_one": Case(batch=1, drafts=1, dim=64, hq=4, hkv=4, block=64, dtype=F32, kv=F32, context=700),
    "fp32_rows_tiles": Case(drafts=70, hq=4, hkv=2, block=128, dtype=F32, kv=F32, context=700, lens=(650, 700)),
    "fp32_q": Case(drafts=7, dtype=F32, lens=(300, 5)),
    "fp32_q_rows": Case(drafts=70, dtype=F32, dim=64, hq=4, lens=(300, 5)),
    "fp32_q_d128_rows": Case(drafts=40, dtype=F32, lens=(300, 5)),
    "fp32_kv_bf16_q": Case(drafts=7, kv=F32, block=16, lens=(300, 5)),
}


@pytest.mark.parametrize("masked", ["tree", "chain"])
@pytest.mark.parametrize("name", CASES)
def test_whole_context(name, masked):
    c = CASES[name]
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    see = random_tree(c) if masked == "tree" else None
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, *tree_exact(c, q, pools, table, see))


SELECTED = {
    "few_rows": Case(drafts=3, topk=4, lens=(300, 17)),
    "rows": Case(drafts=20, topk=5, lens=(300, 299), block=16),
    "bs8": Case(drafts=9, topk=7, block=8, lens=(296, 61)),
    "bs128": Case(drafts=9, topk=3, block=128, context=700, lens=(700, 129)),
    "bs64_long": Case(batch=3, drafts=16, topk=40, block=64, context=9000, lens=(9000, 8000, 70)),
    "mha_d64": Case(drafts=5, topk=6, dim=64, hq=4, hkv=4, lens=(300, 0)),
    "fp32": Case(drafts=6, topk=6, dim=64, dtype=F32, kv=F32, lens=(300, 33)),
    "fp32_q": Case(drafts=6, topk=6, dtype=F32, lens=(300, -1)),
}


@pytest.mark.parametrize("name", SELECTED)
def test_selected_blocks(name):
    c = SELECTED[name]
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    see, sel = random_tree(c), selection(c)
    out, ws = call(c, q, pools, table, see, sel)
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, *tree_exact(c, q, pools, table, see, *sel))


def test_selection_behind_a_sequences_context_adds_nothing():
    """The selection kernels know one length; a shorter sequence's rows may name blocks that
    it does not reach.  They hold NaN here."""
    c = Case(batch=2, drafts=4, topk=8, lens=(300, 40))
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    ids = torch.tensor([0, 1, 2, 3, 5, 6, 8, 9], dtype=torch.int32).expand(2, c.hkv, 8).contiguous()
    cnt = torch.full((2, c.hkv), 8, dtype=torch.int32)
    out, ws = call(c, q, pools, table, None, (ids, cnt))
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, *tree_exact(c, q, pools, table, None, ids, cnt))


@pytest.mark.parametrize("cfg", [Case(batch=2, drafts=9, lens=(0, 70)), Case(batch=2, drafts=70, hq=8, lens=(0, 70)),
                                 Case(batch=2, drafts=9, lens=(0, 70), dtype=F32, kv=F32),
                                 Case(batch=2, drafts=9, lens=(0, 70), dtype=F32)], ids=["bf16", "rows", "fp32", "fp32_q"])
def test_rows_that_see_nothing_are_zero(cfg):
    c = cfg
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    see = random_tree(c)
    see[:, 2] = False
    see[:, 5:7] = False
    out, _ = call(c, q, pools, table, see)
    exact, bound = tree_exact(c, q, pools, table, see)
    check(c, out, exact, bound)
    assert (out[0, 2] == 0).all() and (out[0, 5:7] == 0).all() and (out[1, 2] != 0).any()


@pytest.mark.parametrize("cfg", [Case(batch=2, drafts=40, lens=(37, 129)), Case(batch=1, drafts=9, lens=(37,), hq=2),
                                 Case(batch=2, drafts=9, lens=(0, 70), dtype=F32, kv=F32, dim=64),
                                 Case(batch=2, drafts=70, hq=8, block=16, lens=(37, 129), dim=64),
                                 Case(batch=2, drafts=20, lens=(0, 70), dtype=F32)],
                         ids=["bf16", "few", "fp32", "rows", "fp32_q"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), 1e30])
def test_masked_drafts_may_hold_anything(cfg, value):
    """Drafts whose K and V are NaN, infinite or huge reach exactly the queries that see them:
    the others' rows are those of a tree without these drafts."""
    c = cfg
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    see = random_tree(c)
    odd = [3, c.drafts - 1, c.drafts // 2]
    for b, n in enumerate(c.all_lens):
        for j in odd:
            pg, off = place(c, table, b, torch.tensor([n + j]))
            pools[1][pg, :, off] = value
            if j != 3:
                pools[0][pg, :, off] = value
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    without = see.clone()
    without[:, :, odd] = False
    exact, bound = tree_exact(c, q, pools, table, without)
    for b in range(c.batch):
        clean = ~see[b][:, odd].any(-1)
        assert clean.any() and not clean.all()
        err = (out[b].cpu().double() - exact[b]).abs()[clean]
        assert (err <= bound[b][clean]).all()
        if value != 1e30:
            met = see[b][:, 3]
            assert met.any() and not torch.isfinite(out[b].cpu()[met]).any()


def test_lengths_default_to_n_tokens_and_one_draft_may_drop_its_axis():
    c = Case(batch=2, drafts=1)
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, 1, c.hq, c.dim)
    out, _ = call(c, q, pools, table, lens=None)
    check(c, out, *tree_exact(c, q, pools, table))
    p = c.params()
    flat = torch.empty(c.batch, c.hq, c.dim, device="cuda")
    B.sparse_attn_tree_decode(p, q[:, 0].contiguous().cuda(), pools[0].cuda(), pools[1].cuda(), table.cuda(), flat,
                              workspace(p))
    assert torch.equal(flat, out[:, 0])


@pytest.mark.parametrize("cfg", [Case(drafts=3), Case(drafts=40), Case(drafts=5, dtype=F32, kv=F32)], ids=["few", "rows", "fp32"])
def test_large_scores_and_scale(cfg):
    """Scores in the hundreds (one token takes all the weight) and a scale of the caller's."""
    c = cfg
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim, dtype=F32)
    q = (q * 30).to(c.dtype)
    out, _ = call(c, q, pools, table)
    check(c, out, *tree_exact(c, q, pools, table))
    out, _ = call(c, q, pools, table, p=c.params(softmax_scale=0.01))
    check(c, out, *tree_exact(c, q, pools, table, scale=0.01))


def test_bad_lengths_pages_and_selections_are_reported_and_skipped():
    c = Case(batch=3, drafts=5, topk=6, lens=(300, 200, 300))
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    exact, bound = tree_exact(c, q, pools, table)

    def others_right(out, but):
        for b in range(3):
            if b != but:
                assert ((out[b].cpu().double() - exact[b]).abs() <= bound[b]).all()

    for bad in (-2, 301, 2**31 - 1):
        sl = torch.tensor([300, bad, 300], dtype=torch.int32, device="cuda")
        out, ws = call(c, q, pools, table, lens=sl)
        assert B.sparse_attn_get_device_error(ws) == B.ERR_LENGTH
        others_right(out, 1)
        assert (out[1] == 5.0).all()
    for page in (-1, c.pages, 2**31 - 1):
        bad = table.clone()
        bad[1, 2] = page
        out, ws = call(c, q, pools, bad)
        assert B.sparse_attn_get_device_error(ws) == B.ERR_PAGE
        others_right(out, 1)
        # the block's tokens are left out
        sel = torch.tensor([0, 1, 3, 4, 5, 6], dtype=torch.int32).expand(3, c.hkv, 6).contiguous()
        ref, bnd = tree_exact(c, q, pools, table, None, sel, torch.full((3, c.hkv), 6))
        assert ((out[1].cpu().double() - ref[1]).abs() <= bnd[1]).all()
    ids, cnt = selection(c)
    wrong = ids.clone()
    wrong[1, 0, 0] = 10
    _, ws = call(c, q, pools, table, None, (wrong, cnt))
    assert B.sparse_attn_get_device_error(ws) == B.ERR_SEL_ID
    many = cnt.clone()
    many[1, 1] = 7
    _, ws = call(c, q, pools, table, None, (ids, many))
    assert B.sparse_attn_get_device_error(ws) == B.ERR_SEL_COUNT
    out, ws = call(c, q, pools, table)
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, exact, bound)


def test_results_repeat_bit_for_bit_and_share_a_workspace():
    """The same call again, another stream, and a second problem on the same workspace in
    between: equal bits (shared items are added up in a fixed order)."""
    c = Case(batch=2, drafts=12, context=6000, block=64, lens=(6000, 5000))
    d = Case(batch=2, drafts=12, context=6000, block=64, lens=(333, 5999), seed=1)
    data = []
    for x in (c, d):
        table = x.block_table()
        data.append((x.normal("q", x.batch, x.drafts, x.hq, x.dim).cuda(), [t.cuda() for t in x.fill(x.pools(), table)],
                     table.cuda()))
    first, ws = call(c, *data[0])
    first = first.clone()
    side = torch.cuda.Stream()
    for k in range(3):
        call(d, *data[1], ws=ws)
        torch.cuda.synchronize()
        again, _ = call(c, *data[0], ws=ws, stream=side if k == 1 else None)
        torch.cuda.synchronize()
        assert torch.equal(again, first)


def test_two_captured_graphs_on_one_workspace():
    c = Case(batch=2, drafts=6, context=3000, lens=(100, 2000))
    table = c.block_table()
    pools = c.fill(c.pools(), table, upto=[3006, 3006])
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    p = c.params()
    ws = workspace(p)
    lens = torch.tensor(c.all_lens, dtype=torch.int32, device="cuda")
    gq, gk, gv, gt = q.cuda(), pools[0].cuda(), pools[1].cuda(), table.cuda()
    outs = [torch.zeros(c.batch, c.drafts, c.hq, c.dim, device="cuda") for _ in range(2)]
    masks = [pack_mask(random_tree(dataclasses.replace(c, seed=s))).cuda() for s in range(2)]
    B.sparse_attn_tree_decode(p, gq, gk, gv, gt, outs[0], ws, seq_lens=lens, tree_mask=masks[0])
    torch.cuda.synchronize()
    graphs = []
    for out, mask in zip(outs, masks):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            B.sparse_attn_tree_decode(p, gq, gk, gv, gt, out, ws, seq_lens=lens, tree_mask=mask)
        graphs.append(graph)
    for new in ((100, 2000), (3000, 7), (0, 1)):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        for graph in graphs + graphs[::-1]:
            graph.replay()
        x = dataclasses.replace(c, lens=new)
        for s in range(2):
            see = random_tree(dataclasses.replace(c, seed=s))
            check(x, outs[s], *tree_exact(x, q, pools, table, see))
    assert B.sparse_attn_get_device_error(ws) == 0


def test_chain_of_the_whole_length_is_causal_attention():
    """No context and 200 drafts in a chain: a prompt's causal attention."""
    c = Case(batch=2, drafts=200, hq=4, hkv=2, dim=64, context=0, lens=(0, 0))
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    out, _ = call(c, q, pools, table)
    check(c, out, *tree_exact(c, q, pools, table, chain_mask(200).expand(2, -1, -1)))
