"""Draft-tree attention with more than 16 query rows a KV head over contexts that may be long: the
calls that the tensor-memory kernel takes, at every number of row copies, against 64-bit attention.
The problem's length is large and the sequences are short, so the 64-bit side stays small."""
import dataclasses

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, pack_mask, place, random_tree, tree_exact
from tests.test_gpu_tree import call, check, selection, workspace

pytestmark = pytest.mark.gpu
F32 = torch.float32
LONG = 8000                                       # n_tokens of the problem

# 4 rows a draft: up to 32 rows, 64, 128, and two groups of rows
DRAFTS = {"r28": 7, "r32": 8, "r36": 9, "r64": 16, "r100": 25, "r128": 32, "r180": 45}


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def prepared(c):
    table = c.block_table()
    return table, c.fill(c.pools(), table), c.normal("q", c.batch, c.drafts, c.hq, c.dim)


@pytest.mark.parametrize("masked", ["tree", "chain"])
@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("rows", DRAFTS)
def test_ragged_lengths(rows, dim, masked):
    c = Case(batch=6, drafts=DRAFTS[rows], dim=dim, block=16, context=LONG, lens=(700, 37, 0, 129, -1, 255))
    table, pools, q = prepared(c)
    see = random_tree(c) if masked == "tree" else None
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, *tree_exact(c, q, pools, table, see))


@pytest.mark.parametrize("block", [8, 32, 64, 128])
@pytest.mark.parametrize("rows", ["r28", "r64", "r100"])
def test_block_sizes(rows, block):
    dim = 64 if block == 128 else 128
    c = Case(batch=3, drafts=DRAFTS[rows], dim=dim, block=block, context=LONG, lens=(513, 128 - DRAFTS[rows], 1))
    table, pools, q = prepared(c)
    see = random_tree(c)
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, *tree_exact(c, q, pools, table, see))


@pytest.mark.parametrize("rows,dim", [("r28", 128), ("r64", 128), ("r100", 128), ("r180", 128), ("r28", 64), ("r64", 64),
                                      ("r100", 64)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), 1e30])
def test_masked_drafts_may_hold_anything(rows, dim, value):
    """Drafts whose K and V are NaN, infinite or huge reach exactly the queries that see them."""
    c = Case(batch=3, drafts=DRAFTS[rows], dim=dim, block=16, context=LONG, lens=(37, 300, 121))
    table, pools, q = prepared(c)
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
        assert ((out[b].cpu().double() - exact[b]).abs()[clean] <= bound[b][clean]).all()
        if value != 1e30:
            met = see[b][:, 3]
            assert met.any() and not torch.isfinite(out[b].cpu()[met]).any()


@pytest.mark.parametrize("rows", ["r28", "r64", "r100"])
def test_rows_that_see_nothing_are_zero(rows):
    c = Case(batch=3, drafts=DRAFTS[rows], context=LONG, lens=(0, 70, 0))
    table, pools, q = prepared(c)
    see = random_tree(c)
    see[:, 2] = False
    see[:, 5:7] = False
    see[2] = False                                # a sequence without context whose queries see nothing
    out, ws = call(c, q, pools, table, see)
    check(c, out, *tree_exact(c, q, pools, table, see))
    assert (out[0, 2] == 0).all() and (out[0, 5:7] == 0).all() and (out[2] == 0).all() and (out[1, 2] != 0).any()
    assert B.sparse_attn_get_device_error(ws) == 0


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("rows", ["r28", "r64", "r100", "r180"])
def test_selected_blocks(rows, dim):
    c = Case(batch=4, drafts=DRAFTS[rows], dim=dim, topk=240, context=LONG, lens=(700, 299, 33, 0))
    table, pools, q = prepared(c)
    see, sel = random_tree(c), selection(c)
    out, ws = call(c, q, pools, table, see, sel)
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, *tree_exact(c, q, pools, table, see, *sel))


@pytest.mark.parametrize("rows,dim", [("r28", 128), ("r64", 64), ("r28", 64)])
def test_many_short_sequences(rows, dim):
    """More items than parts: whole items, several to a CTA.  Twice, for equal bits."""
    c = Case(batch=90, drafts=DRAFTS[rows], dim=dim, context=300, lens=tuple((37 * i) % 301 - (i == 17) * 700 for i in range(90)))
    c = dataclasses.replace(c, lens=tuple(max(-1, n) for n in c.lens))
    table, pools, q = prepared(c)
    see = random_tree(c)
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, *tree_exact(c, q, pools, table, see))
    again, _ = call(c, q, pools, table, see, ws=ws)
    assert torch.equal(again, out)


@pytest.mark.parametrize("rows,dim,batch", [("r28", 64, 38), ("r28", 128, 38), ("r64", 64, 60), ("r100", 128, 20)])
def test_items_split_between_parts(rows, dim, batch):
    """Few long sequences among short ones: parts of one item on several CTAs, joined by the last of
    them or by a launch of its own.  Three times on one workspace, for equal bits."""
    c = Case(batch=batch, drafts=DRAFTS[rows], dim=dim, hq=8, block=64, context=2500,
             lens=tuple(2500 - 7 * i if i % 9 == 0 else 61 * i % 500 for i in range(batch)))
    table, pools, q = prepared(c)
    out, ws = call(c, q, pools, table)
    first = out.clone()
    assert B.sparse_attn_get_device_error(ws) == 0
    for _ in range(2):
        again, _ = call(c, q, pools, table, ws=ws)
        assert torch.equal(again, first)
    # the 64-bit side of some sequences only
    some = [0, 1, 9, batch - 1]
    d = dataclasses.replace(c, lens=tuple(n if i in some else -1 for i, n in enumerate(c.lens)))
    exact, bound = tree_exact(d, q, pools, table)
    for b in some:
        assert ((out[b].cpu().double() - exact[b]).abs() <= bound[b]).all()


def test_two_captured_graphs_on_one_workspace_and_another_stream():
    c = Case(batch=2, drafts=16, context=LONG, lens=(100, 700))
    table = c.block_table()
    pools = c.fill(c.pools(), table, upto=[1016, 1016])
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    p, lens = c.params(), torch.tensor(c.all_lens, dtype=torch.int32, device="cuda")
    ws = workspace(p)
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
    side = torch.cuda.Stream()
    for new in ((100, 700), (1000, 7), (0, 1)):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for graph in graphs + graphs[::-1]:
                graph.replay()
        side.synchronize()
        x = dataclasses.replace(c, lens=new)
        for s in range(2):
            see = random_tree(dataclasses.replace(c, seed=s))
            check(x, outs[s], *tree_exact(x, q, pools, table, see))
    assert B.sparse_attn_get_device_error(ws) == 0


def test_many_calls_back_to_back():
    """Calls that overlap at their ends (the next one starts while the last one finishes) and share
    a workspace: 200 of two problems in turn, every result the first one's bits."""
    probs = [Case(batch=2, drafts=16, context=LONG, lens=(3000, 100)), Case(batch=5, drafts=9, dim=64, context=LONG, seed=1,
                                                                            lens=(1, 2000, -1, 300, 64))]
    data, size = [], 0
    for x in probs:
        table = x.block_table()
        data.append((x.normal("q", x.batch, x.drafts, x.hq, x.dim).cuda(), [t.cuda() for t in x.fill(x.pools(), table)],
                     table.cuda(), torch.tensor(x.all_lens, dtype=torch.int32, device="cuda"), x.params()))
        size = max(size, B.sparse_attn_tree_workspace_size(data[-1][4]))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    B.sparse_attn_workspace_init(ws)
    outs = [[torch.zeros(x.batch, x.drafts, x.hq, x.dim, device="cuda") for _ in range(100)] for x in probs]
    for k in range(100):
        for (q, pools, table, lens, p), o in zip(data, outs):
            B.sparse_attn_tree_decode(p, q, pools[0], pools[1], table, o[k], ws, seq_lens=lens)
    torch.cuda.synchronize()
    assert B.sparse_attn_get_device_error(ws) == 0
    for o in outs:
        assert all(torch.equal(x, o[0]) for x in o)
        assert torch.isfinite(o[0]).all()


def test_bad_lengths_and_pages_are_reported_and_skipped():
    c = Case(batch=3, drafts=16, context=LONG, lens=(300, 200, 300))
    table, pools, q = prepared(c)
    exact, bound = tree_exact(c, q, pools, table)
    for bad in (-2, LONG + 1, 2**31 - 1):
        sl = torch.tensor([300, bad, 300], dtype=torch.int32, device="cuda")
        out, ws = call(c, q, pools, table, lens=sl)
        assert B.sparse_attn_get_device_error(ws) == B.ERR_LENGTH
        assert (out[1] == 5.0).all()
        for b in (0, 2):
            assert ((out[b].cpu().double() - exact[b]).abs() <= bound[b]).all()
    for page in (-1, c.pages, 2**31 - 1):
        bad = table.clone()
        bad[1, 2] = page
        out, ws = call(c, q, pools, bad)
        assert B.sparse_attn_get_device_error(ws) == B.ERR_PAGE
        sel = torch.tensor([0, 1, 3, 4, 5, 6], dtype=torch.int32).expand(3, c.hkv, 6).contiguous()
        ref, bnd = tree_exact(c, q, pools, table, None, sel, torch.full((3, c.hkv), 6))
        assert ((out[1].cpu().double() - ref[1]).abs() <= bnd[1]).all()
        for b in (0, 2):
            assert ((out[b].cpu().double() - exact[b]).abs() <= bound[b]).all()


def test_two_streams_at_once():
    """Two problems, each with its own workspace, on two streams without any order between them."""
    probs = [Case(batch=2, drafts=16, context=LONG, lens=(3000, 100)), Case(batch=1, drafts=7, context=LONG, seed=1, lens=(5000,)),
             Case(batch=2, drafts=3, seed=2)]
    data, expect = [], []
    for x in probs:
        table = x.block_table()
        q, pools = x.normal("q", x.batch, x.drafts, x.hq, x.dim).cuda(), [t.cuda() for t in x.fill(x.pools(), table)]
        lens, p = torch.tensor(x.all_lens, dtype=torch.int32, device="cuda"), x.params()
        data.append((p, q, pools[0], pools[1], table.cuda(), lens, workspace(p)))
        expect.append(call(x, q, pools, table)[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in probs]
    outs = [[torch.zeros_like(e) for _ in range(30)] for e in expect]
    torch.cuda.synchronize()
    for k in range(30):
        for (p, q, kp, vp, table, lens, ws), o, s in zip(data, outs, streams):
            B.sparse_attn_tree_decode(p, q, kp, vp, table, o[k], ws, seq_lens=lens, stream=s)
    torch.cuda.synchronize()
    for (*_, ws), o, e in zip(data, outs, expect):
        assert B.sparse_attn_get_device_error(ws) == 0
        assert all(torch.equal(x, e) for x in o)


def test_growing_context_under_one_parameter_set():
    """The problem's length only bounds the sequences': right with little room above them and with much
    (the two kernels)."""
    for room in (300, LONG):
        c = Case(batch=2, drafts=9, context=room, lens=(299, 64))
        table, pools, q = prepared(c)
        out, ws = call(c, q, pools, table)
        check(c, out, *tree_exact(c, q, pools, table))
        assert B.sparse_attn_get_device_error(ws) == 0
