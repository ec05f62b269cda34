"""Accepted drafts moved to the end of the context, and the whole speculative loop: append,
select, tree attention, commit, metadata."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from query_guided_block_gb300.decoder import DraftDecoder, SparseDecoder
from tests.draft_reference import Case, pack_mask, place, random_tree, rotate, rotation_bound, tree_exact

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


def box_of(c, pool, table, upto):
    lo = torch.full((c.batch, c.hkv, c.nb_cap, c.dim), 3.0, dtype=c.kv)
    hi = torch.full_like(lo, -3.0)
    for b, n in enumerate(upto):
        for j in range(-(-max(0, n) // c.block)):
            pg, off = place(c, table, b, torch.arange(j * c.block, min(n, (j + 1) * c.block)))
            lo[b, :, j], hi[b, :, j] = pool[pg, :, off].amin(0), pool[pg, :, off].amax(0)
    return lo, hi


def commit(c, pools, table, path, path_len, lens, box=None, ws=None):
    p = c.params()
    ws = workspace(p) if ws is None else ws
    new = torch.full((c.batch,), 77, dtype=torch.int32, device="cuda")
    lo, hi = (None, None) if box is None else box
    B.sparse_attn_commit_drafts(p, path.cuda(), torch.tensor(path_len, dtype=torch.int32, device="cuda"), *pools, table.cuda(),
                                new, ws, seq_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                kmin=lo, kmax=hi)
    return new.tolist(), B.sparse_attn_get_device_error(ws)


CASES = {
    "mixed": (Case(batch=5, drafts=16, lens=(0, 31, 290, -1, 64)),
              [[0, 2, 5, 15], [0, 1, 2, 3], [3, 7, 8, 9], [0, 1, 2, 3], [15, 0, 0, 0]], [4, 4, 3, 2, 1]),
    "overlapping": (Case(batch=1, drafts=33, lens=(300,), block=8), [list(range(1, 33))], [32]),
    "nothing": (Case(batch=2, drafts=4, lens=(10, 20)), [[0], [0]], [0, 0]),
    "long": (Case(batch=1, drafts=700, hq=1, hkv=1, lens=(100,), block=128), [list(range(1, 700, 2))], [350]),
    "fp32": (Case(batch=2, drafts=40, lens=(33, 299), dtype=F32, kv=F32), [list(range(0, 40, 2)), list(range(20, 40))], [20, 19]),
    "d64": (Case(batch=2, drafts=9, dim=64, block=16, lens=(7, 300)), [[1, 3, 8], [0, 4, 5]], [3, 3]),
}


@pytest.mark.parametrize("with_box", [True, False])
@pytest.mark.parametrize("name", CASES)
def test_commit_moves_the_path(name, with_box):
    c, path, path_len = CASES[name]
    path = torch.tensor(path, dtype=torch.int32)
    table = c.block_table()
    k, v = c.fill(c.pools(empty=0.5), table)
    lo, hi = box_of(c, k, table, c.all_lens)
    gk, gv, glo, ghi = k.cuda(), v.cuda(), lo.cuda(), hi.cuda()
    new, flags = commit(c, (gk, gv), table, path, path_len, c.all_lens, (glo, ghi) if with_box else None)
    assert flags == 0
    after = [n + m if n >= 0 else n for n, m in zip(c.all_lens, path_len)]
    assert new == after
    want_k, want_v = k.clone(), v.clone()
    for b, (n, m) in enumerate(zip(c.all_lens, path_len)):
        if n < 0:
            continue
        sp, so = place(c, table, b, n + path[b, :m].long())
        dp, do = place(c, table, b, n + torch.arange(m))
        want_k[dp, :, do], want_v[dp, :, do] = k[sp, :, so], v[sp, :, so]
    assert torch.equal(gk.cpu(), want_k) and torch.equal(gv.cpu(), want_v)
    if with_box:
        touched = [n if m > 0 else -1 for n, m in zip(after, path_len)]
        lo2, hi2 = box_of(c, want_k, table, after)
        for b, n in enumerate(touched):
            if n >= 0:
                lo[b], hi[b] = lo2[b], hi2[b]
    assert torch.equal(glo.cpu(), lo) and torch.equal(ghi.cpu(), hi)


def test_bad_paths_and_pages_are_reported_and_move_nothing():
    c = Case(batch=3, drafts=8, lens=(100, 40, 300))
    table = c.block_table()
    k, v = c.fill(c.pools(empty=0.5), table)
    good = torch.tensor([[0, 2, 5, 7]] * 3, dtype=torch.int32)

    def attempt(path=good, lens=(100, 40, 300), n=(4, 4, 4), bt=table):
        gk, gv = k.cuda(), v.cuda()
        new, flags = commit(c, (gk, gv), bt, path, list(n), list(lens))
        pg, off = place(c, table, 1, torch.arange(40, 48))
        return new, flags, torch.equal(gk.cpu()[pg, :, off], k[pg, :, off]) and torch.equal(gv.cpu()[pg, :, off], v[pg, :, off])

    assert attempt() == ([104, 44, 304], 0, False)
    for row in ([0, 2, 2, 7], [5, 2, 6, 7], [-1, 2, 5, 7], [0, 2, 5, 8], [0, 2, 5, 2**31 - 1], [-2**31, 2, 5, 7]):
        path = good.clone()
        path[1] = torch.tensor(row)
        assert attempt(path=path) == ([104, 40, 304], B.ERR_LENGTH, True), row
    for n in (-1, 5, 2**31 - 1):
        assert attempt(n=(4, n, 4)) == ([104, 40, 304], B.ERR_LENGTH, True)
    for bad in (-2, 301):
        assert attempt(lens=(100, bad, 300)) == ([104, bad, 304], B.ERR_LENGTH, True)
    bt = table.clone()
    bt[1, 1] = c.pages
    assert attempt(bt=bt) == ([104, 40, 304], B.ERR_PAGE, True)
    # without lengths: n_tokens
    new, flags = commit(c, (k.cuda(), v.cuda()), table, good, [1, 2, 3], None)
    assert (new, flags) == ([301, 302, 303], 0)


@pytest.mark.parametrize("graph", [False, True])
def test_the_speculative_loop(graph):
    """Three steps of append, tree attention and commit (replayed as one graph, or eager): the
    outputs equal attention over what a cache filled token by token holds, and the key box
    equals build_meta's at the end."""
    c = Case(batch=3, drafts=6, context=200, room=0, lens=(150, 0, 97), block=16, hq=8, hkv=2)
    table = c.block_table()
    k0, v0 = c.fill(c.pools(empty=0.0), table, upto=[150, 0, 97])
    lo, hi = box_of(c, k0, table, c.all_lens)
    gk, gv, gt, glo, ghi = k0.cuda(), v0.cuda(), table.cuda(), lo.cuda(), hi.cuda()
    p = c.params()
    dec = DraftDecoder(p, torch.tensor(c.all_lens, dtype=torch.int32, device="cuda"))
    rows = c.batch * c.drafts
    freq = 10000.0 ** (-torch.arange(c.dim // 2, dtype=torch.float64) / (c.dim // 2))
    st = dict(q=torch.zeros(rows, c.hq, c.dim, dtype=BF), k=torch.zeros(rows, c.hkv, c.dim, dtype=BF),
              v=torch.zeros(rows, c.hkv, c.dim, dtype=BF), pos=torch.zeros(rows, dtype=torch.int32),
              mask=torch.zeros(c.batch, c.drafts, 1, dtype=torch.int32), path=torch.zeros(c.batch, 4, dtype=torch.int32),
              n=torch.zeros(c.batch, dtype=torch.int32))
    st = {n: t.cuda() for n, t in st.items()}
    q_out = torch.empty_like(st["q"])
    gf = freq.cuda()

    def step():
        dec.append(st["q"], st["k"], st["v"], gf, q_out, gk, gv, gt, positions=st["pos"])
        dec.decode(q_out.view(c.batch, c.drafts, c.hq, c.dim), gk, gv, gt, tree_mask=st["mask"])
        dec.commit(st["path"], st["n"], gk, gv, gt, kmin=glo, kmax=ghi)

    captured = None
    if graph:
        dec.seq_lens.fill_(-1)                    # warm up on an inactive batch
        step()
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        dec.seq_lens.copy_(torch.tensor(c.all_lens, dtype=torch.int32))
    lens = c.all_lens
    for s in range(3):
        x = Case(**{**c.__dict__, "lens": tuple(lens), "seed": s})
        see = random_tree(x)
        q_new, k_new, v_new = (x.normal(w, c.batch, c.drafts, h, c.dim) for w, h in (("q", c.hq), ("k", c.hkv), ("v", c.hkv)))
        depth = see.sum(-1) - 1
        pos = torch.tensor(lens)[:, None] + depth
        path = torch.zeros(c.batch, 4, dtype=torch.int32)
        n = torch.zeros(c.batch, dtype=torch.int32)
        for b in range(c.batch):                  # the path to the last draft, cut to 4
            way = see[b, c.drafts - 1 - b].nonzero().flatten()[:4]
            path[b, : len(way)] = way.to(torch.int32)
            n[b] = len(way) - (1 if b == s else 0)
        for name, t in dict(q=q_new.flatten(0, 1), k=k_new.flatten(0, 1), v=v_new.flatten(0, 1), pos=pos.flatten().int(),
                            mask=pack_mask(see), path=path, n=n).items():
            st[name].copy_(t)
        # the same append into copies: what the pages hold with the drafts in place
        ck, cv, cq = gk.clone(), gv.clone(), torch.empty_like(q_out)
        dec.append(st["q"], st["k"], st["v"], gf, cq, ck, cv, gt, positions=st["pos"])
        k, v = ck.cpu(), cv.cpu()
        if captured is not None:
            captured.replay()
        else:
            step()
        assert torch.equal(q_out, cq)
        qr = cq.view(c.batch, c.drafts, c.hq, c.dim).cpu()
        for b in range(c.batch):
            pg, off = place(c, table, b, lens[b] + torch.arange(c.drafts))
            rk, mk = rotate(k_new[b], pos[b], freq, B.ROTATE_HALVES)
            rq, mq = rotate(q_new[b], pos[b], freq, B.ROTATE_HALVES)
            assert ((k[pg, :, off].double() - rk).abs() <= rotation_bound(rk, mk, BF)).all()
            assert ((qr[b].double() - rq).abs() <= rotation_bound(rq, mq, BF)).all()
            assert torch.equal(v[pg, :, off], v_new[b])
        exact, bound = tree_exact(x, qr, (k, v), table, see)
        assert ((dec.out.cpu().double() - exact).abs() <= bound).all()
        for b in range(c.batch):
            m = int(n[b])
            sp, so = place(c, table, b, lens[b] + path[b, :m].long())
            dp, do = place(c, table, b, lens[b] + torch.arange(m))
            k[dp, :, do], v[dp, :, do] = k[sp, :, so], v[sp, :, so]
        lens = [a + int(m) for a, m in zip(lens, n)]
        assert dec.seq_lens.tolist() == lens
    assert dec.device_error() == 0
    # K and V of the committed tokens moved untouched, and the box is build_meta's
    rmin, rmax = torch.zeros_like(glo), torch.zeros_like(ghi)
    for b, n in enumerate(lens):
        pg, off = place(c, table, b, torch.arange(n))
        assert torch.equal(gk.cpu()[pg, :, off], k[pg, :, off]) and torch.equal(gv.cpu()[pg, :, off], v[pg, :, off])
        pb = B.make_params(1, c.hq, c.hkv, c.dim, n, c.block, c.pages, 0, 1, capacity_tokens=c.capacity)
        ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        B.sparse_attn_build_meta(pb, gk, gt[b:b + 1].contiguous(), rmin[b:b + 1], rmax[b:b + 1], None, ws)
        nb = -(-n // c.block)
        assert torch.equal(glo[b, :, :nb], rmin[b, :, :nb]) and torch.equal(ghi[b, :, :nb], rmax[b, :, :nb])


def test_select_then_tree_over_the_selection():
    """sparse_attn_select's rows feed the tree attention as they are."""
    c = Case(batch=2, drafts=8, context=2000, block=32, topk=10, window=100)
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    p = c.params()
    dec = SparseDecoder(p)
    gk, gv, gt = pools[0].cuda(), pools[1].cuda(), table.cuda()
    dec.build_meta(gk, gt)
    dec.select(q.cuda())
    assert dec.device_error() == 0
    tree = DraftDecoder(p, torch.full((2,), 2000, dtype=torch.int32, device="cuda"))
    see = random_tree(c)
    out = tree.decode(q.cuda(), gk, gv, gt, tree_mask=pack_mask(see).cuda(), sel_ids=dec.sel_ids, sel_count=dec.sel_count)
    exact, bound = tree_exact(c, q, pools, table, see, dec.sel_ids.cpu(), dec.sel_count.cpu())
    assert ((out.cpu().double() - exact).abs() <= bound).all()
    assert tree.device_error() == 0


def test_pools_larger_than_four_gigabytes():
    """Pages whose byte and element offsets pass 32 bits."""
    pages, hkv, bs, dim = 20000, 8, 128, 128      # 5.2 GB a pool
    k = torch.zeros(pages, hkv, bs, dim, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    p = B.make_params(1, 8, hkv, dim, 256, bs, pages, 0, 1, num_queries=4, capacity_tokens=384)
    table = torch.tensor([[19990, 17000, 19999]], dtype=torch.int32, device="cuda")
    c = Case(batch=1, hq=8, hkv=hkv, block=bs, context=256, drafts=4, lens=(254,))
    small_table = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    pools = [torch.full((c.pages, hkv, bs, dim), float("nan"), dtype=BF) for _ in range(2)]
    c.fill(pools, small_table, upto=[254])
    for mine, pool in zip((k, v), pools):
        mine[table[0].long()] = pool[:3].nan_to_num().cuda()
    dec = DraftDecoder(p, torch.tensor([254], dtype=torch.int32, device="cuda"))
    kn, vn = c.normal("kn", 4, hkv, dim), c.normal("vn", 4, hkv, dim)
    q = c.normal("q", 1, 4, 8, dim)
    dec.append(None, kn.cuda(), vn.cuda(), None, None, k, v, table)
    pg, off = place(c, small_table, 0, torch.arange(254, 258))
    pools[0][pg, :, off], pools[1][pg, :, off] = kn, vn
    out = dec.decode(q.cuda(), k, v, table)
    exact, bound = tree_exact(c, q, pools, small_table)
    assert ((out.cpu().double() - exact).abs() <= bound).all()
    dec.commit(torch.tensor([[1, 3]], dtype=torch.int32, device="cuda"), torch.tensor([2], dtype=torch.int32, device="cuda"),
               k, v, table)
    assert torch.equal(k[17000, :, 126].cpu(), kn[1]) and torch.equal(v[17000, :, 127].cpu(), vn[3])
    assert dec.seq_lens.tolist() == [256] and dec.device_error() == 0
