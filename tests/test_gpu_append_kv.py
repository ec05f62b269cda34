"""Appending rotated keys, values and the key box through the C ABI, against 64-bit rotation
and against the metadata calls; nothing but the new tokens' places may change."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, place, rotate, rotation_bound

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


def inv_freq(rotary, base=10000.0):
    return base ** (-torch.arange(rotary // 2, dtype=torch.float64) / (rotary // 2)) if rotary else None


def run(c, counts, rotary=None, pairing=B.ROTATE_HALVES, fused=False, positions=None, with_q=True, box=True,
        uniform=False, pad_rows=0, alias=False, base=10000.0):
    """One append against the 64-bit rotation.  counts: new rows per sequence."""
    rotary = c.dim if rotary is None else rotary
    lens, n = c.all_lens, sum(counts)
    rows = n + pad_rows
    table = c.block_table()
    k_pool, v_pool = c.fill(c.pools(empty=0.25), table, upto=[max(0, x) for x in lens])
    width = (c.hq + 2 * c.hkv) * c.dim
    if fused:
        qkv = c.normal("qkv", rows, width)
        parts = [c.hq * c.dim, c.hkv * c.dim, c.hkv * c.dim]
        q, k, v = (x.unflatten(1, (-1, c.dim)) for x in qkv.split(parts, 1))
        gq, gk, gv = (x.unflatten(1, (-1, c.dim)) for x in qkv.cuda().split(parts, 1))
    else:
        q, k, v = c.normal("q", rows, c.hq, c.dim), c.normal("k", rows, c.hkv, c.dim), c.normal("v", rows, c.hkv, c.dim)
        gq, gk, gv = q.cuda(), k.cuda(), v.cuda()
    freq = inv_freq(rotary, base)
    p = c.params()
    ws = workspace(p)
    # the box before: of the tokens that are there (untouched rows keep a marker)
    nb = c.nb_cap
    kmin = torch.full((c.batch, c.hkv, nb, c.dim), 7.0, dtype=c.kv)
    kmax = torch.full_like(kmin, -7.0)
    for b, old in enumerate(lens):
        for j in range(-(-max(0, old) // c.block)):
            t = torch.arange(j * c.block, min(old, (j + 1) * c.block))
            pg, off = place(c, table, b, t)
            keys = k_pool[pg, :, off]
            kmin[b, :, j], kmax[b, :, j] = keys.amin(0), keys.amax(0)
    g = dict(k=k_pool.cuda(), v=v_pool.cuda(), bt=table.cuda(), lo=kmin.cuda(), hi=kmax.cuda())
    q_out = gq if alias else torch.full((rows, c.hq, c.dim), 9.0, dtype=c.dtype, device="cuda")
    cu = None if uniform else torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda")
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    B.sparse_attn_append_kv(p, gq if with_q else None, gk, gv, None if freq is None else freq.cuda(),
                            q_out if with_q else None, g["k"], g["v"], g["bt"], ws, cu_rows=cu, seq_lens=sl,
                            positions=None if positions is None else positions.cuda(), pairing=pairing,
                            kmin=g["lo"] if box else None, kmax=g["hi"] if box else None)
    assert B.sparse_attn_get_device_error(ws) == 0

    # rows -> tokens
    want_k, want_v, want_q = k_pool.clone(), v_pool.clone(), (q if alias else torch.full_like(q, 9.0)).clone()
    r = 0
    for b, (old, cnt) in enumerate(zip(lens, counts)):
        if old < 0 or cnt == 0:
            r += cnt
            continue
        sl_rows = slice(r, r + cnt)
        t = torch.arange(old, old + cnt)
        pos = t if positions is None else positions[sl_rows]
        pg, off = place(c, table, b, t)
        rk, mk = rotate(k[sl_rows], pos, freq, pairing)
        got = g["k"].cpu()[pg, :, off].double()
        assert ((got - rk).abs() <= rotation_bound(rk, mk, c.kv)).all(), f"keys of sequence {b}"
        want_k[pg, :, off] = g["k"].cpu()[pg, :, off]
        want_v[pg, :, off] = v[sl_rows].to(c.kv)
        if with_q:
            rq, mq = rotate(q[sl_rows], pos, freq, pairing)
            gotq = q_out.cpu()[sl_rows].double()
            assert ((gotq - rq).abs() <= rotation_bound(rq, mq, c.dtype)).all(), f"queries of sequence {b}"
            want_q[sl_rows] = q_out.cpu()[sl_rows]
        if rotary < c.dim:                        # channels behind the rotation: rounded once at most
            assert torch.equal(g["k"].cpu()[pg, :, off][..., rotary:], k[sl_rows][..., rotary:].to(c.kv))
        r += cnt
    assert torch.equal(g["k"].cpu(), want_k) and torch.equal(g["v"].cpu(), want_v)
    if with_q:
        assert torch.equal(q_out.cpu(), want_q)
    # the box: of the stored keys, untouched rows as they were
    for b, (old, cnt) in enumerate(zip(lens, counts)):
        if old < 0 or cnt == 0 or not box:
            continue
        for j in range(old // c.block, (old + cnt - 1) // c.block + 1):
            t = torch.arange(j * c.block, min(old + cnt, (j + 1) * c.block))
            pg, off = place(c, table, b, t)
            keys = want_k[pg, :, off]
            kmin[b, :, j], kmax[b, :, j] = keys.amin(0), keys.amax(0)
    assert torch.equal(g["lo"].cpu(), kmin) and torch.equal(g["hi"].cpu(), kmax)


CASES = {
    "one_token": (Case(batch=1, lens=(300,)), [1], {}),
    "one_token_empty_context": (Case(batch=1, lens=(0,)), [1], {}),
    "decode_batch": (Case(batch=5, lens=(300, 31, 32, 0, 299)), [1] * 5, dict(uniform=True)),
    "ragged_with_empty_rows": (Case(batch=6, lens=(3, 300, 64, 0, 17, 250), drafts=90), [5, 0, 90, 33, 1, 64], {}),
    "inactive_and_padding": (Case(batch=4, lens=(40, -1, 7, -1), drafts=20), [9, 4, 20, 0], dict(pad_rows=11)),
    "pairs": (Case(batch=2, lens=(100, 31), drafts=70), [70, 2], dict(pairing=B.ROTATE_PAIRS)),
    "partial_halves": (Case(batch=2, lens=(100, 31), drafts=70), [70, 2], dict(rotary=48)),
    "partial_pairs_d64": (Case(batch=2, dim=64, lens=(100, 31), drafts=70), [7, 69], dict(rotary=16, pairing=B.ROTATE_PAIRS)),
    "no_rotation": (Case(batch=2, lens=(100, 31), drafts=70), [70, 2], dict(rotary=0)),
    "fused_projection": (Case(batch=3, lens=(1, 2, 3), drafts=65), [65, 64, 63], dict(fused=True)),
    "keys_only_no_box": (Case(batch=2, lens=(33, 5), drafts=40), [40, 12], dict(with_q=False, box=False)),
    "in_place_queries": (Case(batch=2, lens=(33, 5), drafts=40), [40, 12], dict(alias=True)),
    "fp32": (Case(batch=2, dim=64, hq=4, hkv=4, block=64, lens=(100, 300), drafts=200, dtype=F32, kv=F32), [200, 77], {}),
    "fp32_d128_pairs": (Case(batch=2, block=16, lens=(100, 300), drafts=40, dtype=F32, kv=F32), [33, 40],
                        dict(pairing=B.ROTATE_PAIRS)),
    "fp32_rows_bf16_cache": (Case(batch=2, block=8, lens=(100, 3), drafts=100, dtype=F32), [100, 23], {}),
    "bf16_rows_fp32_cache": (Case(batch=2, block=128, lens=(100, 300), drafts=300, kv=F32), [300, 129], {}),
    "many_heads": (Case(batch=2, hq=64, hkv=64, block=128, lens=(129, 0), drafts=130), [130, 128], {}),
    "one_kv_head": (Case(batch=3, hq=8, hkv=1, dim=64, block=8, lens=(8, 16, 300), drafts=9), [9, 8, 7], {}),
    "rows_longer_than_a_step": (Case(batch=80, hq=64, hkv=8, context=40, lens=tuple(7 * i % 41 for i in range(80)), drafts=5),
                                [i % 6 for i in range(80)], {}),
    "keys_only_one_head": (Case(batch=2, hq=8, hkv=1, lens=(33, 5), drafts=130), [130, 64], dict(with_q=False)),
    "long_prompt": (Case(batch=1, hq=4, hkv=2, dim=64, block=16, context=1000, lens=(77,), drafts=900), [900], {}),
    "more_sequences_than_threads": (Case(batch=401, hq=2, hkv=1, dim=64, block=8, context=9,
                                         lens=tuple(i % 10 for i in range(401)), drafts=3), [i % 4 for i in range(401)], {}),
}


@pytest.mark.parametrize("name", CASES)
def test_append_matches_the_rotation_in_64_bits(name):
    c, counts, kw = CASES[name]
    run(c, counts, **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_and_shared_positions(dtype):
    """Positions in the millions (an fp32 angle would be off by a tenth), drafts of one depth
    at one position, negative ones too."""
    c = Case(batch=2, lens=(100, 31), drafts=40, dtype=dtype)
    pos = torch.tensor([2_000_000 + i // 3 for i in range(40)] + [-5, -5, 131071, 0, 50_000_000], dtype=torch.int32)
    run(c, [40, 5], positions=pos)
    run(c, [40, 5], positions=pos, base=500000.0, pairing=B.ROTATE_PAIRS)


@pytest.mark.parametrize("kv", [BF, F32])
def test_box_equals_the_metadata_calls(kv):
    """Appending in several steps with the box kept on the way leaves what build_meta makes of
    the pages, bit for bit."""
    c = Case(batch=3, context=500, lens=(0, 0, 0), kv=kv, block=32, drafts=0, room=20)
    table = c.block_table()
    k, v = (x.cuda() for x in c.pools(empty=0.0))
    bt = table.cuda()
    p = c.params(num_queries=1)
    ws = workspace(p)
    lo = torch.zeros(c.batch, c.hkv, c.nb_cap, c.dim, dtype=kv, device="cuda")
    hi = torch.zeros_like(lo)
    freq = inv_freq(c.dim).cuda()
    at = 0
    for step in (1, 30, 1, 1, 31, 200, 7, 229):
        rows = c.batch * step
        kn, vn = (c.normal(f"{what}{at}", rows, c.hkv, c.dim).cuda() for what in "kv")
        lens = torch.full((c.batch,), at, dtype=torch.int32, device="cuda")
        B.sparse_attn_append_kv(p, None, kn, vn, freq, None, k, v, bt, ws, seq_lens=lens, kmin=lo, kmax=hi)
        at += step
        pn = c.params(n_tokens=at, num_queries=1)
        rmin, rmax = torch.zeros_like(lo), torch.zeros_like(hi)
        B.sparse_attn_build_meta(pn, k, bt, rmin, rmax, None, ws)
        assert B.sparse_attn_get_device_error(ws) == 0
        nb = -(-at // c.block)
        assert torch.equal(lo[:, :, :nb], rmin[:, :, :nb]) and torch.equal(hi[:, :, :nb], rmax[:, :, :nb])
    assert at == c.context
    # without lengths: the rows end at n_tokens
    k2, v2 = k.clone(), v.clone()
    B.sparse_attn_append_kv(c.params(num_queries=1), None, kn, vn, freq, None, k2, v2, bt, ws)
    assert torch.equal(k2, k) and torch.equal(v2, v)


def test_bad_lengths_rows_and_pages_are_reported_and_skipped():
    c = Case(batch=4, lens=(10, 10, 10, 10), context=300, drafts=5)
    table = c.block_table()
    rows = 20
    kn, vn = c.normal("k", rows, c.hkv, c.dim).cuda(), c.normal("v", rows, c.hkv, c.dim).cuda()
    p, freq = c.params(), inv_freq(c.dim).cuda()
    ws = workspace(p)

    def attempt(lens=(10, 10, 10, 10), cu=(0, 5, 10, 15, 20), bt=table):
        k, v = (x.cuda() for x in c.pools(empty=0.5))
        B.sparse_attn_append_kv(p, None, kn, vn, freq, None, k, v, bt.cuda(), ws,
                                cu_rows=torch.tensor(cu, dtype=torch.int32, device="cuda"),
                                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
        flags = B.sparse_attn_get_device_error(ws)
        written = []
        for b in range(4):
            pg, off = place(c, table, b, torch.arange(10, 15))
            written.append(bool((k.cpu()[pg, :, off] != 0.5).any()))
        return flags, written, int((k != 0.5).any(-1).sum())

    full = 5 * c.hkv
    assert attempt() == (0, [True] * 4, 4 * full)
    for lens in ((10, -2, 10, 10), (10, c.capacity - 4, 10, 10), (10, 2**31 - 1, 10, 10)):
        flags, written, n = attempt(lens=lens)
        assert flags == B.ERR_LENGTH and written == [True, False, True, True] and n == 3 * full
    for cu in ((0, 5, 3, 15, 20), (0, 5, 10, 15, 21), (-3, 2, 10, 15, 20), (0, 5, 10, 15, 2**31 - 1)):
        flags, _, _ = attempt(cu=cu)
        assert flags == B.ERR_LENGTH
    bad = table.clone()
    bad[2, 0] = c.pages
    flags, written, n = attempt(bt=bad)
    assert flags == B.ERR_PAGE and written == [True, True, False, True] and n == 3 * full
    bad[2, 0] = -1
    assert attempt(bt=bad)[0] == B.ERR_PAGE
    assert attempt()[0] == 0


def test_another_stream_and_a_replayed_graph():
    """A captured append follows lengths that change between replays."""
    c = Case(batch=2, lens=(10, 40), drafts=30)
    table = c.block_table().cuda()
    k, v = (x.cuda() for x in c.pools(empty=0.0))
    p, freq = c.params(), inv_freq(c.dim).cuda()
    ws = workspace(p)
    kn, vn = c.normal("k", 2, c.hkv, c.dim).cuda(), c.normal("v", 2, c.hkv, c.dim).cuda()
    lens = torch.tensor(c.all_lens, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        B.sparse_attn_append_kv(p, None, kn, vn, freq, None, k, v, table, ws, seq_lens=lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.sparse_attn_append_kv(p, None, kn, vn, freq, None, k, v, table, ws, seq_lens=lens)
        lens += 1
    for step in range(3):
        kn.copy_(c.normal(f"k{step}", 2, c.hkv, c.dim))
        graph.replay()
        k2, v2 = k.clone(), v.clone()
        at = torch.tensor([10 + step, 40 + step], dtype=torch.int32, device="cuda")
        B.sparse_attn_append_kv(p, None, kn, vn, freq, None, k2, v2, table, ws, seq_lens=at)
        assert torch.equal(k, k2) and torch.equal(v, v2)
        for b in range(2):
            pg, off = place(c, table.cpu(), b, torch.tensor([10 + step, 40 + step])[b:b + 1])
            rk, mk = rotate(kn[b:b + 1].cpu(), at[b:b + 1].cpu(), freq.cpu(), B.ROTATE_HALVES)
            got = k.cpu()[pg, :, off].double()
            assert ((got - rk).abs() <= rotation_bound(rk, mk, c.kv)).all()
    assert lens.tolist() == [13, 43] and B.sparse_attn_get_device_error(ws) == 0
