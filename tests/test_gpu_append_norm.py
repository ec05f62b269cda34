"""Head norms and positions of several axes on the way into the cache, against 64 bits; where nothing of
it is asked for, the bits of the plain append."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, place
from tests.long_reference import norm_bound, rms, rotate_axes

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def workspace():
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    B.sparse_attn_workspace_init(ws)
    return ws


def cuda(x):
    return None if x is None else x.cuda()


def run(c, counts, rotary=None, pairing=B.ROTATE_HALVES, axes=1, axis_of=None, norm="qk", per_head=False, fused=False,
        eps=1e-6, positions=None, scale=1.0, with_q=True, alias=False, box=True):
    rotary = c.dim if rotary is None else rotary
    lens, n = c.all_lens, sum(counts)
    table = c.block_table()
    k_pool, v_pool = c.fill(c.pools(empty=0.25), table, upto=[max(0, x) for x in lens])
    x = c.normal("qkv", n, (c.hq + 2 * c.hkv) * c.dim, dtype=F32).mul(scale).to(c.dtype)
    parts = [c.hq * c.dim, c.hkv * c.dim, c.hkv * c.dim]
    gx = x.cuda()
    if not fused:
        q, k, v = (y.contiguous().unflatten(1, (-1, c.dim)) for y in x.split(parts, 1))
        gq, gk, gv = (y.contiguous().unflatten(1, (-1, c.dim)) for y in gx.split(parts, 1))
    else:
        q, k, v = (y.unflatten(1, (-1, c.dim)) for y in x.split(parts, 1))
        gq, gk, gv = (y.unflatten(1, (-1, c.dim)) for y in gx.split(parts, 1))
    freq = 10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) / max(1, rotary // 2))
    qw = 1 + 0.3 * c.normal("qw", *((c.hq, c.dim) if per_head else (c.dim,)), dtype=F32) if "q" in norm else None
    kw = 1 + 0.3 * c.normal("kw", *((c.hkv, c.dim) if per_head else (c.dim,)), dtype=F32) if "k" in norm else None
    half = rotary // 2
    if axes > 1 and axis_of is None:
        axis_of = torch.arange(half) * axes // half if pairing == B.ROTATE_HALVES else torch.arange(half) % axes
    if axes > 1 and positions is None:
        positions = torch.randint(0, 70000, (axes, n), generator=c.gen("pos"))
    p = c.params()
    ws = workspace()
    g = dict(k=k_pool.cuda(), v=v_pool.cuda(), bt=table.cuda())
    kmin = torch.full((c.batch, c.hkv, c.nb_cap, c.dim), 7.0, dtype=c.kv)
    kmax = torch.full_like(kmin, -7.0)
    for b, old in enumerate(lens):
        for j in range(-(-max(0, old) // c.block)):
            t = torch.arange(j * c.block, min(old, (j + 1) * c.block))
            pg, off = place(c, table, b, t)
            kmin[b, :, j], kmax[b, :, j] = k_pool[pg, :, off].amin(0), k_pool[pg, :, off].amax(0)
    lo, hi = kmin.cuda(), kmax.cuda()
    q_out = gq if alias else torch.full((n, c.hq, c.dim), 9.0, dtype=c.dtype, device="cuda")
    cu = torch.tensor([0] + torch.tensor(counts).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    B.sparse_attn_append_kv_norm(
        p, gq if with_q else None, gk, gv, cuda(qw), cuda(kw), eps, freq.cuda() if rotary else None,
        q_out if with_q else None, g["k"], g["v"], g["bt"], ws, cu_rows=cu,
        seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
        positions=None if positions is None else positions.to(torch.int32).cuda(),
        axis_of=None if axes == 1 else axis_of.to(torch.int32).cuda(), pairing=pairing, kmin=lo if box else None,
        kmax=hi if box else None)
    assert B.sparse_attn_get_device_error(ws) == 0
    got_k, got_v = g["k"].cpu(), g["v"].cpu()
    want_k, want_v = k_pool.clone(), v_pool.clone()
    r = 0
    for b, (old, cnt) in enumerate(zip(lens, counts)):
        if old < 0 or cnt == 0:
            r += cnt
            continue
        rows = slice(r, r + cnt)
        t = torch.arange(old, old + cnt)
        at = t[None] if positions is None else (positions[:, rows] if axes > 1 else positions[None, rows])
        angle = at[axis_of.long() if axes > 1 else torch.zeros(half, dtype=torch.long)].t().double() * freq
        pg, off = place(c, table, b, t)
        nk = rms(k[rows], kw, eps) if kw is not None else k[rows].double()
        want, mag = rotate_axes(nk, angle, pairing)
        err = (got_k[pg, :, off].double() - want).abs()
        assert (err <= norm_bound(want, mag, c.kv)).all(), f"keys of sequence {b}: {err.max()}"
        want_k[pg, :, off], want_v[pg, :, off] = got_k[pg, :, off], v[rows].to(c.kv)
        if with_q:
            nq = rms(q[rows], qw, eps) if qw is not None else q[rows].double()
            want, mag = rotate_axes(nq, angle, pairing)
            err = (q_out[rows].cpu().double() - want).abs()
            assert (err <= norm_bound(want, mag, c.dtype)).all(), f"queries of sequence {b}: {err.max()}"
        for j in range(old // c.block, (old + cnt - 1) // c.block + 1):
            t = torch.arange(j * c.block, min(old + cnt, (j + 1) * c.block))
            pg, off = place(c, table, b, t)
            kmin[b, :, j], kmax[b, :, j] = want_k[pg, :, off].amin(0), want_k[pg, :, off].amax(0)
        r += cnt
    assert torch.equal(got_k, want_k) and torch.equal(got_v, want_v)       # nothing else changed
    if box:
        assert torch.equal(lo.cpu(), kmin) and torch.equal(hi.cpu(), kmax)


CASES = {
    "one_token": (Case(batch=1, lens=(131,), drafts=1, room=40), [1], {}),
    "ragged": (Case(batch=4, lens=(0, 31, 130, 5), context=130, room=200), [1, 70, 0, 133], dict(fused=True)),
    "inactive": (Case(batch=3, lens=(7, -1, 64), context=64, room=60), [9, 5, 33], {}),
    "queries_only": (Case(batch=2, lens=(3, 40), room=60), [5, 41], dict(norm="q")),
    "keys_only": (Case(batch=2, lens=(3, 40), room=60), [5, 41], dict(norm="k")),
    "no_queries": (Case(batch=2, lens=(3, 40), room=60), [5, 41], dict(norm="k", with_q=False)),
    "per_head": (Case(batch=2, lens=(3, 40), room=60), [5, 41], dict(per_head=True)),
    "no_rotation": (Case(batch=2, lens=(3, 40), room=60), [5, 41], dict(rotary=0)),
    "partial_pairs": (Case(batch=2, lens=(3, 40), room=60, dim=64, hq=4, hkv=4), [5, 41],
                      dict(rotary=32, pairing=B.ROTATE_PAIRS)),
    "fp32": (Case(batch=2, lens=(3, 40), room=60, dtype=F32, kv=F32), [5, 41], dict(axes=2)),
    "fp32_64": (Case(batch=2, lens=(3, 40), room=60, dtype=F32, kv=F32, dim=64), [5, 41], dict(fused=True, eps=1e-2)),
    "fp32_to_bf16": (Case(batch=2, lens=(3, 40), room=60, dtype=F32), [5, 41], dict(axes=3)),
    "bf16_to_fp32": (Case(batch=2, lens=(3, 40), room=60, kv=F32, dim=64), [5, 41], dict(axes=4, per_head=True)),
    "three_axes": (Case(batch=2, lens=(3, 40), room=200, hq=16, hkv=2), [101, 41], dict(axes=3, fused=True)),
    "axes_in_turn": (Case(batch=2, lens=(3, 40), room=60), [5, 41], dict(axes=3, pairing=B.ROTATE_PAIRS)),
    "eight_axes_no_norm": (Case(batch=2, lens=(3, 40), room=60), [5, 41], dict(axes=8, norm="")),
    "positions_of_one_axis": (Case(batch=2, lens=(3, 40), room=60), [5, 41],
                              dict(positions=torch.arange(46) * 1000003 % (1 << 22))),
    "in_place": (Case(batch=2, lens=(3, 40), room=60), [5, 41], dict(alias=True)),
    "no_box": (Case(batch=2, lens=(3, 40), room=60), [5, 41], dict(box=False)),
    "block_8": (Case(batch=2, lens=(3, 40), room=160, block=8), [77, 41], {}),
    "block_128": (Case(batch=2, lens=(3, 140), room=400, block=128), [277, 41], dict(axes=2)),
    "large": (Case(batch=1, lens=(3,), room=60, dtype=F32, kv=F32), [20], dict(scale=1e25)),     # squares past fp32
    "small": (Case(batch=1, lens=(3,), room=60, dtype=F32, kv=F32), [20], dict(scale=1e-12, eps=1e-30)),
    "large_bf16": (Case(batch=1, lens=(3,), room=60, dim=64), [20], dict(scale=3e37)),
}


@pytest.mark.parametrize("name", CASES)
def test_against_64_bits(name):
    c, counts, kw = CASES[name]
    run(c, counts, **kw)


def test_zero_rows_stay_zero():
    c = Case(batch=1, lens=(3,), room=60)
    run(c, [9], scale=0.0)


def test_without_norm_and_axes_it_is_the_append():
    c = Case(batch=2, lens=(3, 40), room=60)
    table = c.block_table().cuda()
    q, k, v = (c.normal(n, 46, h, c.dim).cuda() for n, h in (("q", c.hq), ("k", c.hkv), ("v", c.hkv)))
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).cuda()
    cu = torch.tensor([0, 5, 46], dtype=torch.int32, device="cuda")
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    got = []
    for norm in (False, True):
        pools = [x.cuda() for x in c.pools(empty=0.0)]
        out = torch.zeros_like(q)
        if norm:
            B.sparse_attn_append_kv_norm(c.params(), q, k, v, None, None, 0.0, freq, out, *pools, table, workspace(),
                                         cu_rows=cu, seq_lens=lens)
        else:
            B.sparse_attn_append_kv(c.params(), q, k, v, freq, out, *pools, table, workspace(), cu_rows=cu, seq_lens=lens)
        got.append([out, *pools])
    assert all(torch.equal(x, y) for x, y in zip(*got))


def test_an_axis_out_of_range_is_reported():
    c = Case(batch=1, lens=(3,), room=60)
    k = c.normal("k", 4, c.hkv, c.dim).cuda()
    pools = [x.cuda() for x in c.pools(empty=0.0)]
    axis = torch.zeros(64, dtype=torch.int32)
    axis[5], axis[9] = 2, -1
    ws = workspace()
    B.sparse_attn_append_kv_norm(c.params(), None, k, k, None, None, 0.0,
                                 torch.ones(64, dtype=torch.float64, device="cuda"), None, *pools, c.block_table().cuda(), ws,
                                 seq_lens=torch.tensor([3], dtype=torch.int32, device="cuda"),
                                 positions=torch.zeros(2, 4, dtype=torch.int32, device="cuda"), axis_of=axis.cuda())
    assert B.sparse_attn_get_device_error(ws) == B.ERR_LENGTH
