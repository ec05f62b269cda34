"""What draft-tree attention promises beyond fp32 accuracy in general: weights enter the product with
all their 24 bits, and sums over long contexts do not drift.  Scores are whole numbers here that
every partial sum holds exactly, and all values are positive, so that neither hides the other; each
bound is shown to catch the mistake that it is for, planted in the 64-bit side."""
import math

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import U, Case, pack_mask, place
from tests.test_gpu_tree import call, workspace

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LONG = 8000                                       # n_tokens of the problems that the tensor-memory kernel takes
SCALE = 1 / 32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def whole(c, what, *shape):
    return torch.randint(-3, 4, shape, generator=c.gen(what)).float()


def weight_error(far):
    """Relative error of a weight at that base-2 distance from the row's largest: the scale is rounded
    once (1/32 is exact), the distance from the reference, which is at most 6 below the largest, once
    (U each), and exp2 gives 2^-22."""
    return math.log(2) * U * (2 * far + 6) + 2 ** -22


FEW = {
    "r32": Case(batch=3, hq=2, hkv=2, drafts=32, context=LONG, lens=(0, 0, 0), block=8, topk=1001),
    "r28_g4": Case(batch=3, hq=8, hkv=2, drafts=7, context=LONG, lens=(0, 0, 0), block=8, topk=1001),
    "r64": Case(batch=3, hq=2, hkv=2, drafts=64, context=LONG, lens=(0, 0, 0), block=8, topk=1001),
    "r64_d64": Case(batch=3, hq=2, hkv=2, dim=64, drafts=64, context=LONG, lens=(0, 0, 0), block=8, topk=1001),
    "r32_d64": Case(batch=3, hq=2, hkv=2, dim=64, drafts=32, context=LONG, lens=(0, 0, 0), block=8, topk=1001),
    "r128": Case(batch=3, hq=2, hkv=2, drafts=128, context=LONG, lens=(0, 0, 0), block=8, topk=1001),
    "r128_d64": Case(batch=3, hq=2, hkv=2, dim=64, drafts=128, context=LONG, lens=(0, 0, 0), block=8, topk=1001),
    "few": Case(batch=8, hq=8, hkv=2, drafts=4, lens=(0,) * 8, block=8),
    "small_rows": Case(batch=2, hq=2, hkv=2, drafts=64, lens=(0, 0), block=8),
    "fp32_q": Case(batch=2, hq=2, hkv=2, drafts=64, lens=(0, 0), block=8, dtype=F32),
    "fp32": Case(batch=2, hq=2, hkv=2, drafts=64, lens=(0, 0), block=8, dtype=F32, kv=F32),
    "fp32_few": Case(batch=8, hq=8, hkv=2, dim=64, drafts=4, lens=(0,) * 8, block=8, dtype=F32, kv=F32),
}


@pytest.mark.parametrize("shift", [0, 5, 10, 13])
@pytest.mark.parametrize("name", FEW)
def test_weights_keep_their_bits(name, shift):
    """No context and queries that see two drafts each, so that few roundings are left.  `shift`
    selected blocks behind the context move the drafts to other places of the tile."""
    c = FEW[name]
    table = c.block_table()
    pools = c.pools()
    for b in range(c.batch):
        page, off = place(c, table, b, torch.arange(c.drafts))
        pools[0][page, :, off] = whole(c, f"k{b}", c.drafts, c.hkv, c.dim).to(c.kv)
        pools[1][page, :, off] = (1 + torch.rand(c.drafts, c.hkv, c.dim, generator=c.gen(f"v{b}"))).to(c.kv)
    q = whole(c, "q", c.batch, c.drafts, c.hq, c.dim).to(c.dtype)
    see = torch.eye(c.drafts, dtype=torch.bool).expand(c.batch, -1, -1).clone()
    other = torch.randint(0, c.drafts - 1, (c.batch, c.drafts), generator=c.gen("other"))
    other += (other >= torch.arange(c.drafts)).long()              # any but the query itself
    see.scatter_(2, other[..., None], True)
    sel = None
    p = c.params(softmax_scale=SCALE)
    if shift:
        width = B.sparse_attn_sel_stride(p)
        ids = torch.arange(width, dtype=torch.int32).expand(c.batch, c.hkv, width).contiguous()
        sel = (ids, torch.full((c.batch, c.hkv), min(shift, width), dtype=torch.int32))
    out, ws = call(c, q, pools, table, see, sel, p=p)
    assert B.sparse_attn_get_device_error(ws) == 0
    out = out.cpu().double()
    caught = 0.0
    G = c.hq // c.hkv
    for b in range(c.batch):
        page, off = place(c, table, b, torch.arange(c.drafts))
        for h in range(c.hq):
            k, v = pools[0][page, h // G, off].double(), pools[1][page, h // G, off].double()
            s = (q[b, :, h].double() @ k.T * SCALE).masked_fill(~see[b], -math.inf)
            far = ((s.amax(-1, keepdim=True) - s) / math.log(2)).masked_fill(~see[b], 0.0)
            w = torch.exp(s - s.amax(-1, keepdim=True))
            total = w.sum(-1, keepdim=True)
            exact = w @ v / total
            # Two weights; at most two matrix steps for each of three parts, off by two units 2^-23 each,
            # one merge of shares, the total, the division and its product half a unit each.  fp32 K/V:
            # weights and values keep 22 bits, and their small parts' product is left out.
            rel = 2 * (w / total * weight_error(far)).sum(-1, keepdim=True) + 6 * 2 ** -22 + 8 * U
            if c.kv == F32:
                rel = rel + 3 * 2 ** -22
            err = (out[b, :, h] - exact).abs() / exact
            assert (err <= rel).all(), f"off by {float((err / rel).max()):.3g} times the bound"
            # the mistake that this is for: weights of two bf16 parts
            cut = (torch.exp2(torch.ceil(s.amax(-1, keepdim=True) / math.log(2)) * -1) * torch.exp(s)).float()
            one = (cut.view(torch.int32) & -65536).view(F32)
            two = ((cut - one).view(torch.int32) & -65536).view(F32)
            planted = (one.double() + two.double()) @ v / cut.double().sum(-1, keepdim=True)
            caught = max(caught, float(((planted - exact).abs() / exact / rel).max()))
    if c.kv == BF:
        assert caught > 1.5, "the bound would let two parts pass"


DRIFT = {                                         # (heads a KV head, drafts, D, K/V, query type, tile, matrix steps a tile)
    "r28": (4, 7, 128, BF, BF, 128, 24), "r64": (4, 16, 128, BF, BF, 128, 24), "r128": (4, 32, 128, BF, BF, 128, 24),
    "r64_d64": (4, 16, 64, BF, BF, 128, 24), "few": (4, 2, 128, BF, BF, 64, 3), "fp32_q": (4, 8, 64, BF, F32, 64, 12),
    "fp32": (4, 8, 64, F32, F32, 64, 24),
}


@pytest.mark.parametrize("name", DRIFT)
def test_long_sums_do_not_drift(name):
    """As many sequences over one context of 16K tokens as fill the GPU, so that one CTA adds up a whole
    context (they share its pages).  A sum kept in the matrix unit is cut off at every step."""
    G, drafts, dim, kv, qt, tile, steps = DRIFT[name]
    n, block = 16384, 64
    batch = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    c = Case(batch=batch, hq=G, hkv=1, dim=dim, block=block, context=n, drafts=drafts, dtype=qt, kv=kv)
    ctx = n // block
    pages = ctx + batch
    table = torch.empty(batch, ctx + 1, dtype=torch.int32)
    table[:, :ctx] = torch.randperm(ctx, generator=c.gen("table"))
    table[:, ctx] = ctx + torch.arange(batch)
    k = whole(c, "k", pages, 1, block, dim).to(kv)
    v = (1 + torch.rand(pages, 1, block, dim, generator=c.gen("v"))).to(kv)
    q = whole(c, "q", batch, drafts, G, dim).to(qt)
    p = c.params(num_pages=pages, softmax_scale=SCALE)
    ws = workspace(p)
    out = torch.empty(batch, drafts, G, dim, device="cuda")
    see = torch.eye(drafts, dtype=torch.bool).expand(batch, -1, -1)
    B.sparse_attn_tree_decode(p, q.cuda(), k.cuda(), v.cuda(), table.cuda(), out, ws, tree_mask=pack_mask(see).cuda())
    assert B.sparse_attn_get_device_error(ws) == 0
    tiles = -(-n // tile)
    # A tile's product: its steps, two units 2^-23 each, of a running sum.  Sums over the tiles (of the
    # output and of the total) and over a thread's weights round to nearest, each by at most U of a
    # running sum: independent errors of deviation U / sqrt(3), eight deviations allowed.
    rounding = 8 / math.sqrt(3) * U * (2 * math.sqrt(tiles) + math.sqrt(tile / 4))
    for b in (0, 1, batch // 2, batch - 1):
        page = table[b].long()
        kk, vv = k[page].flatten(0, 2).double(), v[page].flatten(0, 2).double()
        kk, vv = kk[: n + drafts], vv[: n + drafts]
        ok = torch.cat([torch.ones(drafts, n, dtype=torch.bool), see[b]], 1)[:, None].expand(-1, G, -1)
        s = (q[b].double() @ kk.T * SCALE).masked_fill(~ok, -math.inf)
        far = ((s.amax(-1, keepdim=True) - s) / math.log(2)).masked_fill(~ok, 0.0)
        w = torch.softmax(s, -1)
        exact = w @ vv
        rel = 2 * (w * weight_error(far)).sum(-1, keepdim=True) + steps * 2 ** -22 + rounding + 8 * U
        if kv == F32:
            rel = rel + 3 * 2 ** -22
        err = (out[b].cpu().double() - exact).abs() / exact
        assert (err <= rel).all(), f"off by {float((err / rel).max()):.3g} times the bound"
    # the mistake that this is for: the same sums cut to 24 bits at every step of the matrix unit
    x = (w[0, 0, :n, None] / w[0, 0].max() * vv[:n, :4]).view(n // 16, 16, 4).sum(1)
    if steps < 12:
        x = x[::4]
    x = x.repeat_interleave(3, 0) / 3                              # three parts' products
    total = torch.zeros(4, dtype=torch.float64)
    for term in x:
        total += term
        unit = torch.exp2(torch.floor(torch.log2(total)) - 23)
        total = torch.floor(total / unit) * unit
    drift = ((x.sum(0) - total) / x.sum(0)).max()
    assert drift > 1.2 * float(rel[0, 0]), "the bound would let a running sum pass"
