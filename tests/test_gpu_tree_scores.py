"""Draft-tree attention where scores are large: of either sign, from 2e4 to beyond 2^31 in base 2, on
both kernels.  Scores are whole numbers that every partial sum holds exactly, so the weights are known
well whatever their size, and a row's tokens lie close enough together for several to count."""
import math

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import U, Case, chain_mask, place, random_tree, tree_exact
from tests.test_gpu_tree import call

pytestmark = pytest.mark.gpu
F32 = torch.float32
LONG = 8000                                       # n_tokens of the problems with more than 16 rows

KINDS = {
    "r28": dict(drafts=7, context=LONG), "r28_d64": dict(drafts=7, context=LONG, dim=64),
    "r64": dict(drafts=16, context=LONG), "r64_d64": dict(drafts=16, context=LONG, dim=64),
    "r100": dict(drafts=25, context=LONG), "r100_d64": dict(drafts=25, context=LONG, dim=64),
    "r180": dict(drafts=45, context=LONG),
    "few": dict(drafts=3), "small_rows": dict(drafts=9), "fp32": dict(drafts=7, dtype=F32, kv=F32),
    "fp32_rows": dict(drafts=20, dtype=F32, kv=F32, dim=64), "fp32_q": dict(drafts=7, dtype=F32),
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def scored(c, sign):
    """Queries and keys whose scores are sign * 32 a (D - 1) + d with a in 33 .. 64 a query row and d
    in 0 .. 16 a token; every value fits bf16, every partial sum 24 bits."""
    g = c.gen("scored")
    flip = torch.where(torch.rand(c.dim, generator=g) < 0.5, -1.0, 1.0)
    flip[0] = 1.0
    a = torch.randint(33, 65, (c.batch, c.drafts, c.hq, 1), generator=g).float()
    q = a * flip
    q[..., 0] = 1.0
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    for b, n in enumerate(c.all_lens):
        t = torch.arange(n + c.drafts)
        page, off = place(c, table, b, t)
        k = (sign * 32 * flip).expand(len(t), c.hkv, c.dim).clone()
        k[..., 0] = torch.randint(0, 17, (len(t), c.hkv), generator=g).float()
        pools[0][page, :, off] = k.to(c.kv)
    return q.to(c.dtype), table, pools


def expected(c, q, pools, table, see, scale):
    """Attention in 64 bits and how far an fp32 output may be off.

    Scores are exact.  What the exponent of a weight is off by, relative to the row's largest: the
    scale in base 2 is rounded twice (2 U of the distance), the distance from the reference once (U of
    it; the reference lies at most 6 below the largest: U (far + 6)), exp2 gives 2^-22.  At 1e11 and
    beyond the next score is 2^19 away: only equal ones of the largest count.
    The weighted sum: at most 24 matrix steps a tile of two units 2^-23 and 8 tiles and shares of half
    a unit, the total likewise; fp32 K/V keep 22 bits of weights and values (2^-22 each, and as much
    for the product left out).  A last division and product."""
    out = torch.zeros(c.batch, c.drafts, c.hq, c.dim, dtype=torch.float64)
    bound = torch.zeros_like(out)
    G = c.hq // c.hkv
    for b, n in enumerate(c.all_lens):
        t = torch.arange(n + c.drafts)
        page, off = place(c, table, b, t)
        for h in range(c.hq):
            k, v = pools[0][page, h // G, off].double(), pools[1][page, h // G, off].double()
            s = q[b, :, h].double() @ k.T * scale
            ok = torch.cat([torch.ones(c.drafts, n, dtype=torch.bool), see[b]], 1)
            s = s.masked_fill(~ok, -math.inf)
            far = (s.amax(-1, keepdim=True) - s).masked_fill(~ok, 0.0)
            p = torch.softmax(s, -1)
            out[b, :, h] = p @ v
            err = U * (3 * far + 6) + 2 ** -22
            mag = p @ v.abs()
            steps = (24 + 8) * 2 ** -22 + (3 * 2 ** -22 if c.kv == F32 else 0)
            bound[b, :, h] = (p * err) @ v.abs() + (p * err).sum(-1, keepdim=True) * mag + (2 * steps + 4 * U) * mag
    return out, bound


@pytest.mark.parametrize("logit", [2e4, 1e5, 3e6, 1e11, 1e30])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("kind", KINDS)
def test_large_scores_of_either_sign(kind, sign, logit):
    c = Case(batch=3, lens=(37, 300, 121), block=16, **KINDS[kind])
    q, table, pools = scored(c, sign)
    scale = float(torch.tensor(logit / (64 * 32 * (c.dim - 1)), dtype=F32))
    see = random_tree(c)
    out, ws = call(c, q, pools, table, see, p=c.params(softmax_scale=scale))
    assert B.sparse_attn_get_device_error(ws) == 0
    exact, bound = expected(c, q, pools, table, see, scale)
    err = (out.cpu().double() - exact).abs()
    assert (err <= bound).all(), f"{int((~(err <= bound)).any(-1).sum())} of {err[..., 0].numel()} rows are wrong"


def test_large_scores_split_between_parts():
    """A long context whose largest scores lie apart: shares are joined by their references."""
    for kind in ("r28", "r64", "r100", "few", "fp32"):
        kw = {**KINDS[kind], "context": 5000}
        c = Case(batch=2, lens=(4500, 700), block=64, **kw)
        q, table, pools = scored(c, 1)
        scale = float(torch.tensor(1e5 / (64 * 32 * (c.dim - 1)), dtype=F32))
        see = chain_mask(c.drafts).expand(c.batch, -1, -1)
        out, ws = call(c, q, pools, table, p=c.params(softmax_scale=scale))
        assert B.sparse_attn_get_device_error(ws) == 0
        exact, bound = expected(c, q, pools, table, see, scale)
        assert ((out.cpu().double() - exact).abs() <= bound + 64 * U * exact.abs().amax(-1, keepdim=True)).all(), kind


@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_see_huge_keys(kind):
    """Two drafts with keys of 1e30: a query that sees them attends to them alone (equal scores share),
    or, where its score is as low as that, not at all."""
    c = Case(batch=3, lens=(37, 300, 121), block=16, **KINDS[kind])
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    see = random_tree(c)
    odd = [c.drafts // 2, c.drafts - 1]
    without = see.clone()
    without[:, :, odd] = False
    exact, bound = tree_exact(c, q, pools, table, without)
    for b, n in enumerate(c.all_lens):
        for j in odd:
            page, off = place(c, table, b, torch.tensor([n + j]))
            pools[0][page, :, off] = 1e30
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    met = up = 0
    for b, n in enumerate(c.all_lens):
        page, off = place(c, table, b, torch.arange(n, n + c.drafts))
        v = pools[1][page, :, off].double()                        # [Q, Hkv, D]
        for i in range(c.drafts):
            mine = [j for j in odd if see[b, i, j]]
            if not mine:
                continue
            met += 1
            for h in range(c.hq):
                total = float(q[b, i, h].double().sum())
                got = out[b, i, h].cpu().double()
                assert torch.isfinite(got).all()
                if abs(total) < 1e-2:             # its sign is within the rounding of the sum
                    continue
                if total < 0:
                    assert ((got - exact[b, i, h]).abs() <= bound[b, i, h]).all()
                else:
                    up += 1
                    want = v[mine, h // (c.hq // c.hkv)].mean(0)
                    # equal weights: a product and a sum of two, the total, the division
                    assert ((got - want).abs() <= 8 * 2 ** -22 * v[mine, h // (c.hq // c.hkv)].abs().mean(0) + 1e-30).all()
    assert met > 0 and up > 0
