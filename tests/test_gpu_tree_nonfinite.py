"""Drafts that hold infinities and NaN reach every query that sees them, wherever the work is cut: a
share of the tokens whose scores are all NaN, a value whose weight is too small for fp32."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, chain_mask, place, tree_exact
from tests.test_gpu_tree import call

pytestmark = pytest.mark.gpu
F32 = torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


# Context lengths that put the drafts into a share of their own: 16 tokens (a warp's share of a tile
# with few rows), 2048 and 4096 (the only tile of the last part: 33 tiles in parts of two)
NAN_KEYS = {
    "warp_share": Case(batch=1, drafts=1, context=16, lens=(16,)),
    "warp_share_48": Case(batch=1, drafts=2, context=48, lens=(48,)),
    "warp_share_fp32": Case(batch=1, drafts=1, context=16, lens=(16,), dtype=F32, kv=F32),
    "last_part": Case(batch=1, drafts=1, hq=4, hkv=1, context=2048, lens=(2048,)),
    "last_part_fp32": Case(batch=1, drafts=2, hq=4, hkv=1, dim=64, context=2048, lens=(2048,), dtype=F32, kv=F32),
    "last_part_joined_apart": Case(batch=1, drafts=4, hq=4, hkv=1, context=2048, lens=(2048,)),
    "last_part_r28": Case(batch=1, drafts=7, hq=16, hkv=4, context=8000, lens=(4096,)),
    "last_part_r64": Case(batch=1, drafts=16, hq=16, hkv=4, context=8000, lens=(4096,)),
    "last_part_r100": Case(batch=1, drafts=25, hq=16, hkv=4, context=8000, lens=(4096,)),
    "last_part_r100_d64": Case(batch=1, drafts=25, hq=16, hkv=4, dim=64, context=8000, lens=(4096,)),
}


@pytest.mark.parametrize("name", NAN_KEYS)
def test_nan_keys_alone_in_a_share(name):
    """Every query sees one draft, its own, whose key is NaN for the odd drafts (the first one where
    there is only one): those rows are NaN, the others are as without."""
    c = NAN_KEYS[name]
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    see = torch.eye(c.drafts, dtype=torch.bool).expand(c.batch, -1, -1).clone()
    exact, bound = tree_exact(c, q, pools, table, see)
    bad = torch.arange(c.drafts) % 2 == (1 if c.drafts > 1 else 0)
    page, off = place(c, table, 0, c.all_lens[0] + torch.arange(c.drafts)[bad])
    pools[0][page, :, off] = NAN
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    out = out.cpu()
    assert torch.isnan(out[0, bad]).all(), f"{int((~torch.isnan(out[0, bad])).any(-1).sum())} rows lost their NaN"
    assert ((out.double() - exact).abs()[0, ~bad] <= bound[0, ~bad]).all()


VALUES = {
    "few": Case(batch=2, drafts=3, lens=(37, 300)),
    "few_parts": Case(batch=1, drafts=2, hq=4, hkv=1, context=2048, lens=(2048,)),
    "small_rows": Case(batch=1, drafts=9, lens=(37,)),
    "fp32": Case(batch=2, drafts=7, lens=(37, 300), dtype=F32, kv=F32, dim=64),
    "fp32_parts": Case(batch=1, drafts=2, hq=4, hkv=1, dim=64, context=2048, lens=(2048,), dtype=F32, kv=F32),
    "fp32_q": Case(batch=2, drafts=7, lens=(37, 300), dtype=F32),
    "r28": Case(batch=2, drafts=7, context=8000, lens=(37, 300)),
    "r28_parts": Case(batch=1, drafts=7, hq=16, hkv=4, context=8000, lens=(4096,)),
    "r64": Case(batch=2, drafts=16, context=8000, lens=(37, 300)),
    "r100": Case(batch=2, drafts=25, context=8000, lens=(37, 300)),
    "few_alone": Case(batch=1, drafts=2, hq=4, hkv=1, context=2048, lens=(2048,)),
    "joined_apart_alone": Case(batch=1, drafts=4, hq=4, hkv=1, context=2048, lens=(2048,)),
    "r28_alone": Case(batch=1, drafts=7, hq=16, hkv=4, context=8000, lens=(4096,)),
    "r64_alone": Case(batch=1, drafts=16, hq=16, hkv=4, context=8000, lens=(4096,)),
    "r100_alone": Case(batch=1, drafts=25, hq=16, hkv=4, context=8000, lens=(4096,)),
    "r100_parts": Case(batch=1, drafts=25, hq=16, hkv=4, dim=64, context=8000, lens=(4096,)),
}


@pytest.mark.parametrize("value", [INF, -INF, NAN])
@pytest.mark.parametrize("name", VALUES)
def test_values_whose_weight_is_too_small(name, value):
    """Draft 1 holds `value` in one channel and a key whose weight is far below 2^-149: that channel is
    not finite in the rows that see it, all others are as without the draft.  In the cases `alone` no
    query sees another draft, so that the last part of the row has no weight at all."""
    c = VALUES[name]
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    q[..., 5] = 4.0
    see = chain_mask(c.drafts).expand(c.batch, -1, -1).clone()
    if name.endswith("alone"):
        see[:] = False
        see[:, 1:, 1] = True
    for b, n in enumerate(c.all_lens):
        page, off = place(c, table, b, torch.tensor([n + 1]))
        key = torch.zeros(1, c.hkv, c.dim, dtype=c.kv)
        key[..., 5] = -2000.0                     # the score: -8000 / sqrt(D), below -700
        pools[0][page, :, off] = key
    exact, bound = tree_exact(c, q, pools, table, see)             # the draft's weight is 0 there
    for b, n in enumerate(c.all_lens):
        page, off = place(c, table, b, torch.tensor([n + 1]))
        row = pools[1][page, :, off]
        row[..., 3] = value
        pools[1][page, :, off] = row
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    out = out.cpu()
    rest = torch.arange(c.dim) != 3
    assert ((out.double() - exact).abs()[..., rest] <= bound[..., rest]).all()
    assert ((out.double() - exact).abs()[:, 0] <= bound[:, 0]).all()
    hit = ~torch.isfinite(out[:, 1:, :, 3])
    assert hit.all(), f"{int((~hit).sum())} of {hit.numel()} rows that see the draft are finite there"


@pytest.mark.parametrize("value", [0.5, INF])
@pytest.mark.parametrize("name", ["few", "few_parts", "small_rows", "r28", "r28_parts", "r64", "r100", "r100_parts"])
def test_scores_of_minus_infinity(name, value):
    """Draft 1 has a key that is infinite in one channel, and scores of -infinity: its weight is 0, also
    in rows that see nothing else; an infinite value of it shows in its channel all the same."""
    c = VALUES[name]
    if name == "few":
        c = Case(**{**c.__dict__, "lens": (0, 300)})               # the first sequence has no context
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    q[..., 5] = 4.0
    see = chain_mask(c.drafts).expand(c.batch, -1, -1).clone()
    if name == "few":
        see[0, 2] = torch.tensor([False, True, False])
    without = see.clone()
    without[:, :, 1] = False
    exact, bound = tree_exact(c, q, pools, table, without)
    for b, n in enumerate(c.all_lens):
        page, off = place(c, table, b, torch.tensor([n + 1]))
        key, row = pools[0][page, :, off], pools[1][page, :, off]
        key[..., 5], row[..., 3] = -INF, value
        pools[0][page, :, off], pools[1][page, :, off] = key, row
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    out = out.cpu()
    rest = torch.arange(c.dim) != 3 if value == INF else torch.ones(c.dim, dtype=torch.bool)
    assert ((out.double() - exact).abs()[..., rest] <= bound[..., rest]).all()
    if value == INF:
        assert not torch.isfinite(out[..., 3][see[:, :, 1]]).any()
