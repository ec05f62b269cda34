"""One workspace under problems of different shapes, in stream order: every result has the bits that a
workspace of its own gives."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case
from tests.test_gpu_tree import call

pytestmark = pytest.mark.gpu
F32 = torch.float32

# 400 items of few rows, most of them split between CTAs; one long sequence; tensor-memory items;
# an fp32 batch; 300 items of which the last CTA joins the parts
PROBLEMS = {
    "many": Case(batch=200, hq=8, hkv=2, dim=64, block=16, context=1400, drafts=1, lens=tuple(600 + 4 * i for i in range(200))),
    "one": Case(batch=1, hq=8, hkv=2, drafts=1, context=6000),
    "rows": Case(batch=20, hq=16, hkv=4, drafts=8, context=3000, lens=tuple(3000 - 137 * i for i in range(20))),
    "fp32": Case(batch=75, hq=4, hkv=4, dim=64, drafts=2, context=900, dtype=F32, kv=F32, lens=tuple(900 - 11 * (i % 40) for i in range(75))),
    "three": Case(batch=3, hq=8, hkv=1, drafts=2, context=9000, lens=(9000, 5000, 333)),
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def test_problems_of_different_shapes_share_a_workspace():
    data, alone, size = {}, {}, 0
    for name, c in PROBLEMS.items():
        table = c.block_table()
        pools = c.fill(c.pools(empty=0.0), table)
        data[name] = (c.normal("q", c.batch, c.drafts, c.hq, c.dim).cuda(), [x.cuda() for x in pools], table.cuda())
        alone[name], _ = call(c, *data[name])
        size = max(size, B.sparse_attn_tree_workspace_size(c.params()))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    B.sparse_attn_workspace_init(ws)
    names = list(PROBLEMS)
    order = names + names[::-1] + ["many", "rows", "many", "three", "rows", "one", "many", "fp32", "many"]
    for step, name in enumerate(order):
        c = PROBLEMS[name]
        got, _ = call(c, *data[name], ws=ws)
        assert torch.equal(got, alone[name]), f"call {step} ({name}): {int((got != alone[name]).any(-1).sum())} rows differ"
    assert B.sparse_attn_get_device_error(ws) == 0
