"""Draft-tree attention over selections where the single-query kernels do not fit: fp32 K/V with large
pages, several queries over fp32 K/V, two-level selections of several queries."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, random_tree, tree_exact
from tests.test_gpu_tree import call, check, selection

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


CASES = {
    "fp32_bs128_one": (Case(batch=2, drafts=1, topk=3, block=128, context=900, lens=(900, 130), dtype=F32, kv=F32), {}),
    "fp32_bs128": (Case(batch=2, drafts=5, topk=3, block=128, context=900, lens=(900, 130), dtype=F32, kv=F32), {}),
    "fp32_kv_bs64": (Case(batch=2, drafts=20, topk=5, block=64, context=900, lens=(700, 65), kv=F32), {}),
    "two_level": (Case(batch=2, drafts=9, topk=6, block=32, context=900, lens=(900, 40)),
                  dict(two_level=True, coarse_block=128, topk_coarse=3)),
    "two_level_fp32": (Case(batch=2, drafts=3, topk=6, block=32, context=900, lens=(900, 40), dtype=F32, kv=F32),
                       dict(two_level=True, coarse_block=128, topk_coarse=3)),
}


@pytest.mark.parametrize("name", CASES)
def test_selections_that_other_calls_do_not_take(name):
    c, over = CASES[name]
    p = c.params(**over)
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    see, sel = random_tree(c), selection(c)
    assert sel[0].shape[-1] == B.sparse_attn_sel_stride(p)
    out, ws = call(c, q, pools, table, see, sel, p=p)
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, *tree_exact(c, q, pools, table, see, *sel))
