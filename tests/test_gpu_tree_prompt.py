"""Draft-tree attention with as many drafts as it takes: chunks of prompts as chains, and trees of that
size, on both kernels."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case, random_tree, tree_exact
from tests.test_gpu_tree import call, check

pytestmark = pytest.mark.gpu
F32 = torch.float32

CASES = {
    "tensor_core_1024": Case(batch=2, hq=4, hkv=2, dim=64, drafts=1024, context=100, lens=(77, 0), block=16),
    "tensor_core_g8": Case(batch=2, hq=8, hkv=1, drafts=300, context=200, lens=(200, 33), block=64),
    "warp_level_993": Case(batch=1, hq=1, hkv=1, dim=64, drafts=993, context=30, lens=(29,), block=8),
    "fp32_1024": Case(batch=1, hq=2, hkv=1, dim=64, drafts=1024, context=30, lens=(5,), dtype=F32, kv=F32),
    "fp32_q_600": Case(batch=2, hq=2, hkv=1, drafts=600, context=70, lens=(70, -1), dtype=F32),
}


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


@pytest.mark.parametrize("masked", ["tree", "chain"])
@pytest.mark.parametrize("name", CASES)
def test_many_drafts(name, masked):
    c = CASES[name]
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    see = random_tree(c) if masked == "tree" else None
    out, ws = call(c, q, pools, table, see)
    assert B.sparse_attn_get_device_error(ws) == 0
    check(c, out, *tree_exact(c, q, pools, table, see))
