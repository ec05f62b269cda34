"""Committing where no sequence has a path."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import Case
from tests.test_gpu_tree import workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def test_commit_without_any_path():
    """path_stride 0: nothing is accepted, the lengths are handed on."""
    c = Case(batch=3, drafts=4, lens=(10, 20, -1))
    table = c.block_table()
    k, v = c.fill(c.pools(empty=0.5), table)
    gk, gv = k.cuda(), v.cuda()
    new = torch.full((3,), 77, dtype=torch.int32, device="cuda")
    ws = workspace(c.params())
    B.sparse_attn_commit_drafts(c.params(), torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                                torch.zeros(3, dtype=torch.int32, device="cuda"), gk, gv, table.cuda(), new, ws,
                                seq_lens=torch.tensor(c.all_lens, dtype=torch.int32, device="cuda"))
    assert new.tolist() == [10, 20, -1] and torch.equal(gk.cpu(), k) and torch.equal(gv.cpu(), v)
    assert B.sparse_attn_get_device_error(ws) == 0
    B.sparse_attn_commit_drafts(c.params(), torch.empty(3, 0, dtype=torch.int32, device="cuda"),
                                torch.tensor([0, 1, 0], dtype=torch.int32, device="cuda"), gk, gv, table.cuda(), new, ws,
                                seq_lens=torch.tensor(c.all_lens, dtype=torch.int32, device="cuda"))
    assert new.tolist() == [10, 20, -1] and B.sparse_attn_get_device_error(ws) == B.ERR_LENGTH
