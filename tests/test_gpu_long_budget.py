"""A LongContextDecoder that was made without a budget."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from query_guided_block_gb300.decoder import LongContextDecoder

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def test_weights_and_eviction_need_a_budget():
    p = B.make_params(1, 8, 2, 64, 60, 16, 10, 0, 1, num_queries=4, capacity_tokens=64)
    dec = LongContextDecoder(p, torch.tensor([20], dtype=torch.int32, device="cuda"))
    pool = torch.zeros(10, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    q, k = (torch.randn(4, h, 64, device="cuda").to(torch.bfloat16) for h in (8, 2))
    dec.append(None, k, k, None, None, pool, pool.clone(), table)
    with pytest.raises(ValueError, match="keep_tokens: 0"):
        dec.decode_weighed(q.view(1, 4, 8, 64), pool, pool, table)
    with pytest.raises(ValueError, match="keep_tokens: 0"):
        dec.evict(0, 0, pool, pool, table, table[:, :1])
    assert dec.device_error() == 0
