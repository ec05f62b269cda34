"""What weighed attention's workspace holds (no GPU needed)."""
import pytest
import torch

from query_guided_block_gb300 import binding as B

BF, F32 = torch.bfloat16, torch.float32


def size(batch, hq, hkv, drafts, capacity, q=BF, kv=BF):
    return B.sparse_attn_weigh_workspace_size(B.make_params(batch, hq, hkv, 128, capacity - drafts, 64, 1000, 0, 1, kv_dtype=kv,
                                                            q_dtype=q, num_queries=drafts, capacity_tokens=capacity))


@pytest.mark.parametrize("batch, hq, hkv, drafts, q, kv", [(16, 32, 8, 1, BF, BF), (16, 32, 8, 4, BF, BF), (4, 32, 8, 32, F32, BF),
                                                           (4, 32, 8, 32, F32, F32), (4, 32, 8, 32, BF, F32), (3, 8, 1, 1, BF, BF)])
def test_kept_scores_are_four_bytes_a_row_and_token(batch, hq, hkv, drafts, q, kv):
    sizes = [size(batch, hq, hkv, drafts, n, q, kv) for n in (6400, 64000, 128000)]
    for (a, b), tokens in zip(zip(sizes, sizes[1:]), (57600, 64000)):
        assert abs(b - a - 4 * batch * drafts * hq * tokens) <= 256


@pytest.mark.parametrize("batch, hq, hkv, drafts, most", [(4, 32, 8, 8, 256 << 20), (64, 32, 8, 5, 256 << 20), (4, 32, 8, 32, 3 << 20),
                                                          (64, 64, 8, 64, 3 << 20)])
def test_bf16_beyond_16_rows_keeps_a_bounded_number(batch, hq, hkv, drafts, most):
    short = size(batch, hq, hkv, drafts, 64 + drafts)                      # next to no scores
    for capacity in (1000, 20000, 130000, 400000):
        assert size(batch, hq, hkv, drafts, capacity) <= short + most
