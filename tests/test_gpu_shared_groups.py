"""Groups of sequences out of order, which may overlap: reported, whatever they name."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def call(batch, cuts, prefix, n, drafts=1, dtype=BF, hq=32, hkv=8, block=64, lens=None):
    """All sequences over the same page; out is 5 before the call."""
    groups, cap = len(cuts) - 1, n + drafts
    p = B.make_params(batch, hq, hkv, 64, n, block, 1, 0, 1, kv_dtype=dtype, q_dtype=dtype, num_queries=drafts, capacity_tokens=cap)
    pools = [torch.ones(1, hkv, block, 64, dtype=dtype, device="cuda") for _ in range(2)]
    table = torch.zeros(batch, -(-cap // block), dtype=torch.int32, device="cuda")
    q = torch.ones(batch, drafts, hq, 64, dtype=dtype, device="cuda")
    out = torch.full(q.shape, 5.0, device="cuda")
    ws = torch.full((B.sparse_attn_shared_workspace_size(p, groups),), 0xAB, dtype=torch.uint8, device="cuda")
    B.sparse_attn_workspace_init(ws[:256])
    prefixes = prefix if isinstance(prefix, list) else [prefix] * groups
    B.sparse_attn_shared_decode(p, q, *pools, table, int32(cuts), int32(prefixes), out, ws,
                                seq_lens=None if lens is None else int32(lens))
    return B.sparse_attn_get_device_error(ws), out


CALLS = {
    "one_launch": dict(batch=4, cuts=[0, 4, 0, 4], prefix=100, n=200),
    "one_launch_fp32": dict(batch=4, cuts=[0, 4, 0, 4, 0, 4], prefix=100, n=200, dtype=F32),
    "two_launches_fp32": dict(batch=40, cuts=[0, 40, 0, 40], prefix=100, n=200, dtype=F32),
    "tensor_cores": dict(batch=40, cuts=[0, 40, 0, 40], prefix=3000, n=3200),
    "many_groups": dict(batch=300, cuts=[0, 300] * 200, prefix=10, n=20, hq=4, hkv=1),
    "one_sequence_twice": dict(batch=3, cuts=[0, 3, 2, 3], prefix=50, n=100),
    "backwards": dict(batch=3, cuts=[3, 2, 1, 0], prefix=50, n=100),
    "far_apart": dict(batch=600, cuts=[0, *range(1, 600), 600, 599], prefix=50, n=100, hq=4, hkv=1),
}


@pytest.mark.parametrize("name", CALLS)
def test_groups_out_of_order_are_reported(name):
    flags, _ = call(**CALLS[name])
    assert flags == B.ERR_LENGTH


@pytest.mark.parametrize("cuts, bad", [([0, 1024] * 512 + [0], True), ([0] + [1024] * 1024, False), (list(range(1025)), False)])
def test_groups_whose_tiles_are_more_than_32_bits_hold(cuts, bad):
    """128K tokens x 1024 sequences x 16 rows x 8 heads x 512 groups that are all the batch make 2^33 tiles of 64 tokens x
    16 rows; without the overlap they are 2^24.  Out of order, every sequence is by itself then: values of one
    everywhere give one but for the rounding of a total and a division, which 2^-11 covers."""
    flags, out = call(batch=1024, cuts=cuts, prefix=131000, n=131072, drafts=4)
    assert flags == (B.ERR_LENGTH if bad else 0) and ((out - 1).abs() <= 2.0 ** -11).all()


@pytest.mark.parametrize("kw", [dict(batch=4, prefix=100, n=200), dict(batch=40, prefix=3000, n=3200),
                                dict(batch=40, prefix=100, n=200, dtype=F32), dict(batch=300, prefix=10, n=20, hq=4, hkv=1)])
def test_groups_that_cover_the_batch_are_not(kw):
    """Every group of one, all in one, empty ones between them; values of one everywhere: every row is one but for
    the rounding of its sums and its division, a few units 2^-24 for each of up to 3200 tokens, at most 2^-11."""
    n = kw["batch"]
    for cuts in (list(range(n + 1)), [0, n], [0, 0, 1, 1, n, n], [0, n // 2, n // 2, n]):
        flags, out = call(cuts=cuts, **kw)
        assert flags == 0 and ((out - 1).abs() <= 2.0 ** -11).all()


def test_members_that_are_inactive_count_as_members():
    flags, out = call(batch=4, cuts=[0, 4], prefix=100, n=200, lens=[-1, 150, -1, 100])
    assert flags == 0 and (out[[0, 2]] == 5.0).all() and ((out[[1, 3]] - 1).abs() <= 2.0 ** -11).all()


def test_the_next_call_is_not_concerned():
    """One workspace, a bad call and a good one."""
    p = B.make_params(4, 32, 8, 64, 200, 64, 1, 0, 1, num_queries=1, capacity_tokens=201)
    pools = [torch.ones(1, 8, 64, 64, dtype=BF, device="cuda") for _ in range(2)]
    table, q = torch.zeros(4, 4, dtype=torch.int32, device="cuda"), torch.ones(4, 1, 32, 64, dtype=BF, device="cuda")
    ws = torch.full((B.sparse_attn_shared_workspace_size(p, 3),), 0xAB, dtype=torch.uint8, device="cuda")
    B.sparse_attn_workspace_init(ws[:256])
    for cuts, bad in (([0, 4, 0, 4], True), ([0, 1, 4, 4], False), ([0, 4, 0, 4], True), ([0, 4, 4, 4], False)):
        out = torch.full(q.shape, 5.0, device="cuda")
        B.sparse_attn_shared_decode(p, q, *pools, table, int32(cuts), int32([100, 64, 70]), out, ws)
        assert B.sparse_attn_get_device_error(ws) == (B.ERR_LENGTH if bad else 0)
        assert bad or ((out - 1).abs() <= 2.0 ** -11).all()
