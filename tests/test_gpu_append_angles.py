"""Sines and cosines that an append rotates by, taken out of it with rows of ones and zeros."""
import math

import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from tests.draft_reference import U
from tests.test_gpu_tree import workspace

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


@pytest.mark.parametrize("first", [0, 100_000, 2_000_000, -70_000])
@pytest.mark.parametrize("pairing", [B.ROTATE_HALVES, B.ROTATE_PAIRS])
def test_angles_are_good_to_fp32(pairing, first):
    """A pair (1, 0) becomes (cos, sin), without a rounding of its own.

    The angle: a 64-bit fraction of a turn, less the nearest quarter; what is left is cut to 2^-34 of a turn
    (3.7e-10) and rounded to fp32 where it is below 1/4 of a half turn (2^-27 of a half turn, 2.4e-8),
    the frequency in turns is off by 2^-52 of itself (2 million radians: 4.5e-10) and the 64-bit side's
    angle by as much: 0.43 U in all.  sinpi and cospi are good to a unit in the last place, U below 1."""
    dim, rows = 128, 4096
    half = dim // 2
    p = B.make_params(1, 1, 1, dim, 0, 32, rows // 32 + 1, 0, 1, kv_dtype=F32, q_dtype=F32, capacity_tokens=rows)
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    freq[3] = 2 * math.pi / 8                                      # eighths of a turn, the quarters' borders
    q = torch.zeros(rows, 1, dim, device="cuda")
    a = torch.arange(half) if pairing == B.ROTATE_HALVES else 2 * torch.arange(half)
    b = a + (half if pairing == B.ROTATE_HALVES else 1)
    q[..., a] = 1.0
    k = torch.zeros(rows, 1, dim, device="cuda")
    out = torch.empty_like(q)
    pools = [torch.zeros(rows // 32 + 1, 1, 32, dim, device="cuda") for _ in range(2)]
    table = torch.arange(rows // 32, dtype=torch.int32, device="cuda")[None]
    pos = (first + torch.arange(rows, dtype=torch.int32))
    ws = workspace(p)
    B.sparse_attn_append_kv(p, q, k, k, freq.cuda(), out, *pools, table, ws, seq_lens=torch.zeros(1, dtype=torch.int32, device="cuda"),
                            positions=pos.cuda(), pairing=pairing)
    assert B.sparse_attn_get_device_error(ws) == 0
    angle = pos.double()[:, None] * freq
    got = out[:, 0].cpu().double()
    for channels, want in ((a, angle.cos()), (b, angle.sin())):
        err = (got[:, channels] - want).abs().max()
        assert err <= 1.43 * U, f"off by {float(err / U):.3g} half steps of 1"
