"""Page table, lengths and weights behind an eviction, against the same in Python."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def expected(table, lens, new_lens, new_table, weights, keep, keep_lens, sure, n_tokens, bs, pages):
    table, old, weights = [list(r) for r in table], [list(r) for r in table], weights.clone()
    active = [0 <= n <= n_tokens for n in lens]
    reads = [{p for j, p in enumerate(r) if on and j * bs < n and 0 <= p < pages} for r, n, on in zip(old, lens, active)]
    out = list(lens)
    for b, n in enumerate(lens):
        k = keep if keep_lens is None else keep_lens[b]
        if not active[b] or not sure <= k <= keep:
            continue
        width = len(new_table[b])
        table[b][:width] = new_table[b]
        for j in range(width, len(table[b])):
            if any(old[b][j] in r for x, r in enumerate(reads) if x != b):
                table[b][j] = -1
        weights[b, :, new_lens[b]:] = 0
        out[b] = new_lens[b]
    return table, out, weights


def run(batch, nb, bs, keep, width, n_tokens, capacity, lens, pages, keep_lens=None, sure=0, seed=0, hkv=2, with_weights=True,
        spread=None):
    g = torch.Generator().manual_seed(seed)
    table = torch.randint(0, pages, (batch, nb), generator=g)
    for b in range(batch):                                                 # a page once a row
        table[b] = torch.randperm(pages, generator=g)[:nb]
    if spread:
        table *= spread                                                    # pages that hash alike or far apart
        pages *= spread
    table[torch.rand(table.shape, generator=g) < 0.1] = -1
    table[torch.rand(table.shape, generator=g) < 0.05] = pages + 5
    new = torch.randint(-1, pages, (batch, width), generator=g)
    p = B.make_params(batch, hkv, hkv, 64, n_tokens, bs, pages, 0, 1, capacity_tokens=capacity)
    new_lens = [min(n, keep if keep_lens is None else keep_lens[b]) if n >= 0 else n for b, n in enumerate(lens)]
    weights = torch.rand(batch, hkv, nb * bs, generator=g)
    want = expected(table.tolist(), lens, new_lens, new.tolist(), weights, keep, keep_lens, sure, n_tokens, bs, pages)
    size = B.sparse_attn_evict_workspace_size(p, keep)
    room = torch.full((size + 1024,), 0xAB, dtype=torch.uint8, device="cuda")
    ws = room[:size]
    B.sparse_attn_workspace_init(ws[:256])
    t, w, n = table.to(torch.int32).cuda(), weights.cuda(), int32(lens)
    for _ in range(2):
        t.copy_(table), w.copy_(weights), n.copy_(int32(lens))
        B.sparse_attn_evict_adopt(p, keep, sure, 0, n, int32(new_lens), t, new.to(torch.int32).cuda(), ws,
                                  None if keep_lens is None else int32(keep_lens), w if with_weights else None)
        assert t.tolist() == want[0] and n.tolist() == want[1]
        assert torch.equal(w.cpu(), want[2] if with_weights else weights)
    assert B.sparse_attn_get_device_error(ws) == 0 and (room[size:] == 0xAB).all()


CASES = {
    "one": dict(batch=1, nb=10, bs=16, keep=32, width=2, n_tokens=150, capacity=160, lens=[150], pages=20),
    "few_pages": dict(batch=5, nb=10, bs=16, keep=32, width=2, n_tokens=150, capacity=160, lens=[150, 100, 7, 0, 149], pages=12),
    "inactive": dict(batch=5, nb=10, bs=16, keep=32, width=3, n_tokens=150, capacity=160, lens=[150, -1, 151, -7, 33], pages=15),
    "budgets": dict(batch=5, nb=10, bs=8, keep=33, width=5, n_tokens=80, capacity=80, lens=[80, 70, 60, 50, 40], pages=15, sure=5,
                    keep_lens=[33, -1, 5, 4, 34]),
    "odd_ends": dict(batch=6, nb=10, bs=8, keep=80, width=10, n_tokens=80, capacity=77, lens=[1, 2, 3, 77, 5, 66], pages=15,
                     keep_lens=[1, 2, 3, 77, 4, 61]) | dict(n_tokens=77),
    "whole_rows": dict(batch=4, nb=10, bs=16, keep=32, width=10, n_tokens=150, capacity=160, lens=[150, 3, 64, 10], pages=12),
    "no_weights": dict(batch=4, nb=10, bs=16, keep=32, width=2, n_tokens=150, capacity=160, lens=[150, 3, 64, 10], pages=12,
                       with_weights=False),
    "many": dict(batch=300, nb=40, bs=8, keep=64, width=8, n_tokens=320, capacity=320, lens=[(37 * i) % 321 for i in range(300)],
                 pages=6000),
    "many_shared": dict(batch=200, nb=40, bs=8, keep=64, width=8, n_tokens=320, capacity=320, lens=[(37 * i) % 321 for i in range(200)],
                        pages=60),
    "pages_far_apart": dict(batch=50, nb=40, bs=8, keep=64, width=8, n_tokens=320, capacity=320, lens=[(37 * i) % 321 for i in range(50)],
                            pages=900, spread=1 << 16),
    "long_kept": dict(batch=3, nb=1300, bs=8, keep=5002, width=626, n_tokens=10400, capacity=10400, lens=[10397, 4096, 4097], pages=3500),
    "long_rows": dict(batch=3, nb=1000, bs=8, keep=500, width=63, n_tokens=8000, capacity=8000, lens=[8000, 7001, 600], pages=2500,
                      hkv=8),
}


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("name", CASES)
def test_against_python(name, seed):
    run(seed=seed, **CASES[name])


def test_the_workspace_goes_by_the_page_table():
    """A pool that grows needs no other workspace."""
    sizes = {B.sparse_attn_evict_workspace_size(B.make_params(4, 2, 2, 64, 150, 16, n, 0, 1, capacity_tokens=160), 32)
             for n in (10, 1000, 10 ** 6)}
    assert len(sizes) == 1
