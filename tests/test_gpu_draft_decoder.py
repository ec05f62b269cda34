"""A DraftDecoder's contexts against the length that its parameters name."""
import pytest
import torch

from query_guided_block_gb300 import binding as B
from query_guided_block_gb300.build import build
from query_guided_block_gb300.decoder import DraftDecoder
from tests.draft_reference import Case, place, tree_exact

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build()
    B.lib()


def test_a_decoder_follows_its_parameters():
    """Contexts may grow past the length that a DraftDecoder began with: its `p` is replaced by one with
    a larger n_tokens (or a tighter one), and the workspace stays."""
    c = Case(batch=2, drafts=4, context=40, room=200, lens=(39, 12), block=16)
    table = c.block_table()
    pools = c.fill(c.pools(), table)
    gk, gv, gt = pools[0].cuda(), pools[1].cuda(), table.cuda()
    q = c.normal("q", c.batch, c.drafts, c.hq, c.dim)
    dec = DraftDecoder(c.params(), torch.tensor(c.all_lens, dtype=torch.int32, device="cuda"))
    path = torch.tensor([[0, 1, 3], [0, 2, 3]], dtype=torch.int32)
    dec.commit(path.cuda(), torch.tensor([3, 2], dtype=torch.int32, device="cuda"), gk, gv, gt)
    assert dec.seq_lens.tolist() == [42, 14]
    dec.decode(q.cuda(), gk, gv, gt)
    assert dec.device_error() == B.ERR_LENGTH                      # 42 of at most 40 tokens
    x = Case(**{**c.__dict__, "lens": (42, 14)})
    new_k, new_v = x.normal("kn", 8, c.hkv, c.dim), x.normal("vn", 8, c.hkv, c.dim)
    for bound in (44, 42):
        dec.p = c.params(n_tokens=bound)
        dec.append(None, new_k.cuda(), new_v.cuda(), None, None, gk, gv, gt)
        out = dec.decode(q.cuda(), gk, gv, gt)
        assert dec.device_error() == 0
        k, v = gk.cpu(), gv.cpu()
        page, off = place(c, table, 0, torch.arange(42, 46))
        assert torch.equal(k[page, :, off], new_k[:4])
        exact, limit = tree_exact(x, q, (k, v), table)
        assert ((out.cpu().double() - exact).abs() <= limit).all()
