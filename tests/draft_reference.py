"""Plain 64-bit statements of the cache-growing and draft-tree operators, their error bounds,
and small cases for them (test code only; CPU tensors in, CPU tensors out)."""
from __future__ import annotations

import dataclasses
import math

import torch

from query_guided_block_gb300 import binding as B

U = 2.0 ** -24                                    # half a step of fp32, relative


def half_step(t: torch.dtype) -> float:
    return torch.finfo(t).eps / 2


@dataclasses.dataclass
class Case:
    batch: int = 2
    hq: int = 8
    hkv: int = 2
    dim: int = 128
    block: int = 32
    context: int = 300                            # the longest one
    lens: tuple = None                            # per sequence; None: `context` each
    drafts: int = 7
    room: int = 0                                 # more capacity than context + drafts needs
    dtype: torch.dtype = torch.bfloat16
    kv: torch.dtype = torch.bfloat16
    topk: int = 8
    window: int = 0
    seed: int = 0

    @property
    def capacity(self):
        return self.context + self.drafts + self.room

    @property
    def nb_cap(self):
        return -(-self.capacity // self.block)

    @property
    def pages(self):
        return self.batch * self.nb_cap + 3       # some pages belong to nobody

    @property
    def all_lens(self):
        return list(self.lens) if self.lens is not None else [self.context] * self.batch

    def params(self, **over):
        kw = dict(batch=self.batch, num_q_heads=self.hq, num_kv_heads=self.hkv, head_dim=self.dim,
                  n_tokens=self.context, block_size=self.block, num_pages=self.pages,
                  window_tokens=self.window, topk=self.topk, kv_dtype=self.kv, q_dtype=self.dtype,
                  num_queries=self.drafts, capacity_tokens=self.capacity)
        kw.update(over)
        return B.make_params(**kw)

    def gen(self, what):
        import zlib
        return torch.Generator().manual_seed(zlib.crc32(f"{what}/{self.seed}/{self}".encode()))

    def normal(self, what, *shape, dtype=None):
        return torch.randn(*shape, generator=self.gen(what)).to(dtype or self.dtype)

    def block_table(self):
        return torch.randperm(self.pages, generator=self.gen("table"))[: self.batch * self.nb_cap].view(
            self.batch, self.nb_cap).to(torch.int32)

    def pools(self, empty=float("nan")):
        """Pools that hold `empty` everywhere (the tests fill what may be read)."""
        shape = (self.pages, self.hkv, self.block, self.dim)
        return torch.full(shape, empty, dtype=self.kv), torch.full(shape, empty, dtype=self.kv)

    def fill(self, pools, table, upto=None):
        """N(0, 1) keys and values for tokens [0, upto[b]) of every sequence (default: the
        context and the drafts)."""
        g = self.gen("kv")
        for b, n in enumerate(self.all_lens):
            n = max(0, n) + self.drafts if upto is None else upto[b]
            t = torch.arange(n)
            page = table[b].long()[t // self.block]
            for pool in pools:
                pool[page, :, t % self.block] = torch.randn(n, self.hkv, self.dim, generator=g).to(self.kv)
        return pools


def place(case, table, b, t):
    return table[b].long()[t // case.block], t % case.block


def chain_mask(q):
    return torch.tril(torch.ones(q, q, dtype=torch.bool))


def random_tree(case):
    """[B, Q, Q] ancestors-and-self of random trees, parents before children."""
    g = case.gen("tree")
    see = torch.zeros(case.batch, case.drafts, case.drafts, dtype=torch.bool)
    for b in range(case.batch):
        for i in range(case.drafts):
            see[b, i, i] = True
            if i > 0:
                parent = int(torch.randint(-1, i, (1,), generator=g))
                if parent >= 0:
                    see[b, i] |= see[b, parent]
    return see


def pack_mask(see):
    bsz, q, _ = see.shape
    w = -(-q // 32)
    words = torch.zeros(bsz, q, w, dtype=torch.int64)
    for j in range(q):
        words[:, :, j // 32] |= see[:, :, j].long() << (j % 32)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


# ------------------------------------------------------------------- append --

def rotate(x, pos, inv_freq, pairing):
    """x [n, H, D] in 64 bits; returns (rotated, |x_a| + |x_b| per channel)."""
    x = x.double()
    out, mag = x.clone(), x.abs()
    if inv_freq is None:
        return out, mag
    half = inv_freq.numel()
    a = torch.arange(half) if pairing == B.ROTATE_HALVES else 2 * torch.arange(half)
    b = a + half if pairing == B.ROTATE_HALVES else a + 1
    angle = pos.double()[:, None] * inv_freq.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return out, mag


def rotation_bound(exact, mag, dtype):
    """A rotated channel is x_a c - x_b s in fp32.  The angle in half turns is a 32-bit fraction
    (2^-32 of a turn) rounded to fp32 (2^-25): at most 9.6e-8 in the angle, 1.61 U; sinpi and
    cospi add one unit in the last place of values below 1, 2^-24 = U (a step, documented),
    the product and the sum two roundings.  Five U of |x_a| + |x_b| cover 1.61 + 1 + 2; then the
    rounding to the stored type."""
    delta = 5 * U * mag
    return delta + half_step(dtype) * (exact.abs() + delta)


# --------------------------------------------------------------------- tree --

def tree_exact(case, q, pools, table, see=None, sel_ids=None, sel_count=None, scale=None):
    """(out, bound): [B, Q, Hq, D] in 64 bits and how far an fp32 output may be off.

    The bound: a score is a chain of D / 8 + 2 matrix steps and additions (twice that with
    split operands counts the small parts' steps, whose errors are 2^-8 of these), each off
    by at most two units 2^-23 of the sum of magnitudes; operands kept to 2^-21 or better; the
    scaled score is rounded (U of it) and exp2 is good to 2^-21.  A weight is held to
    2^-17.  The weighted sum is a chain of n / 8 steps plus 64 merges, each two units 2^-23 of
    sum p |v|.  Errors of scores reach the output through every weight and through the
    total: twice."""
    lens = case.all_lens
    G = case.hq // case.hkv
    scale = 1 / math.sqrt(case.dim) if scale is None else scale
    out = torch.zeros(case.batch, case.drafts, case.hq, case.dim, dtype=torch.float64)
    bound = torch.full_like(out, 1e-30)
    see = chain_mask(case.drafts).expand(case.batch, -1, -1) if see is None else see
    for b, n in enumerate(lens):
        if n < 0:
            continue
        for h in range(case.hkv):
            if sel_ids is None:
                ctx = torch.arange(n)
            else:
                blk = sel_ids[b, h, : int(sel_count[b, h])].long()
                ctx = (blk[:, None] * case.block + torch.arange(case.block)).reshape(-1)
                ctx = ctx[ctx < n]
            t = torch.cat([ctx, torch.arange(n, n + case.drafts)])
            page, off = place(case, table, b, t)
            k, v = pools[0][page, h, off].double(), pools[1][page, h, off].double()
            for i in range(case.drafts):
                ok = torch.cat([torch.ones(len(ctx), dtype=torch.bool), see[b, i]])
                if not ok.any():
                    continue
                ki, vi = k[ok], v[ok]
                for head in range(h * G, (h + 1) * G):
                    qi = q[b, i, head].double()
                    s = ki @ qi * scale
                    p = torch.softmax(s, 0)
                    out[b, i, head] = p @ vi
                    err_s = ((case.dim / 8 + 2) * 2 ** -22 + 2 ** -21) * (ki.abs() @ qi.abs()) * scale
                    err_p = err_s + s.abs() * 2 * U + 2 ** -21 + 2 ** -17
                    chain = (ok.sum() / 8 + 64) * 2 ** -22
                    mag = p @ vi.abs()
                    bound[b, i, head] = (p * err_p) @ vi.abs() + (p * err_p).sum() * mag + 2 * chain * mag
    return out, bound
