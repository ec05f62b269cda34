"""Plain 64-bit statements of the norm append, shared prefixes, weighed attention and eviction, and the
bounds that an fp32 computation of them keeps (test code only; CPU tensors in, CPU tensors out)."""
from __future__ import annotations

import math

import torch

from query_guided_block_gb300 import binding as B
from tests.draft_reference import U, chain_mask, half_step, place


def rms(x, weight, eps):
    """x [n, H, D] in 64 bits, normed over D."""
    x = x.double()
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def rotate_axes(x, angle, pairing):
    """x [n, H, D] in 64 bits turned by angle [n, rotary / 2]; returns (rotated, |x_a| + |x_b| per channel)."""
    out, mag = x.clone(), x.abs()
    half = angle.shape[1]
    if half == 0:
        return out, mag
    a = torch.arange(half) if pairing == B.ROTATE_HALVES else 2 * torch.arange(half)
    b = a + half if pairing == B.ROTATE_HALVES else a + 1
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    mag[..., a] = mag[..., b] = x[..., a].abs() + x[..., b].abs()
    return out, mag


def norm_bound(exact, mag, dtype):
    """A sum of squares is two chains of 8 products, one addition and at most three exchanges: 12
    roundings, U each of a sum of positive terms, which the root halves; the mean and eps add a rounding
    each, the reciprocal root two units in the last place, 4 U, then come two products:
    12 / 2 + 2 + 4 + 2 = 14 U of a normed channel.  The rotation adds 5 U of |x_a| + |x_b|
    (draft_reference.rotation_bound); 20 U cover both with their products.  Then the rounding to the
    stored type."""
    delta = 20 * U * mag
    return delta + half_step(dtype) * (exact.abs() + delta)


def attention_exact(case, q, pools, table, see=None, scale=None, weights=None):
    """(out, bound, weights, weights' bound) in 64 bits; see [B, Q, Q] (None: a chain).

    A score is a chain of D / 8 + 2 matrix steps and additions, each off by at most two units 2^-23 of
    the sum of magnitudes; fp32 operands are kept to 2^-21.  Scaling rounds twice (U of the score
    each) and exp2 is good to 2^-21.  With bf16 values a weight is held exactly, with fp32 ones weight,
    value and the left-out product of the small parts are 2^-21 each.  A row's total is a chain of at most
    n / 4 + 64 additions, a channel one of n / 32 + 64 steps and merges of 2^-22.  Errors of the weights
    reach a result directly and through the total.  The rows of a KV head add up in a chain of R.  Below
    2^-126 of the row's largest, exp2 gives 0 (flushed) and a row's total is at least 1 of the largest, so
    every weight may be off by 2^-126 besides."""
    lens, G = case.all_lens, case.hq // case.hkv
    scale = 1 / math.sqrt(case.dim) if scale is None else scale
    out = torch.zeros(case.batch, case.drafts, case.hq, case.dim, dtype=torch.float64)
    bound = torch.full_like(out, 1e-30)
    w_out = None if weights is None else weights.double().clone()
    w_bound = None if weights is None else torch.zeros_like(w_out)
    see = chain_mask(case.drafts).expand(case.batch, -1, -1) if see is None else see
    held = 2.0 ** -21 if case.kv == torch.bfloat16 else 4 * 2.0 ** -21
    for b, n in enumerate(lens):
        if n < 0:
            continue
        t = torch.arange(n + case.drafts)
        page, off = place(case, table, b, t)
        for h in range(case.hkv):
            k, v = pools[0][page, h, off].double(), pools[1][page, h, off].double()
            sums, err = torch.zeros(len(t), dtype=torch.float64), torch.zeros(len(t), dtype=torch.float64)
            for i in range(case.drafts):
                ok = torch.cat([torch.ones(n, dtype=torch.bool), see[b, i]])
                if not ok.any():
                    continue
                ki, vi, m = k[ok], v[ok], int(ok.sum())
                for head in range(h * G, (h + 1) * G):
                    qi = q[b, i, head].double()
                    s = ki @ qi * scale
                    p = torch.softmax(s, 0)
                    out[b, i, head] = p @ vi
                    err_p = ((case.dim / 8 + 2) * 2 ** -22 + 2 ** -21) * (ki.abs() @ qi.abs()) * scale + s.abs() * 2 * U + held
                    total = (p * err_p).sum() + (m / 4 + 64) * U
                    mag = p @ vi.abs()
                    bound[b, i, head] = (p * err_p) @ vi.abs() + (total + (m / 32 + 64) * 2 ** -22) * mag
                    sums[ok] += p
                    err[ok] += p * (err_p + total)
            if w_out is not None:
                old = torch.where(t < n, w_out[b, h, : len(t)], torch.zeros(()).double())
                w_out[b, h, : len(t)] = old + sums
                w_bound[b, h, : len(t)] = err + (case.drafts * G + 2) * U * sums + U * (old + sums) + case.drafts * G * 2.0 ** -126
    return out, bound, w_out, w_bound


def kept_tokens(row, n, k, sinks, recent):
    """Indexes of the kept ones of n tokens with these weights, ascending."""
    if n <= k:
        return list(range(n))
    sure = set(range(sinks)) | set(range(n - recent, n))
    rest = sorted((t for t in range(n) if t not in sure), key=lambda t: (-row[t], t))
    return sorted(sure | set(rest[: k - len(sure)]))
