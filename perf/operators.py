"""Timed cases of the operators that grow a paged K/V cache and verify drafted tokens.

* ``append``: new tokens' keys and values go into the page pools, queries and keys are
  rotated to their positions on the way, and the per-block key box follows.
* ``tree``: attention of a tree of drafted tokens over the cached context (all of it, or
  each KV head's selected blocks) and over the drafts that a query may see.
* ``commit``: the accepted path of a draft tree moves to the end of the context.

``run`` computes them in elementary torch operations, or with the library's calls when
``own`` is set.  Layouts are those of include/sparse_attn.h.
"""
import math

import numpy as np
import torch

own = False

HALVES, PAIRS = 1, 2                       # channel pairing of the rotation
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _append(name, **kw):
    base = dict(op="append", batch=1, rows=1, context=4096, ragged=False, hq=32, hkv=8, dim=128, block=32,
                dtype="bf16", kv="bf16", rotary=128, pairing=HALVES, box=True, fused_input=True)
    return {"name": name, **base, **kw}


def _tree(name, **kw):
    base = dict(op="tree", batch=1, drafts=8, context=4096, ragged=False, hq=32, hkv=8, dim=128, block=32,
                dtype="bf16", kv="bf16", select=0, chain=False)
    return {"name": name, **base, **kw}


def _commit(name, **kw):
    base = dict(op="commit", batch=1, drafts=16, path=4, context=4096, ragged=False, hq=32, hkv=8, dim=128, block=32,
                dtype="bf16", kv="bf16", box=True)
    return {"name": name, **base, **kw}


def listed():
    return [
        # one user's next token far into a 128K context: nothing but latency
        _append("append_one_token", context=131071),
        # a serving batch's next tokens, contexts of all lengths
        _append("append_batch_decode", batch=128, context=1000, ragged=True, block=64),
        # prompts of all lengths packed into one batch behind cached prefixes
        _append("append_ragged_prompts", batch=16, rows=4001, context=1500, ragged=True, block=64),
        # an fp32 cache, the rotation on a part of the channels in neighbouring pairs, odd counts
        _append("append_fp32_partial", batch=3, rows=333, context=777, ragged=True, hq=4, hkv=4, dim=64, block=64,
                dtype="f32", kv="f32", rotary=32, pairing=PAIRS, fused_input=False),
        # one user's single token over a short context
        _tree("tree_one_token", drafts=1, context=777),
        # a draft tree of one user far into a long context
        _tree("tree_long_context", drafts=24, context=131072, block=64),
        # a batch of draft trees over contexts of all lengths, every cached token read
        _tree("tree_batch", batch=16, drafts=16, context=32768, ragged=True, block=64),
        # wide trees: as much arithmetic as memory traffic
        _tree("tree_wide", batch=8, drafts=64, context=16384, block=64),
        # a draft tree per sequence over each KV head's selected blocks of a 128K context
        _tree("tree_selected_128k", batch=16, drafts=16, context=131072, select=80),
        # an fp32 cache with fp32 queries, a chain of drafts
        _tree("tree_fp32_chain", drafts=7, context=4096, hq=4, hkv=4, dim=64, block=64, dtype="f32", kv="f32",
              chain=True),
        # one user's accepted drafts, and a batch's
        _commit("commit_one", context=131072),
        _commit("commit_batch", batch=64, drafts=63, path=12, context=1000, ragged=True, block=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "append", "tree", "tree", "tree", "commit"])
    hkv, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    c = dict(op=op, batch=_log(rng, 1, 128), context=_log(rng, 1, 131072), ragged=rng.random() < 0.6,
             hq=hkv * group, hkv=hkv, dim=dim, block=rng.choice([16, 32, 64, 128]), dtype="bf16", kv="bf16")
    kind = rng.random()
    if kind < 0.2:
        c["dtype"] = "f32"
    if kind < 0.12:
        c["kv"] = "f32"
    if op == "append":
        c.update(rows=_log(rng, 1, 8192), rotary=rng.choice([dim, dim, dim // 2]), pairing=rng.choice([HALVES, PAIRS]),
                 box=rng.random() < 0.7, fused_input=rng.random() < 0.7)
        size, most = c["rows"], 60000
    elif op == "tree":
        c.update(drafts=_log(rng, 1, 64), select=0, chain=rng.random() < 0.25)
        if rng.random() < 0.3:
            c["select"] = _log(rng, 4, 96)
        size, most = c["context"] + c["drafts"], 520000
        if c["kv"] == "f32":
            most = 66000                   # the larger part of fp32 use: checks at moderate lengths
    else:
        c.update(drafts=_log(rng, 5, 64), box=rng.random() < 0.7)
        c["path"] = rng.randint(1, max(1, c["drafts"] // 4))
        size, most = c["context"], 260000
    # a pool of at most about two million tokens, and no more work than the largest listed case
    most = min(most * 8 // hkv, 2000000)
    if size > most:
        if op == "append":
            c["rows"] = most
        else:
            c["context"] = most - c.get("drafts", 0)
        size = most
    c["batch"] = max(1, min(c["batch"], most // size, 2000000 // (c["context"] + size)))
    top = [max(w[k] for w in map(work, listed())) for k in ("bytes", "flops")]
    while work(c)["bytes"] > top[0] or work(c)["flops"] > top[1]:
        if c["batch"] > 1:
            c["batch"] = max(1, c["batch"] * 3 // 4)
        else:
            c["context"] = c["context"] * 3 // 4
    return c


# ------------------------------------------------------------------ sizes --

def _spread(n, most, step):
    """n whole numbers in [most // 2, most], the first one `most`; a function of the case alone."""
    return [most - (i * step) % (most // 2 + 1) for i in range(n)]


def _lens(c):
    return _spread(c["batch"], c["context"], 7919) if c["ragged"] else [c["context"]] * c["batch"]


def _counts(c):
    """New rows of each sequence."""
    return _spread(c["batch"], c["rows"], 613) if c["ragged"] else [c["rows"]] * c["batch"]


def _paths(c):
    return [1 + (i * 5 + c["path"] - 1) % c["path"] for i in range(c["batch"])]


def _selected(c):
    """Selected blocks of each sequence's units."""
    return [min(c["select"], -(-n // c["block"])) for n in _lens(c)]


def work(case):
    c = case
    e, ekv, D = (2 if c["dtype"] == "bf16" else 4), (2 if c["kv"] == "bf16" else 4), c["dim"]
    if c["op"] == "append":
        n = sum(_counts(c))
        b = n * (c["hq"] + 2 * c["hkv"]) * D * e + n * c["hq"] * D * e + n * 2 * c["hkv"] * D * ekv + n * 4
        if c["box"]:
            for old, add in zip(_lens(c), _counts(c)):
                first, last = old // c["block"], (old + add - 1) // c["block"]
                b += 2 * c["hkv"] * D * ekv * (last - first + 1 + (1 if old % c["block"] else 0))
        return {"bytes": b, "flops": 3 * n * (c["hq"] + c["hkv"]) * c["rotary"]}
    if c["op"] == "commit":
        n = sum(_paths(c))
        b = n * 2 * c["hkv"] * D * ekv * 2 + n * 4 + 12 * c["batch"]
        if c["box"]:
            for old, add in zip(_lens(c), _paths(c)):
                first, last = old // c["block"], (old + add - 1) // c["block"]
                b += 2 * c["hkv"] * D * ekv * (last - first + 1 + (1 if old % c["block"] else 0))
        return {"bytes": b, "flops": 0}
    Q, bs = c["drafts"], c["block"]
    tokens = [min(n, k * bs) for n, k in zip(_lens(c), _selected(c))] if c["select"] else _lens(c)
    keys = sum(t + Q for t in tokens)
    b = keys * c["hkv"] * D * 2 * ekv + c["batch"] * Q * c["hq"] * D * (e + 4) + c["batch"] * Q * 4 * -(-Q // 32)
    b += 4 * sum(-(-(n + Q) // bs) for n in _lens(c)) if not c["select"] else 8 * c["hkv"] * sum(_selected(c))
    return {"bytes": b, "flops": 4 * Q * c["hq"] * D * keys}


# ----------------------------------------------------------------- inputs --

def _tree_parents(c, g):
    """Parents of each sequence's drafts, parents before children: -1 is the context's last token."""
    B, Q = c["batch"], c["drafts"]
    u = torch.rand(B, Q, generator=g, device="cuda")
    parent = (u * torch.arange(Q, device="cuda")).long()          # uniform below the node itself
    if c.get("chain"):
        parent = torch.arange(-1, Q - 1, device="cuda").expand(B, Q).clone()
    parent[:, 0] = -1
    return parent


def _ancestors(parent):
    """[B, Q, Q] truth values: draft j is draft i or one of its ancestors."""
    Q = parent.shape[1]
    step = (parent[:, :, None] == torch.arange(Q, device=parent.device)) | torch.eye(Q, dtype=torch.bool, device=parent.device)
    return torch.linalg.matrix_power(step.double(), Q) > 0.5       # at most 2^Q walks: exact enough to tell from none


def _pack_bits(see):
    """[B, Q, Q] truth values -> [B, Q, ceil(Q / 32)] int32 words, bit j % 32 of word j // 32."""
    B, Q, _ = see.shape
    W = -(-Q // 32)
    bits = torch.zeros(B, Q, W * 32, dtype=torch.int64, device=see.device)
    bits[:, :, :Q] = see
    words = (bits.view(B, Q, W, 32) << torch.arange(32, device=see.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62))
    dev, B, D, bs = "cuda", c["batch"], c["dim"], c["block"]
    dt, kvt = DTYPES[c["dtype"]], DTYPES[c["kv"]]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    lens = _lens(c)
    room = c["rows"] if c["op"] == "append" else c["drafts"]
    capacity = c["context"] + room
    nb_cap = -(-capacity // bs)
    pages = B * nb_cap
    s = {"case": c, "capacity": capacity, "num_pages": pages}
    s["block_table"] = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(B, nb_cap)
    s["k_pages"] = normal(pages, c["hkv"], bs, D, dtype=kvt)
    s["v_pages"] = normal(pages, c["hkv"], bs, D, dtype=kvt)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if c.get("box"):
        # a box as N(0, 1) keys leave it, around zero
        s["kmin"] = -normal(B, c["hkv"], nb_cap, D, dtype=kvt).abs() - 1.5
        s["kmax"] = normal(B, c["hkv"], nb_cap, D, dtype=kvt).abs() + 1.5

    if c["op"] == "append":
        counts = _counts(c)
        n, hq, hkv = sum(counts), c["hq"], c["hkv"]
        if c["fused_input"]:               # one projection's output, [rows, q | k | v]
            qkv = normal(n, (hq + 2 * hkv) * D)
            q, k, v = qkv.split([hq * D, hkv * D, hkv * D], dim=1)
        else:
            q, k, v = normal(n, hq * D), normal(n, hkv * D), normal(n, hkv * D)
        s["q_new"], s["k_new"], s["v_new"] = q.view(n, hq, D), k.view(n, hkv, D), v.view(n, hkv, D)
        s["cu_rows"] = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device=dev)
        s["row_seq"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(counts, device=dev), output_size=n)
        half = c["rotary"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        s["q_out"] = torch.empty(n, hq, D, dtype=dt, device=dev)
    elif c["op"] == "tree":
        Q = c["drafts"]
        s["q"] = normal(B, Q, c["hq"], D)
        s["mask"] = _pack_bits(_ancestors(_tree_parents(c, g)))
        s["out"] = torch.empty(B, Q, c["hq"], D, dtype=torch.float32, device=dev)
        if c["select"]:
            nb = -(-c["context"] // bs)    # the longest sequence's context
            blocks = (s["lens"] + bs - 1) // bs
            key = torch.rand(B, c["hkv"], nb, generator=g, device=dev)
            j = torch.arange(nb, device=dev, dtype=torch.int32)
            key = key.masked_fill(j >= blocks[:, None, None], 2.0)
            key = key.masked_fill(j == blocks[:, None, None] - 1, -1.0)        # the local window
            top = min(c["select"], nb)
            s["sel_count"] = torch.clamp(blocks, max=top).to(torch.int32)[:, None].expand(B, c["hkv"]).contiguous()
            ids = key.argsort(dim=-1)[..., :top]
            ids = ids.masked_fill(torch.arange(top, device=dev) >= s["sel_count"][..., None], nb)
            ids = ids.sort(dim=-1).values
            s["sel_ids"] = ids.masked_fill(ids == nb, 0).to(torch.int32)       # unused entries name block 0
    else:
        P, Q = c["path"], c["drafts"]
        # strictly ascending accepted drafts: the first one, then some behind the accepted region
        key = torch.rand(B, Q, generator=g, device=dev)
        key[:, :P] = 2.0
        key[:, 0] = -1.0
        s["path"] = key.argsort(dim=1)[:, :P].sort(dim=1).values.to(torch.int32)
        s["path_len"] = torch.tensor(_paths(c), dtype=torch.int32, device=dev)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=dev)
    if own:
        from query_guided_block_gb300 import binding as lib
        top = max(1, c.get("select") or 1)
        s["params"] = lib.make_params(B, c["hq"], c["hkv"], D, c["context"], bs, pages, 0, top, kv_dtype=kvt, q_dtype=dt,
                                      num_queries=c.get("drafts", 1), capacity_tokens=capacity)
        size = lib.sparse_attn_tree_workspace_size(s["params"])
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=dev)
        lib.sparse_attn_workspace_init(s["ws"])
    return s


# ----------------------------------------------------------- plain forms --

def _rotate(x, angle, rotary, pairing):
    """The first `rotary` channels of x [rows, heads, D] fp32 turned by angle [rows, rotary / 2] fp64."""
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r, rest = x[..., :rotary], x[..., rotary:]
    if pairing == HALVES:
        a, b = r[..., : rotary // 2], r[..., rotary // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, rest], -1)


def _widen_box(s, seq, token, old, keys):
    """Per-channel minimum / maximum of the stored keys [rows, Hkv, D] into their blocks' rows of the box."""
    c = s["case"]
    B, hkv, nb_cap, D = s["kmin"].shape
    block = token // c["block"]
    row = (seq[:, None] * hkv + torch.arange(hkv, device=seq.device)) * nb_cap + block[:, None]      # [rows, Hkv]
    index = row.reshape(-1, 1).expand(-1, D)
    fresh = (block * c["block"] >= old)[:, None].expand(-1, hkv).reshape(-1)       # no cached token in the block
    x = keys.float().reshape(-1, D)
    for name, start, how in (("kmin", math.inf, "amin"), ("kmax", -math.inf, "amax")):
        flat = s[name].view(-1, D)
        new = flat.float()
        new[row.reshape(-1)[fresh]] = start
        new.scatter_reduce_(0, index, x, how)
        flat.copy_(new)


def _plain_append(s):
    c = s["case"]
    seq = s["row_seq"]
    first = s["cu_rows"].long()[seq]
    old = s["lens"].long()[seq]
    token = old + torch.arange(seq.numel(), device=seq.device) - first
    angle = token.double()[:, None] * s["inv_freq"]
    dt = s["q_new"].dtype
    q = _rotate(s["q_new"].float(), angle, c["rotary"], c["pairing"]).to(dt)
    k = _rotate(s["k_new"].float(), angle, c["rotary"], c["pairing"]).to(s["k_pages"].dtype)
    page = s["block_table"].long()[seq, token // c["block"]]
    s["k_pages"][page, :, token % c["block"]] = k
    s["v_pages"][page, :, token % c["block"]] = s["v_new"].to(s["v_pages"].dtype)
    if c["box"]:
        _widen_box(s, seq, token, old, k)
        return {"q": q, "k": s["k_pages"], "v": s["v_pages"], "kmin": s["kmin"], "kmax": s["kmax"]}
    return {"q": q, "k": s["k_pages"], "v": s["v_pages"]}


def _plain_tree(s):
    c = s["case"]
    B, Q, hq, D = s["q"].shape
    hkv, bs, dev = c["hkv"], c["block"], s["q"].device
    G = hq // hkv
    lens = s["lens"].long()
    bt = s["block_table"].long()
    if c["select"]:
        ids = s["sel_ids"].long()                                                  # [B, Hkv, S]
        there = torch.arange(ids.shape[-1], device=dev) < s["sel_count"][..., None]
        page = bt[torch.arange(B, device=dev)[:, None, None], ids]
        head = torch.arange(hkv, device=dev)[None, :, None]
        k, v = s["k_pages"][page, head].float(), s["v_pages"][page, head].float()  # [B, Hkv, S, bs, D]
        token = ids[..., None] * bs + torch.arange(bs, device=dev)
        valid = (there[..., None] & (token < lens[:, None, None, None])).flatten(2)
        k, v = k.flatten(2, 3), v.flatten(2, 3)
    else:
        nb = -(-c["context"] // bs)
        k = s["k_pages"][bt[:, :nb]].float().permute(0, 2, 1, 3, 4).flatten(2, 3)  # [B, Hkv, nb * bs, D]
        v = s["v_pages"][bt[:, :nb]].float().permute(0, 2, 1, 3, 4).flatten(2, 3)
        valid = (torch.arange(nb * bs, device=dev) < lens[:, None])[:, None].expand(B, hkv, nb * bs)
    at = lens[:, None] + torch.arange(Q, device=dev)                               # the drafts' tokens
    page = torch.gather(bt, 1, at // bs)
    kd = s["k_pages"][page, :, at % bs].float().transpose(1, 2)                    # [B, Hkv, Q, D]
    vd = s["v_pages"][page, :, at % bs].float().transpose(1, 2)
    j = torch.arange(Q, device=dev)
    see = ((s["mask"][:, :, j // 32] >> (j % 32)) & 1).bool()                      # [B, Q, Q]
    allow = torch.cat([valid[:, :, None].expand(B, hkv, Q, valid.shape[-1]), see[:, None].expand(B, hkv, Q, Q)], -1)
    allow = allow[:, :, :, None].expand(B, hkv, Q, G, allow.shape[-1]).flatten(2, 3)
    q = s["q"].float().view(B, Q, hkv, G, D).transpose(1, 2).flatten(2, 3)         # [B, Hkv, Q * G, D]
    score = torch.cat([q @ k.transpose(-1, -2), q @ kd.transpose(-1, -2)], -1) / math.sqrt(D)
    score = score.masked_fill(~allow, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp()
    total = p.sum(-1, keepdim=True)
    n = k.shape[2]
    out = p[..., :n] @ v + p[..., n:] @ vd
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return out.view(B, hkv, Q, G, D).transpose(1, 2).reshape(B, Q, hq, D)


def _plain_commit(s):
    c = s["case"]
    B, P = s["path"].shape
    dev, bs = s["path"].device, c["block"]
    bt, lens = s["block_table"].long(), s["lens"].long()
    i = torch.arange(P, device=dev)
    seq, i = (i < s["path_len"][:, None]).nonzero(as_tuple=True)
    src, dst = lens[seq] + s["path"].long()[seq, i], lens[seq] + i
    sp, dp = bt[seq, src // bs], bt[seq, dst // bs]
    k, v = s["k_pages"][sp, :, src % bs], s["v_pages"][sp, :, src % bs]
    s["k_pages"][dp, :, dst % bs] = k
    s["v_pages"][dp, :, dst % bs] = v
    out = {"k": s["k_pages"], "v": s["v_pages"], "lens": s["lens"] + s["path_len"]}
    if c["box"]:
        _widen_box(s, seq, dst, lens[seq], k)
        out.update(kmin=s["kmin"], kmax=s["kmax"])
    return out


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"append": _plain_append, "tree": _plain_tree, "commit": _plain_commit}[c["op"]](s)
    from query_guided_block_gb300 import binding as lib
    if c["op"] == "append":
        lib.sparse_attn_append_kv(s["params"], s["q_new"], s["k_new"], s["v_new"], s["inv_freq"], s["q_out"], s["k_pages"],
                                  s["v_pages"], s["block_table"], s["ws"], cu_rows=s["cu_rows"], seq_lens=s["lens"],
                                  pairing=c["pairing"], kmin=s.get("kmin"), kmax=s.get("kmax"))
        out = {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}
    elif c["op"] == "tree":
        lib.sparse_attn_tree_decode(s["params"], s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["out"], s["ws"],
                                    seq_lens=s["lens"], sel_ids=s.get("sel_ids"), sel_count=s.get("sel_count"),
                                    tree_mask=s["mask"])
        return s["out"]
    else:
        lib.sparse_attn_commit_drafts(s["params"], s["path"], s["path_len"], s["k_pages"], s["v_pages"], s["block_table"],
                                      s["new_lens"], s["ws"], seq_lens=s["lens"], kmin=s.get("kmin"), kmax=s.get("kmax"))
        out = {"k": s["k_pages"], "v": s["v_pages"], "lens": s["new_lens"]}
    if c["box"]:
        out.update(kmin=s["kmin"], kmax=s["kmax"])
    return out


# ---------------------------------------------- the definitions in 64 bits --

def _exact_box(s, box, b, tokens, old, keys):
    """The box rows of sequence b's blocks after `tokens` (a list) got the fp64 keys [n, Hkv, D]."""
    bs = s["case"]["block"]
    groups = {}
    for n, t in enumerate(tokens):
        groups.setdefault(t // bs, []).append(n)
    for blk, rows in groups.items():
        part = keys[rows]
        lo, hi = part.min(0).values, part.max(0).values
        if blk * bs < old:
            lo, hi = torch.minimum(lo, box["kmin"][b, :, blk]), torch.maximum(hi, box["kmax"][b, :, blk])
        box["kmin"][b, :, blk], box["kmax"][b, :, blk] = lo, hi


def _exact_append(s):
    c = s["case"]
    bs, half = c["block"], c["rotary"] // 2
    q, k = s["q_new"].double(), s["k_new"].double()
    if c["pairing"] == HALVES:
        one = list(range(half))
        two = list(range(half, c["rotary"]))
    else:
        one = list(range(0, c["rotary"], 2))
        two = list(range(1, c["rotary"], 2))
    pools = {"k": s["k_pages"].double(), "v": s["v_pages"].double()}
    box = {n: s[n].double() for n in ("kmin", "kmax") if n in s}
    r = 0
    for b, (old, count) in enumerate(zip(_lens(c), _counts(c))):
        tokens = list(range(old, old + count))
        at = torch.tensor(tokens, dtype=torch.float64, device=q.device)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=q.device), at[:, None] * s["inv_freq"])[:, None]
        for x in (q, k):
            z = torch.complex(x[r:r + count][..., one], x[r:r + count][..., two]) * turn
            x[r:r + count, :, one] = z.real
            x[r:r + count, :, two] = z.imag
        t = torch.tensor(tokens, device=q.device)
        page = s["block_table"][b].long()[t // bs]
        pools["k"][page, :, t % bs] = k[r:r + count]
        pools["v"][page, :, t % bs] = s["v_new"][r:r + count].double()
        if box:
            _exact_box(s, box, b, tokens, old, k[r:r + count])
        r += count
    return {"q": q, **pools, **box}


def _exact_commit(s):
    c = s["case"]
    bs = c["block"]
    pools = {"k": s["k_pages"].double(), "v": s["v_pages"].double()}
    box = {n: s[n].double() for n in ("kmin", "kmax") if n in s}
    bt, path = s["block_table"].tolist(), s["path"].tolist()
    for b, (old, n) in enumerate(zip(_lens(c), _paths(c))):
        place = {t: (bt[b][t // bs], t % bs) for t in range(old, old + c["drafts"])}
        for name, pool in pools.items():
            moved = [pool[place[old + path[b][i]][0], :, place[old + path[b][i]][1]].clone() for i in range(n)]
            for i in range(n):
                pool[place[old + i][0], :, place[old + i][1]] = moved[i]
            if name == "k" and box:
                _exact_box(s, box, b, list(range(old, old + n)), old, torch.stack(moved))
    return {**pools, "lens": None, **box}


def _exact_tree(s):
    c = s["case"]
    B, Q, hq, D = s["q"].shape
    bs, G = c["block"], hq // c["hkv"]
    if c["hq"] * Q * sum(_lens(c)) * D > 4e12:
        return None
    out = torch.zeros(B, Q, hq, D, dtype=torch.float64, device=s["q"].device)
    words = s["mask"].cpu().numpy().astype(np.uint32)
    see = torch.from_numpy(np.unpackbits(words.view(np.uint8), axis=-1, bitorder="little")[:, :, :Q].astype(bool))
    for b, n in enumerate(_lens(c)):
        draft = torch.arange(n, n + Q, device=out.device)
        for h in range(c["hkv"]):
            if c["select"]:
                blk = s["sel_ids"][b, h, : int(s["sel_count"][b, h])].long()
                t = (blk[:, None] * bs + torch.arange(bs, device=out.device)).reshape(-1)
                t = t[t < n]
            else:
                t = torch.arange(n, device=out.device)
            t = torch.cat([t, draft])
            page = s["block_table"][b].long()[t // bs]
            k, v = s["k_pages"][page, h, t % bs].double(), s["v_pages"][page, h, t % bs].double()
            ok = torch.cat([torch.ones(Q, t.numel() - Q, dtype=torch.bool), see[b]], 1).to(out.device)
            for head in range(h * G, (h + 1) * G):
                logit = torch.einsum("qd,td->qt", s["q"][b, :, head].double(), k) * D ** -0.5
                weight = torch.softmax(torch.where(ok, logit, torch.full_like(logit, -math.inf)), dim=1)
                out[b, :, head] = torch.einsum("qt,td->qd", torch.nan_to_num(weight), v)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "tree": _exact_tree, "commit": _exact_commit}[case["op"]](s)
