"""Timed cases of the operators that serve long contexts from the paged K/V cache.

* ``norm``: new tokens enter the cache; queries and keys get their norm for each head and the
  rotation of their position, which may have several axes, on the way.
* ``shared``: attention of a batch whose groups of sequences share a long prefix.
* ``weigh``: attention that also adds up the weight which each cached token got.
* ``evict``: the tokens with the largest weights are kept, in new pages, the others dropped.

``run`` computes them in elementary torch operations, or with the library's calls when
``own`` is set.  Layouts are those of include/sparse_attn.h.
"""
import math

import numpy as np
import torch

own = False

HALVES, PAIRS = 1, 2                       # channel pairing of the rotation
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _norm(name, **kw):
    base = dict(op="norm", batch=1, rows=1, context=4096, ragged=False, hq=32, hkv=8, dim=128, block=32, dtype="bf16",
                kv="bf16", rotary=128, pairing=HALVES, axes=1, per_head=False, box=True, fused_input=True)
    return {"name": name, **base, **kw}


def _shared(name, **kw):
    base = dict(op="shared", batch=8, groups=1, prefix=4096, context=512, drafts=1, ragged=True, hq=32, hkv=8, dim=128,
                block=32, dtype="bf16", kv="bf16", tree=False)
    return {"name": name, **base, **kw}


def _weigh(name, **kw):
    base = dict(op="weigh", batch=1, context=4096, drafts=1, ragged=False, hq=32, hkv=8, dim=128, block=32, dtype="bf16",
                kv="bf16")
    return {"name": name, **base, **kw}


def _evict(name, **kw):
    base = dict(op="evict", batch=1, context=4096, keep=1024, sinks=4, recent=128, ragged=False, hq=32, hkv=8, dim=128,
                block=32, dtype="bf16", kv="bf16", box=False)
    return {"name": name, **base, **kw}


def listed():
    return [
        # one user's next token far into a 128K context: nothing but latency
        _norm("norm_one_token", context=131071),
        # prompts of all lengths with images in them (time, height, width), packed behind cached prefixes
        _norm("norm_ragged_prompts_3_axes", batch=16, rows=4001, context=1500, ragged=True, block=64, axes=3),
        # an fp32 cache, two axes on a part of the channels in neighbouring pairs, odd counts, a weight for each head
        _norm("norm_fp32_partial_2_axes", batch=3, rows=333, context=777, ragged=True, hq=4, hkv=4, dim=64, block=64,
              dtype="f32", kv="f32", rotary=32, pairing=PAIRS, axes=2, per_head=True, fused_input=False),
        # four samples of one short prompt
        _shared("shared_few_samples", batch=4, prefix=777, context=50),
        # a serving batch behind one long system prompt or document
        _shared("shared_document", batch=64, prefix=32768, context=1024, block=64),
        # several tenants' prompts, draft trees of every user
        _shared("shared_tenants_trees", batch=48, groups=6, prefix=16384, context=2000, drafts=5, tree=True, block=64),
        # one user's single token over a short context
        _weigh("weigh_one_token"),
        # a serving batch's next tokens over contexts of all lengths
        _weigh("weigh_batch", batch=16, context=32768, ragged=True, block=64),
        # the last tokens of long prompts, by whose attention the first eviction goes
        _weigh("weigh_window", batch=4, context=32768, drafts=32, block=64),
        # one user's context down to a quarter
        _evict("evict_one", context=8192, keep=2048),
        # a batch of contexts of all lengths, with the selection's key box
        _evict("evict_batch", batch=16, context=32768, keep=8192, ragged=True, block=64, box=True),
        # one very long context: few rows of weights, each long
        _evict("evict_long", context=131072, keep=16384),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "shared", "shared", "weigh", "weigh", "evict"])
    hkv, group, dim = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    c = dict(op=op, batch=_log(rng, 1, 128), context=_log(rng, 1, 131072), ragged=rng.random() < 0.6,
             hq=hkv * group, hkv=hkv, dim=dim, block=rng.choice([16, 32, 64, 128]), dtype="bf16", kv="bf16")
    kind = rng.random()
    if kind < 0.2:
        c["dtype"] = "f32"
    if kind < 0.12:
        c["kv"] = "f32"
    most = 520000                          # cached tokens of the batch
    if c["dtype"] == "f32":
        most = 66000                       # the larger part of fp32 use: checks at moderate lengths
    if op == "norm":
        c.update(rows=_log(rng, 1, 8192), rotary=rng.choice([dim, dim, dim // 2]), pairing=rng.choice([HALVES, PAIRS]),
                 axes=rng.choice([1, 1, 2, 3, 4]), per_head=rng.random() < 0.2, box=rng.random() < 0.7,
                 fused_input=rng.random() < 0.7)
        size, most = c["rows"], 60000
    elif op == "shared":
        c["groups"] = _log(rng, 1, c["batch"])
        c.update(prefix=_log(rng, 1, 65536), context=_log(rng, 1, 4096), tree=rng.random() < 0.3,
                 drafts=rng.choice([1, 1, 1, _log(rng, 2, 16)]))
        size = c["prefix"] // max(1, c["batch"] // c["groups"]) + c["context"] + c["drafts"]
    elif op == "weigh":
        c["drafts"] = rng.choice([1, 1, _log(rng, 2, 64)])
        size = c["context"] + c["drafts"]
    else:
        c.update(sinks=rng.choice([0, 1, 4]), recent=rng.choice([0, _log(rng, 1, 256)]), box=rng.random() < 0.5)
        c["keep"] = max(c["sinks"] + c["recent"], 1, _log(rng, 1, max(1, c["context"] // 2)))
        size = c["context"] + c["keep"]
    # pools of moderate size, and no more work than the largest listed case
    most = min(most * 8 // hkv, 2000000)
    if size > most:
        if op == "norm":
            c["rows"] = most
        else:
            c["context"] = max(1, most // 4)
        size = most
    c["batch"] = max(1, min(c["batch"], most // size, 2000000 // (c["context"] + size)))
    if op == "shared":
        c["groups"] = min(c["groups"], c["batch"])
    top = [max(w[k] for w in map(work, listed())) for k in ("bytes", "flops")]
    while work(c)["bytes"] > top[0] or work(c)["flops"] > top[1]:
        if c["batch"] > 1:
            c["batch"] = max(1, c["batch"] * 3 // 4)
            if op == "shared":
                c["groups"] = min(c["groups"], c["batch"])
        elif op == "shared" and c["prefix"] > c["context"]:
            c["prefix"] = c["prefix"] * 3 // 4
        else:
            c["context"] = c["context"] * 3 // 4
    return c


# ------------------------------------------------------------------ sizes --

def _spread(n, most, step):
    """n whole numbers in [most // 2, most], the first one `most`; a function of the case alone."""
    return [most - (i * step) % (most // 2 + 1) for i in range(n)]


def _members(c):
    """First sequence of every group, and the batch's end: groups of uneven sizes."""
    B, n = c["batch"], c["groups"]
    cuts = [B * i // n for i in range(n + 1)]
    if c["ragged"]:                        # every second cut moves left where a group of two or more allows it
        for i in range(1, n, 2):
            if cuts[i] - cuts[i - 1] > 1:
                cuts[i] -= 1
    return cuts


def _prefixes(c):
    return _spread(c["groups"], c["prefix"], 7919) if c["ragged"] else [c["prefix"]] * c["groups"]


def _lens(c):
    """Cached tokens of each sequence."""
    part = _spread(c["batch"], c["context"], 7919) if c["ragged"] else [c["context"]] * c["batch"]
    if c["op"] != "shared":
        return part
    cuts, first = _members(c), _prefixes(c)
    return [first[g] + part[b] for g in range(c["groups"]) for b in range(cuts[g], cuts[g + 1])]


def _counts(c):
    """New rows of each sequence."""
    return _spread(c["batch"], c["rows"], 613) if c["ragged"] else [c["rows"]] * c["batch"]


def work(case):
    c = case
    e, ekv, D, hkv = (2 if c["dtype"] == "bf16" else 4), (2 if c["kv"] == "bf16" else 4), c["dim"], c["hkv"]
    lens = _lens(c)
    token = 2 * hkv * D * ekv                              # K and V of one token
    if c["op"] == "norm":
        n = sum(_counts(c))
        b = n * (2 * c["hq"] + 2 * hkv) * D * e + n * token + n * 4 * c["axes"]
        if c["box"]:
            for old, add in zip(lens, _counts(c)):
                first, last = old // c["block"], (old + add - 1) // c["block"]
                b += token * (last - first + 1 + (1 if old % c["block"] else 0))
        return {"bytes": b, "flops": n * (c["hq"] + hkv) * (4 * D + 3 * c["rotary"])}
    if c["op"] == "evict":
        kept = [min(n, c["keep"]) for n in lens]
        b = 4 * hkv * sum(lens) + sum(kept) * (2 * token + 8 * hkv)
        if c["box"]:
            b += token * sum(-(-k // c["block"]) for k in kept)
        return {"bytes": b, "flops": 0}
    Q = c["drafts"]
    rows = c["batch"] * Q * c["hq"]
    seen = sum(lens) + c["batch"] * Q
    if c["op"] == "shared":
        cuts, first = _members(c), _prefixes(c)
        keys = seen - sum(p * (cuts[g + 1] - cuts[g] - 1) for g, p in enumerate(first))
        b = keys * token + rows * D * (e + 4) + 4 * (keys // c["block"] + c["batch"])
    else:
        b = seen * token + rows * D * (e + 4) + 8 * hkv * sum(lens) + 4 * (seen // c["block"] + c["batch"])
    return {"bytes": b, "flops": 4 * Q * c["hq"] * D * seen}


# ----------------------------------------------------------------- inputs --

def _see(c, g):
    """[B, Q, Q] truth values: the drafts that a draft sees, its ancestors and itself."""
    B, Q = c["batch"], c["drafts"]
    parent = torch.arange(-1, Q - 1, device="cuda").expand(B, Q).clone()
    if c.get("tree"):
        parent = (torch.rand(B, Q, generator=g, device="cuda") * torch.arange(Q, device="cuda")).long()
        parent[:, 0] = -1
    step = (parent[:, :, None] == torch.arange(Q, device="cuda")) | torch.eye(Q, dtype=torch.bool, device="cuda")
    return torch.linalg.matrix_power(step.double(), Q) > 0.5       # at most 2^Q walks: exact enough to tell from none


def _pack_bits(see):
    """[B, Q, Q] truth values -> [B, Q, ceil(Q / 32)] int32 words, bit j % 32 of word j // 32."""
    B, Q, _ = see.shape
    W = -(-Q // 32)
    bits = torch.zeros(B, Q, W * 32, dtype=torch.int64, device=see.device)
    bits[:, :, :Q] = see
    words = (bits.view(B, Q, W, 32) << torch.arange(32, device=see.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _int(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _cache(s, c, normal, g, nb_cap):
    """Page table and pools; the sequences of a group share the whole blocks of their prefix."""
    B, bs, dev = c["batch"], c["block"], "cuda"
    extra = B * -(-c["keep"] // bs) if c["op"] == "evict" else 0
    if c["op"] == "shared":
        table = torch.empty(B, nb_cap, dtype=torch.int64)
        cuts, at, copies = _members(c), 0, []
        for n, p in enumerate(_prefixes(c)):
            whole = p // bs
            for b in range(cuts[n], cuts[n + 1]):
                table[b, :whole] = torch.arange(at, at + whole)
            at += whole
            for b in range(cuts[n], cuts[n + 1]):
                table[b, whole:] = torch.arange(at, at + nb_cap - whole)
                if p % bs and b > cuts[n]:  # the block that the prefix ends in: everybody fills a copy
                    copies.append((int(table[cuts[n], whole]), int(table[b, whole]), p % bs))
                at += nb_cap - whole
        pages = at
    else:
        table, copies, pages = torch.arange(B * nb_cap).view(B, nb_cap), [], B * nb_cap + extra
    order = torch.randperm(pages, generator=g, device=dev)
    s["num_pages"] = pages
    s["block_table"] = order[table.to(dev)].to(torch.int32)
    s["k_pages"] = normal(pages, c["hkv"], bs, c["dim"], dtype=DTYPES[c["kv"]])
    s["v_pages"] = normal(pages, c["hkv"], bs, c["dim"], dtype=DTYPES[c["kv"]])
    if extra:
        s["new_table"] = order[B * nb_cap:].to(torch.int32).view(B, -1).contiguous()
    for src, dst, n in copies:
        for pool in (s["k_pages"], s["v_pages"]):
            pool[order[dst], :, :n] = pool[order[src], :, :n]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62))
    dev, B, D, bs, hq, hkv = "cuda", c["batch"], c["dim"], c["block"], c["hq"], c["hkv"]
    dt, kvt = DTYPES[c["dtype"]], DTYPES[c["kv"]]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    lens = _lens(c)
    longest = max(lens)
    capacity = longest + {"norm": c.get("rows"), "evict": 0}.get(c["op"], c.get("drafts"))
    if c["op"] == "evict":
        capacity = max(capacity, c["keep"])
    nb_cap = -(-capacity // bs)
    s = {"case": c, "capacity": capacity, "lens": _int(lens)}
    _cache(s, c, normal, g, nb_cap)
    if c.get("box"):
        # a box as N(0, 1) keys leave it, around zero
        s["kmin"] = -normal(B, hkv, nb_cap, D, dtype=kvt).abs() - 1.5
        s["kmax"] = normal(B, hkv, nb_cap, D, dtype=kvt).abs() + 1.5

    if c["op"] == "norm":
        counts = _counts(c)
        n = sum(counts)
        if c["fused_input"]:               # one projection's output, [rows, q | k | v]
            q, k, v = normal(n, (hq + 2 * hkv) * D).split([hq * D, hkv * D, hkv * D], dim=1)
        else:
            q, k, v = normal(n, hq * D), normal(n, hkv * D), normal(n, hkv * D)
        s["q_new"], s["k_new"], s["v_new"] = q.view(n, hq, D), k.view(n, hkv, D), v.view(n, hkv, D)
        s["q_weight"] = 1 + 0.2 * normal(*((hq, D) if c["per_head"] else (D,)), dtype=torch.float32)
        s["k_weight"] = 1 + 0.2 * normal(*((hkv, D) if c["per_head"] else (D,)), dtype=torch.float32)
        s["cu_rows"] = _int(np.cumsum([0] + counts).tolist())
        s["row_seq"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(counts, device=dev), output_size=n)
        half = c["rotary"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        if c["axes"] > 1:
            # a place in time for every row, and a row and a column of an image that begins there
            token = s["lens"][s["row_seq"]] + torch.arange(n, device=dev) - s["cu_rows"][s["row_seq"]]
            grid = torch.randint(0, 64, (c["axes"], n), generator=g, device=dev)
            grid[0] = 0
            s["positions"] = (token + grid).to(torch.int32).contiguous()
            # the channels' axes: sections of the frequencies, or in turn
            i = torch.arange(half, device=dev)
            s["axis_of"] = (i * c["axes"] // half if c["pairing"] == HALVES else i % c["axes"]).to(torch.int32)
        s["q_out"] = torch.empty(n, hq, D, dtype=dt, device=dev)
    elif c["op"] == "evict":
        # sums of weights as attention leaves them: few tokens have most of it, some never had any
        w = torch.randn(B, hkv, nb_cap * bs, generator=g, device=dev).mul(2.0).exp()
        s["weights"] = torch.where(torch.rand(w.shape, generator=g, device=dev) < 0.1, torch.zeros_like(w), w)
        s["kept"] = torch.full((B, hkv, c["keep"]), -1, dtype=torch.int32, device=dev)
        s["new_lens"] = torch.empty(B, dtype=torch.int32, device=dev)
    else:
        Q = c["drafts"]
        s["q"] = normal(B, Q, hq, D)
        s["out"] = torch.empty(B, Q, hq, D, dtype=torch.float32, device=dev)
        s["see"] = _see(c, g)
        if c["op"] == "shared":
            cuts = _members(c)
            s["cu_seqs"], s["prefix_lens"] = _int(cuts), _int(_prefixes(c))
            sizes = [cuts[i + 1] - cuts[i] for i in range(c["groups"])]
            s["group_of"] = torch.repeat_interleave(torch.arange(c["groups"], device=dev), torch.tensor(sizes, device=dev),
                                                    output_size=B)
            s["most_members"] = max(sizes)
            s["mask"] = _pack_bits(s["see"]) if c["tree"] else None
        else:
            s["weights"] = torch.rand(B, hkv, nb_cap * bs, generator=g, device=dev)
    if own:
        from query_guided_block_gb300 import binding as lib
        p = s["params"] = lib.make_params(B, hq, hkv, D, longest, bs, s["num_pages"], 0, 1, kv_dtype=kvt, q_dtype=dt,
                                          num_queries=c.get("drafts", 1), capacity_tokens=capacity)
        size = {"norm": lambda: 256, "shared": lambda: lib.sparse_attn_shared_workspace_size(p, c["groups"]),
                "weigh": lambda: lib.sparse_attn_weigh_workspace_size(p),
                "evict": lambda: lib.sparse_attn_evict_workspace_size(p, c["keep"])}[c["op"]]()
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=dev)
        lib.sparse_attn_workspace_init(s["ws"])
    return s


# ----------------------------------------------------------- plain forms --

def _rms(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight


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


def _plain_norm(s):
    c = s["case"]
    seq = s["row_seq"]
    old = s["lens"].long()[seq]
    token = old + torch.arange(seq.numel(), device=seq.device) - s["cu_rows"].long()[seq]
    if c["axes"] > 1:
        angle = s["positions"].double()[s["axis_of"].long()].t() * s["inv_freq"]
    else:
        angle = token.double()[:, None] * s["inv_freq"]
    q = _rotate(_rms(s["q_new"].float(), s["q_weight"]), angle, c["rotary"], c["pairing"]).to(s["q_new"].dtype)
    k = _rotate(_rms(s["k_new"].float(), s["k_weight"]), angle, c["rotary"], c["pairing"]).to(s["k_pages"].dtype)
    page = s["block_table"].long()[seq, token // c["block"]]
    s["k_pages"][page, :, token % c["block"]] = k
    s["v_pages"][page, :, token % c["block"]] = s["v_new"].to(s["v_pages"].dtype)
    out = {"q": q, "k": s["k_pages"], "v": s["v_pages"]}
    if c["box"]:
        _widen_box(s, seq, token, old, k)
        out.update(kmin=s["kmin"], kmax=s["kmax"])
    return out


def _context(s, table, blocks):
    """K and V of the first `blocks` blocks of every row of the table, [rows, Hkv, tokens, D] fp32."""
    page = table.long()[:, :blocks]
    return [s[n][page].float().permute(0, 2, 1, 3, 4).flatten(2, 3) for n in ("k_pages", "v_pages")]


def _drafts(s):
    """K and V of the drafts, [B, Hkv, Q, D] fp32."""
    c = s["case"]
    at = s["lens"].long()[:, None] + torch.arange(c["drafts"], device=s["q"].device)
    page = torch.gather(s["block_table"].long(), 1, at // c["block"])
    return [s[n][page, :, at % c["block"]].float().transpose(1, 2) for n in ("k_pages", "v_pages")]


def _rows(s):
    """Queries [B, Hkv, Q * G, D] fp32: the rows of a KV head."""
    B, Q, hq, D = s["q"].shape
    hkv = s["case"]["hkv"]
    return s["q"].float().view(B, Q, hkv, hq // hkv, D).transpose(1, 2).flatten(2, 3)


def _unrows(s, out):
    B, Q, hq, D = s["q"].shape
    hkv = s["case"]["hkv"]
    return out.view(B, hkv, Q, hq // hkv, D).transpose(1, 2).reshape(B, Q, hq, D)


def _draft_rows(s):
    """[B, 1, Q * G, Q]: what the rows see of the drafts."""
    return s["see"].repeat_interleave(s["case"]["hq"] // s["case"]["hkv"], 1)[:, None]


def _plain_shared(s):
    c = s["case"]
    bs, dev = c["block"], s["q"].device
    scale = 1 / math.sqrt(c["dim"])
    q, group, cu = _rows(s), s["group_of"], s["cu_seqs"].long()
    prefix = s["prefix_lens"].long()
    # the prefix, once a group: the members' rows side by side
    place = torch.arange(c["batch"], device=dev) - cu[group]
    side = torch.zeros(c["groups"], s["most_members"], *q.shape[1:], device=dev)
    side[group, place] = q
    side = side.transpose(1, 2).flatten(2, 3)                              # [groups, Hkv, members * rows, D]
    blocks = -(-c["prefix"] // bs)
    k, v = _context(s, s["block_table"][cu[:-1]], blocks)
    score = side @ k.transpose(-1, -2) * scale
    score = score.masked_fill(torch.arange(blocks * bs, device=dev) >= prefix[:, None, None, None], -math.inf)
    top_a = score.amax(-1, keepdim=True)
    p = (score - top_a).exp()
    sum_a, out_a = p.sum(-1, keepdim=True), p @ v

    def of_sequences(x):
        return x.unflatten(2, (s["most_members"], -1)).transpose(1, 2)[group, place]

    top_a, sum_a, out_a = of_sequences(top_a), of_sequences(sum_a), of_sequences(out_a)
    # every sequence's own tokens: the blocks from the one that the prefix ends in
    first = prefix[group] // bs
    blocks = -(-c["context"] // bs) + 1
    own_blocks = (first[:, None] + torch.arange(blocks, device=dev)).clamp(max=s["block_table"].shape[1] - 1)
    k, v = _context(s, torch.gather(s["block_table"].long(), 1, own_blocks), blocks)
    token = first[:, None] * bs + torch.arange(blocks * bs, device=dev)
    there = (token >= prefix[group][:, None]) & (token < s["lens"].long()[:, None])
    kd, vd = _drafts(s)
    score = (q @ k.transpose(-1, -2) * scale).masked_fill(~there[:, None, None], -math.inf)
    score_d = (q @ kd.transpose(-1, -2) * scale).masked_fill(~_draft_rows(s), -math.inf)
    top = torch.maximum(top_a, torch.maximum(score.amax(-1, keepdim=True), score_d.amax(-1, keepdim=True)))
    p, pd, wa = (score - top).exp(), (score_d - top).exp(), (top_a - top).exp()
    total = p.sum(-1, keepdim=True) + pd.sum(-1, keepdim=True) + wa * sum_a
    return _unrows(s, (p @ v + pd @ vd + wa * out_a) / total)


def _plain_weigh(s):
    c = s["case"]
    bs, dev, Q, hkv = c["block"], s["q"].device, c["drafts"], c["hkv"]
    scale = 1 / math.sqrt(c["dim"])
    q, lens = _rows(s), s["lens"].long()
    blocks = -(-c["context"] // bs)
    k, v = _context(s, s["block_table"], blocks)
    kd, vd = _drafts(s)
    token = torch.arange(blocks * bs, device=dev)
    there = token < lens[:, None]
    score = (q @ k.transpose(-1, -2) * scale).masked_fill(~there[:, None, None], -math.inf)
    score_d = (q @ kd.transpose(-1, -2) * scale).masked_fill(~_draft_rows(s), -math.inf)
    top = torch.maximum(score.amax(-1, keepdim=True), score_d.amax(-1, keepdim=True))
    p, pd = (score - top).exp(), (score_d - top).exp()
    total = p.sum(-1, keepdim=True) + pd.sum(-1, keepdim=True)
    out = (p @ v + pd @ vd) / total
    w = s["weights"]
    w[:, :, : blocks * bs] += (p / total).sum(2)                           # zero behind the context
    at = lens[:, None, None] + torch.arange(Q, device=dev)
    w.scatter_(2, at.expand(-1, hkv, -1), (pd / total).sum(2))
    return {"out": _unrows(s, out), "weights": w}


def _plain_evict(s):
    c = s["case"]
    B, hkv, bs, keep, dev = c["batch"], c["hkv"], c["block"], c["keep"], s["lens"].device
    lens = s["lens"].long()[:, None, None]
    n = c["context"]
    token = torch.arange(n, device=dev)
    key = s["weights"][:, :, :n].masked_fill((token < c["sinks"]) | (token >= lens - c["recent"]), math.inf)
    key = key.masked_fill(token >= lens, -1.0)                             # behind everything
    order = key.argsort(dim=-1, descending=True, stable=True)[..., :keep]
    count = lens.clamp(max=keep)                                           # [B, 1, 1]
    ids = order.masked_fill(torch.arange(order.shape[-1], device=dev) >= count, n).sort(dim=-1).values
    live = ids < n
    b, h, i = live.nonzero(as_tuple=True)
    t = ids[b, h, i]
    src, dst = s["block_table"].long()[b, t // bs], s["new_table"].long()[b, i // bs]
    k = s["k_pages"][src, h, t % bs]
    s["k_pages"][dst, h, i % bs] = k
    s["v_pages"][dst, h, i % bs] = s["v_pages"][src, h, t % bs]
    s["weights"][b, h, i] = s["weights"][b, h, t]
    s["kept"][b, h, i] = t.to(torch.int32)
    out = {"k": s["k_pages"], "v": s["v_pages"], "weights": s["weights"], "kept": s["kept"],
           "lens": count.view(B).to(torch.int32)}
    if c["box"]:
        nb_cap, D = s["kmin"].shape[2:]
        row = (b * hkv + h) * nb_cap + i // bs
        for name, start, how in (("kmin", math.inf, "amin"), ("kmax", -math.inf, "amax")):
            flat = s[name].view(-1, D)
            new = flat.float()
            new[row] = start
            new.scatter_reduce_(0, row[:, None].expand(-1, D), k.float(), how)
            flat.copy_(new)
            out[name] = s[name]
    return out


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"norm": _plain_norm, "shared": _plain_shared, "weigh": _plain_weigh, "evict": _plain_evict}[c["op"]](s)
    from query_guided_block_gb300 import binding as lib
    p, ws = s["params"], s["ws"]
    if c["op"] == "norm":
        lib.sparse_attn_append_kv_norm(p, s["q_new"], s["k_new"], s["v_new"], s["q_weight"], s["k_weight"], EPS, s["inv_freq"],
                                       s["q_out"], s["k_pages"], s["v_pages"], s["block_table"], ws, cu_rows=s["cu_rows"],
                                       seq_lens=s["lens"], positions=s.get("positions"), axis_of=s.get("axis_of"),
                                       pairing=c["pairing"], kmin=s.get("kmin"), kmax=s.get("kmax"))
        out = {"q": s["q_out"], "k": s["k_pages"], "v": s["v_pages"]}
    elif c["op"] == "shared":
        lib.sparse_attn_shared_decode(p, s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["cu_seqs"], s["prefix_lens"],
                                      s["out"], ws, seq_lens=s["lens"], tree_mask=s["mask"])
        return s["out"]
    elif c["op"] == "weigh":
        lib.sparse_attn_weigh_decode(p, s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["weights"], s["out"], ws,
                                     seq_lens=s["lens"])
        return {"out": s["out"], "weights": s["weights"]}
    else:
        lib.sparse_attn_evict_tokens(p, c["keep"], c["sinks"], c["recent"], s["weights"], s["k_pages"], s["v_pages"],
                                     s["block_table"], s["new_table"], s["kept"], s["new_lens"], ws, seq_lens=s["lens"],
                                     kmin=s.get("kmin"), kmax=s.get("kmax"))
        out = {"k": s["k_pages"], "v": s["v_pages"], "weights": s["weights"], "kept": s["kept"], "lens": s["new_lens"]}
    if c["box"]:
        out.update(kmin=s["kmin"], kmax=s["kmax"])
    return out


# ---------------------------------------------- the definitions in 64 bits --

def _exact_norm(s):
    c = s["case"]
    bs, half = c["block"], c["rotary"] // 2
    q, k = s["q_new"].double(), s["k_new"].double()
    q, k = (x / (x.square().sum(-1, keepdim=True) / c["dim"] + EPS).sqrt() * s[w].double()
            for x, w in ((q, "q_weight"), (k, "k_weight")))
    one = list(range(half)) if c["pairing"] == HALVES else list(range(0, c["rotary"], 2))
    two = list(range(half, c["rotary"])) if c["pairing"] == HALVES else list(range(1, c["rotary"], 2))
    pools = {"k": s["k_pages"].double(), "v": s["v_pages"].double()}
    box = {n: s[n].double() for n in ("kmin", "kmax") if n in s}
    r = 0
    for b, (old, count) in enumerate(zip(_lens(c), _counts(c))):
        t = torch.arange(old, old + count, device=q.device)
        at = t.double()[None].expand(half, -1)
        if c["axes"] > 1:
            at = torch.stack([s["positions"][int(a), r:r + count].double() for a in s["axis_of"]])
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=q.device), (at * s["inv_freq"][:, None]).t())[:, None]
        for x in (q, k):
            z = torch.complex(x[r:r + count][..., one], x[r:r + count][..., two]) * turn
            x[r:r + count, :, one] = z.real
            x[r:r + count, :, two] = z.imag
        page = s["block_table"][b].long()[t // bs]
        pools["k"][page, :, t % bs] = k[r:r + count]
        pools["v"][page, :, t % bs] = s["v_new"][r:r + count].double()
        for blk in range(old // bs, (old + count - 1) // bs + 1) if box else ():
            lo, hi = max(old, blk * bs), min(old + count, (blk + 1) * bs)
            part = k[r + lo - old:r + hi - old]
            for name, how in (("kmin", torch.minimum), ("kmax", torch.maximum)):
                new = part.amin(0) if name == "kmin" else part.amax(0)
                box[name][b, :, blk] = how(new, box[name][b, :, blk]) if blk * bs < old else new
        r += count
    return {"q": q, **pools, **box}


def _exact_attention(s, weigh):
    c = s["case"]
    B, Q, hq, D = s["q"].shape
    bs, G, dev = c["block"], hq // c["hkv"], s["q"].device
    lens = _lens(c)
    if hq * Q * sum(lens) * D > 4e12:
        return None
    out = torch.zeros(B, Q, hq, D, dtype=torch.float64, device=dev)
    weights = s["weights"].double() if weigh else None
    for b, n in enumerate(lens):
        t = torch.arange(n + Q, device=dev)
        page = s["block_table"][b].long()[t // bs]
        ok = torch.cat([torch.ones(Q, n, dtype=torch.bool, device=dev), s["see"][b]], 1)
        for h in range(c["hkv"]):
            k, v = s["k_pages"][page, h, t % bs].double(), s["v_pages"][page, h, t % bs].double()
            if weigh:
                weights[b, h, n:n + Q] = 0
            for head in range(h * G, (h + 1) * G):
                logit = torch.einsum("qd,td->qt", s["q"][b, :, head].double(), k) * D ** -0.5
                weight = torch.softmax(torch.where(ok, logit, torch.full_like(logit, -math.inf)), dim=1)
                out[b, :, head] = torch.einsum("qt,td->qd", weight, v)
                if weigh:
                    weights[b, h, :n + Q] += weight.sum(0)
    return {"out": out, "weights": weights} if weigh else out


def _exact_evict(s):
    c = s["case"]
    bs, dev = c["block"], s["lens"].device
    pools = {"k": s["k_pages"].double(), "v": s["v_pages"].double()}
    box = {n: s[n].double() for n in ("kmin", "kmax") if n in s}
    weights, kept = s["weights"].double(), s["kept"].clone()
    for b, n in enumerate(_lens(c)):
        for h in range(c["hkv"]):
            row = weights[b, h].cpu().numpy()
            if n <= c["keep"]:
                ids = np.arange(n)
            else:
                sure = np.r_[0:c["sinks"], n - c["recent"]:n]
                rest = np.arange(c["sinks"], n - c["recent"])
                rest = rest[np.lexsort((rest, -row[rest]))][: c["keep"] - sure.size]
                ids = np.sort(np.r_[sure, rest])
            t, i = torch.from_numpy(ids).to(dev), torch.arange(len(ids), device=dev)
            src, dst = s["block_table"][b].long()[t // bs], s["new_table"][b].long()[i // bs]
            for pool in pools.values():
                pool[dst, h, i % bs] = pool[src, h, t % bs]
            weights[b, h, : len(ids)] = torch.from_numpy(row[ids]).to(dev)
            kept[b, h, : len(ids)] = t.to(torch.int32)
            for blk in range(-(-len(ids) // bs) if box else 0):
                part = pools["k"][s["new_table"][b, blk].long(), h, : min(bs, len(ids) - blk * bs)]
                box["kmin"][b, h, blk], box["kmax"][b, h, blk] = part.amin(0), part.amax(0)
    return {**pools, "weights": weights, "kept": None, "lens": None, **box}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "shared": lambda x: _exact_attention(x, False), "weigh": lambda x: _exact_attention(x, True),
            "evict": _exact_evict}[case["op"]](s)
