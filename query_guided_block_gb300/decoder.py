"""Device-buffer plumbing around the C ABI: allocates, with torch, the tensors one
decode problem needs and calls the entry points in order.  No arithmetic of the method
happens here."""
from __future__ import annotations

from typing import Optional

import torch

from . import binding as B


class SparseDecoder:
    """Owns metadata, selection, output and workspace buffers for one problem.

    The KV page pools, block table and queries belong to the caller.
    """

    def __init__(self, params: B.sparse_attn_params, device="cuda"):
        self.p = params
        self.device = torch.device(device)
        p = params
        self.nb = B.sparse_attn_num_blocks(p)
        self.sel_stride = B.sparse_attn_sel_stride(p)
        self.units = p.batch * p.num_kv_heads
        kv = torch.bfloat16 if p.kv_dtype == B.BF16 else torch.float32
        self.kv_dtype = kv
        dev = self.device
        rows_blk, rows_mean = B.meta_rows(p)             # capacity, >= the context's rows
        self.kmin = torch.empty(p.batch, p.num_kv_heads, rows_blk, p.head_dim, dtype=kv, device=dev)
        self.kmax = torch.empty_like(self.kmin)
        self.needs_mean = bool(p.two_level) or p.score_kind == B.SCORE_MEAN
        self.kmean = None
        if self.needs_mean:
            self.kmean = torch.empty(p.batch, p.num_kv_heads, rows_mean, p.head_dim, dtype=torch.float32,
                                     device=dev)
        self.ws_bytes = B.sparse_attn_workspace_size(p)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        B.sparse_attn_workspace_init(self.ws)
        self.sel_ids = torch.empty(p.batch, p.num_kv_heads, self.sel_stride, dtype=torch.int32,
                                   device=dev)
        self.sel_count = torch.empty(p.batch, p.num_kv_heads, dtype=torch.int32, device=dev)
        self.Q = max(1, p.num_queries)
        out_shape = ((p.batch, self.Q, p.num_q_heads, p.head_dim) if self.Q > 1
                     else (p.batch, p.num_q_heads, p.head_dim))
        self.out = torch.empty(out_shape, dtype=torch.float32, device=dev)

    def metadata_bytes(self) -> int:
        n = self.kmin.numel() * self.kmin.element_size() * 2
        if self.kmean is not None:
            n += self.kmean.numel() * 4
        return n

    def build_meta(self, k_pages, block_table, stream=None):
        B.sparse_attn_build_meta(self.p, k_pages, block_table, self.kmin, self.kmax, self.kmean,
                                 self.ws, stream)

    def append_meta(self, n_old, k_pages, block_table, stream=None):
        """Metadata after tokens [n_old, p.n_tokens) were appended to the pages."""
        B.sparse_attn_append_meta(self.p, n_old, k_pages, block_table, self.kmin, self.kmax,
                                  self.kmean, self.ws, stream)

    def select(self, q, reserve_ids=None, stream=None):
        """Selection; with ``reserve_ids`` [B, Hkv, num_reserve] int32 (drawn by the caller)
        the reserve set is united with every unit's top-k."""
        if self.p.num_reserve > 0:
            if reserve_ids is None:
                raise ValueError("this problem has num_reserve > 0: pass reserve_ids")
            B.sparse_attn_select_reserved(self.p, q, self.kmin, self.kmax, self.kmean, reserve_ids,
                                          self.sel_ids, self.sel_count, self.ws, stream)
            return
        B.sparse_attn_select(self.p, q, self.kmin, self.kmax, self.kmean, self.sel_ids,
                             self.sel_count, self.ws, stream)

    def decode(self, q, k_pages, v_pages, block_table, sel_ids=None, sel_count=None, out=None,
               stream=None):
        B.sparse_attn_decode(self.p, q, k_pages, v_pages, block_table,
                             self.sel_ids if sel_ids is None else sel_ids,
                             self.sel_count if sel_count is None else sel_count,
                             self.out if out is None else out, self.ws, stream)

    def step(self, q, k_pages, v_pages, block_table, reserve_ids=None, stream=None):
        """select + decode for one query batch (two launches); returns the output tensor."""
        self.select(q, reserve_ids, stream)
        self.decode(q, k_pages, v_pages, block_table, stream=stream)
        return self.out

    def step_fused(self, q, k_pages, v_pages, block_table, reserve_ids=None, stream=None):
        """select + decode for one query batch in one launch (sparse_attn_step); the same
        results as ``step``.  Raises SparseAttnError (unsupported) for two-level
        selection, fp32 K/V or several queries per sequence."""
        if self.p.num_reserve > 0 and reserve_ids is None:
            raise ValueError("this problem has num_reserve > 0: pass reserve_ids")
        B.sparse_attn_step(self.p, q, self.kmin, self.kmax, self.kmean, reserve_ids, k_pages, v_pages,
                           block_table, self.sel_ids, self.sel_count, self.out, self.ws, stream)
        return self.out

    def device_error(self, stream=None) -> int:
        return B.sparse_attn_get_device_error(self.ws, stream)

    def set_wait_limit(self, cycles: int, stream=None):
        """Bounded-wait limit of this decoder's kernels (SM clocks; 0 = the default)."""
        B.sparse_attn_workspace_set_wait_limit(self.ws, cycles, stream)


class SlotCache:
    """LRU slot-cache state and per-step diff outputs for ``sparse_attn_diff``."""

    def __init__(self, decoder: SparseDecoder, cache_slots: int):
        d = decoder
        dev = d.device
        u, w = d.units, d.sel_stride
        self.decoder = d
        self.cache_slots = cache_slots
        self.slot_block = torch.full((u, cache_slots), -1, dtype=torch.int32, device=dev)
        self.slot_last_use = torch.full((u, cache_slots), -1, dtype=torch.int32, device=dev)
        self.prev_ids = torch.full((u, w), -1, dtype=torch.int32, device=dev)
        self.prev_count = torch.zeros(u, dtype=torch.int32, device=dev)
        names = ("hit_ids", "miss_ids", "miss_slot", "evict_ids", "evict_slot", "new_ids",
                 "dropped_ids")
        self.lists = {n: torch.full((u, w), -1, dtype=torch.int32, device=dev) for n in names}
        self.counts = torch.zeros(u, 5, dtype=torch.int32, device=dev)

    def diff(self, step: int, sel_ids: Optional[torch.Tensor] = None,
             sel_count: Optional[torch.Tensor] = None, stream=None, sel_slot: Optional[torch.Tensor] = None):
        """The step's diff; with `sel_slot` also its slot map, in the same launch."""
        d = self.decoder
        ids = d.sel_ids if sel_ids is None else sel_ids
        cnt = d.sel_count if sel_count is None else sel_count
        L = self.lists
        args = (d.p, step, ids, cnt, self.prev_ids, self.prev_count, self.cache_slots,
                self.slot_block, self.slot_last_use, L["hit_ids"], L["miss_ids"],
                L["miss_slot"], L["evict_ids"], L["evict_slot"], L["new_ids"],
                L["dropped_ids"], self.counts)
        if sel_slot is None:
            B.sparse_attn_diff(*args, d.ws, stream)
        else:
            B.sparse_attn_diff_slots(*args, sel_slot, d.ws, stream)

    def advance(self, sel_ids: Optional[torch.Tensor] = None,
                sel_count: Optional[torch.Tensor] = None):
        """Remember this step's request set as the next step's previous set."""
        d = self.decoder
        self.prev_ids.copy_((d.sel_ids if sel_ids is None else sel_ids).view(self.prev_ids.shape))
        self.prev_count.copy_((d.sel_count if sel_count is None else sel_count).view(-1))


class SlotPool:
    """Per-unit slot pool of K/V page tiles fed from a host-resident page-first store:
    after the diff of a step, ``load_misses`` brings the misses in (one launch),
    ``slot_map`` finds each selected block's slot and ``decode`` attends through it;
    ``decode_io`` does the miss loads and the attention in one pass (after
    ``slot_map``), so that the transfer overlaps the attention over resident blocks."""

    def __init__(self, cache: SlotCache):
        d = cache.decoder
        p = d.p
        self.cache = cache
        shape = (d.units, cache.cache_slots, p.block_size, p.head_dim)
        self.pool_k = torch.zeros(shape, dtype=d.kv_dtype, device=d.device)
        self.pool_v = torch.zeros_like(self.pool_k)
        self.sel_slot = torch.full((d.units, d.sel_stride), -1, dtype=torch.int32, device=d.device)

    def tile_bytes(self) -> int:
        p = self.cache.decoder.p
        return p.block_size * p.head_dim * self.pool_k.element_size()

    def load_misses(self, host_k_pages, host_v_pages, block_table, stream=None):
        c, d = self.cache, self.cache.decoder
        B.sparse_attn_load_misses(d.p, host_k_pages, host_v_pages, block_table, c.lists["miss_ids"],
                                  c.lists["miss_slot"], c.counts, c.cache_slots, self.pool_k,
                                  self.pool_v, d.ws, stream)

    def slot_map(self, stream=None):
        c, d = self.cache, self.cache.decoder
        B.sparse_attn_slot_map(d.p, d.sel_ids, d.sel_count, c.slot_block, c.cache_slots,
                               self.sel_slot, d.ws, stream)

    def decode(self, q, out=None, stream=None):
        c, d = self.cache, self.cache.decoder
        B.sparse_attn_decode_slots(d.p, q, self.pool_k, self.pool_v, c.cache_slots, d.sel_ids,
                                   self.sel_slot, d.sel_count, d.out if out is None else out, d.ws,
                                   stream)

    def decode_io(self, q, host_k_pages, host_v_pages, block_table, out=None, stream=None):
        c, d = self.cache, self.cache.decoder
        B.sparse_attn_decode_slots_io(d.p, q, self.pool_k, self.pool_v, c.cache_slots, d.sel_ids,
                                      self.sel_slot, d.sel_count, host_k_pages, host_v_pages, block_table,
                                      c.lists["miss_ids"], c.lists["miss_slot"], c.counts,
                                      d.out if out is None else out, d.ws, stream)


class DraftDecoder:
    """Speculative decoding over a paged cache: puts drafted tokens behind every sequence's
    context, attends a tree of them over the context and each other, and moves the accepted
    path to the context's end.  Owns the context lengths, the output and the workspace; the
    page pools, the page table (and its key box) belong to the caller.  No call waits for
    the device, so a step can be captured into a CUDA graph.

    ``p.n_tokens`` is the longest context that ``decode`` and ``commit`` take.  A commit may
    carry a context past it (the pages reach as far as ``p.capacity_tokens``); from then on that
    sequence is treated as inactive, its rows of ``out`` stay as they were, and
    ``device_error`` reports ``ERR_LENGTH``, until ``p`` is replaced by parameters with a larger
    ``n_tokens``.  That may be done between any two calls, also to follow the contexts
    closely: the workspace does not depend on ``n_tokens``, and the kernels are chosen by it."""

    def __init__(self, params: B.sparse_attn_params, seq_lens: torch.Tensor):
        p = params
        self.p = p
        self.device = seq_lens.device
        self.Q = max(1, p.num_queries)
        self.seq_lens = seq_lens
        self.new_lens = torch.empty_like(seq_lens)
        self.out = torch.empty(p.batch, self.Q, p.num_q_heads, p.head_dim, dtype=torch.float32, device=self.device)
        with torch.cuda.device(self.device):
            self.ws = torch.empty(B.sparse_attn_tree_workspace_size(p), dtype=torch.uint8, device=self.device)
            B.sparse_attn_workspace_init(self.ws)

    def append(self, q_new, k_new, v_new, inv_freq, q_out, k_pages, v_pages, block_table, cu_rows=None,
               positions=None, pairing=B.ROTATE_HALVES, kmin=None, kmax=None, stream=None):
        """Tokens behind the contexts (drafts, or with ``kmin`` / ``kmax`` tokens that the
        selection's key box covers); the lengths stay as they are."""
        B.sparse_attn_append_kv(self.p, q_new, k_new, v_new, inv_freq, q_out, k_pages, v_pages, block_table, self.ws,
                                cu_rows, self.seq_lens, positions, pairing, kmin, kmax, stream)

    def decode(self, q, k_pages, v_pages, block_table, tree_mask=None, sel_ids=None, sel_count=None, stream=None):
        """Attention of the drafts [B, Q, Hq, D]; returns the output tensor."""
        B.sparse_attn_tree_decode(self.p, q, k_pages, v_pages, block_table, self.out.view(q.shape), self.ws,
                                  self.seq_lens, sel_ids, sel_count, tree_mask, stream)
        return self.out

    def commit(self, path, path_len, k_pages, v_pages, block_table, kmin=None, kmax=None, stream=None):
        """The accepted drafts join the context; ``seq_lens`` holds the new lengths after it."""
        B.sparse_attn_commit_drafts(self.p, path, path_len, k_pages, v_pages, block_table, self.new_lens, self.ws,
                                    self.seq_lens, kmin, kmax, stream)
        if stream is None:
            stream = torch.cuda.current_stream(self.device)
        elif not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=self.device)
        with torch.cuda.stream(stream):
            self.seq_lens.copy_(self.new_lens)

    def device_error(self, stream=None) -> int:
        with torch.cuda.device(self.device):         # whose current stream is the default
            return B.sparse_attn_get_device_error(self.ws, stream)


class LongContextDecoder(DraftDecoder):
    """A DraftDecoder for long contexts: queries and keys normed on their way into the cache and turned by
    positions of several axes, attention for groups of sequences that share a prefix, attention weights added
    up token by token, and eviction by them.  Owns what DraftDecoder owns, the weights and the kept tokens'
    numbers besides.

    ``num_groups`` groups at most share prefixes (0: ``decode_shared`` is not used); with ``keep_tokens``
    contexts are cut down to that many tokens (0: ``decode_weighed`` and ``evict`` are not used).  Every token
    that ``append`` or ``append_norm`` brings in has the weight zero until ``decode_weighed`` adds to it,
    whatever was at its index before: an evicted token, a rejected draft, another request.

    The workspace grows with the scores that ``decode_weighed`` keeps: 4 bytes for each of the B Q Hq query rows and
    each token of the capacity with up to 16 rows a KV head, or with fp32 queries or K/V."""

    def __init__(self, params: B.sparse_attn_params, seq_lens: torch.Tensor, num_groups: int = 0, keep_tokens: int = 0):
        super().__init__(params, seq_lens)
        p, dev = params, self.device
        if keep_tokens > max(p.capacity_tokens, p.n_tokens):
            raise ValueError(f"keep_tokens: {keep_tokens}, a sequence has pages for {max(p.capacity_tokens, p.n_tokens)}")
        self.num_groups, self.keep_tokens = num_groups, keep_tokens
        self.weights = self.kept_ids = None
        size = self.ws.numel()
        with torch.cuda.device(dev):
            if num_groups > 0:
                size = max(size, B.sparse_attn_shared_workspace_size(p, num_groups))
            if keep_tokens > 0:
                size = max(size, B.sparse_attn_weigh_workspace_size(p), B.sparse_attn_evict_workspace_size(p, keep_tokens))
                nb_cap = -(-max(p.capacity_tokens, p.n_tokens) // p.block_size)
                self.weights = torch.zeros(p.batch, p.num_kv_heads, nb_cap * p.block_size, device=dev)
                self.kept_ids = torch.full((p.batch, p.num_kv_heads, keep_tokens), -1, dtype=torch.int32, device=dev)
            if size > self.ws.numel():
                self.ws = torch.empty(size, dtype=torch.uint8, device=dev)
                B.sparse_attn_workspace_init(self.ws)

    def append(self, q_new, k_new, v_new, inv_freq, q_out, k_pages, v_pages, block_table, cu_rows=None,
               positions=None, pairing=B.ROTATE_HALVES, kmin=None, kmax=None, stream=None):
        B.sparse_attn_append_kv(self.p, q_new, k_new, v_new, inv_freq, q_out, k_pages, v_pages, block_table, self.ws,
                                cu_rows, self.seq_lens, positions, pairing, kmin, kmax, stream, self.weights)

    def append_norm(self, q_new, k_new, v_new, q_weight, k_weight, eps, inv_freq, q_out, k_pages, v_pages, block_table,
                    cu_rows=None, positions=None, axis_of=None, pairing=B.ROTATE_HALVES, kmin=None, kmax=None, stream=None):
        """``append`` with head norms (weights or None) and positions of several axes.  Once a sequence has
        been evicted from, a token's index is not its position any more: ``positions`` says it."""
        B.sparse_attn_append_kv_norm(self.p, q_new, k_new, v_new, q_weight, k_weight, eps, inv_freq, q_out, k_pages,
                                     v_pages, block_table, self.ws, cu_rows, self.seq_lens, positions, axis_of, pairing,
                                     kmin, kmax, stream, self.weights)

    def decode_shared(self, q, k_pages, v_pages, block_table, cu_seqs, prefix_lens, tree_mask=None, stream=None):
        """``decode`` for groups of sequences that hold the same first tokens; returns the output tensor."""
        if prefix_lens.numel() > self.num_groups:
            raise ValueError(f"prefix_lens: {prefix_lens.numel()} groups, room for {self.num_groups}")
        B.sparse_attn_shared_decode(self.p, q, k_pages, v_pages, block_table, cu_seqs, prefix_lens, self.out.view(q.shape),
                                    self.ws, self.seq_lens, tree_mask, stream)
        return self.out

    def decode_weighed(self, q, k_pages, v_pages, block_table, stream=None):
        """Attention of a chain of new tokens that adds to ``weights``; returns the output tensor.  Of a chain the
        first tokens are accepted: all by ``accept``, some by ``commit`` with a path 0, 1, 2, ..."""
        self._budget()
        B.sparse_attn_weigh_decode(self.p, q, k_pages, v_pages, block_table, self.weights, self.out.view(q.shape), self.ws,
                                   self.seq_lens, stream)
        return self.out

    def accept(self, stream=None):
        """The new tokens of every active sequence join its context.  A sequence whose context no attention has taken
        (out of range, or longer than ``p.n_tokens``) stays as it is."""
        with torch.cuda.stream(self._stream(stream)):
            taken = (self.seq_lens >= 0) & (self.seq_lens <= self.p.n_tokens)
            self.seq_lens.add_(taken.to(torch.int32), alpha=self.Q)

    def evict(self, sink_tokens, recent_tokens, k_pages, v_pages, block_table, new_table, keep_lens=None, kmin=None,
              kmax=None, stream=None):
        """Cut the contexts down to ``keep_tokens`` (or ``keep_lens``) tokens in the pages of ``new_table``
        [B, n], n >= ceil(keep_tokens / block_size), which must be free ones; ``kept_ids`` says which tokens they
        were.  ``seq_lens`` holds the new lengths after it.  Contexts of any length that has pages are cut, also
        those that an ``accept``, a ``commit`` or a prompt has carried past ``p.n_tokens``.

        The rows of ``block_table`` of the sequences that moved begin with their n new pages.  Of the entries
        behind them, those whose page another sequence's context reads (a shared prefix) become -1: an ``append``
        that gets there reports ``ERR_PAGE`` until the caller names a page.  The others stay, and with them their
        pages, which the sequence grows into next.  So the caller's again are the pages of a moved row's first n
        entries and of those that became -1, unless another row holds them.  What somebody outside of the
        batch or an inactive sequence reads is not looked for: where that may be, ``new_table`` as wide as
        ``block_table`` replaces the whole rows (-1: no page yet)."""
        self._budget()
        width, blocks = new_table.shape[1], -(-self.keep_tokens // self.p.block_size)
        if width > block_table.shape[1]:
            raise ValueError(f"new_table: {width} pages a sequence, block_table has {block_table.shape[1]}")
        p = B.sparse_attn_params.from_buffer_copy(self.p)
        p.n_tokens = max(p.capacity_tokens, p.n_tokens)              # needs no room for drafts behind a context
        kept_in = new_table
        if width > blocks:
            with torch.cuda.stream(self._stream(stream)):
                kept_in = new_table[:, :blocks].contiguous()
        B.sparse_attn_evict_tokens(p, self.keep_tokens, sink_tokens, recent_tokens, self.weights, k_pages, v_pages,
                                   block_table, kept_in, self.kept_ids, self.new_lens, self.ws, self.seq_lens, keep_lens,
                                   kmin, kmax, stream)
        B.sparse_attn_evict_adopt(p, self.keep_tokens, sink_tokens, recent_tokens, self.seq_lens, self.new_lens, block_table,
                                  new_table, self.ws, keep_lens, self.weights, stream)

    def _budget(self):
        if self.weights is None:
            raise ValueError("keep_tokens: 0, so there are no weights to add to or to evict by")

    def _stream(self, stream):
        if stream is None:
            return torch.cuda.current_stream(self.device)
        return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=self.device)
