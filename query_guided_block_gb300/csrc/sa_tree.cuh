// Shared by the draft-tree attention kernels: the token list of a (sequence, KV head) unit,
// how its tiles are dealt to CTAs, and the merge of units that several CTAs share.
//
// A unit's keys are a list of entries of one block each: the context's blocks (or the
// selected ones), then the blocks that hold drafts.  Without a selection both are the blocks
// 0 .. of the sequence and a block may hold context and drafts.  Entry e covers list
// positions e * bs .. e * bs + bs - 1; tiles of T positions are cut from the list.
//
// Work split: the items (unit, row group) lie on one line of tiles that is cut into equal parts
// of `per` tiles, one per CTA, whatever the contexts' lengths are (they are only known on the
// device).  Items begin anywhere, or, when that costs few tiles, at the beginning of a part:
// then no CTA works on two items, and an item that fits one part has nothing to merge.  An
// item that several parts share leaves (m, l, o) per part in the workspace, and the CTA that
// arrives last adds them up in the parts' order, so the result does not depend on timing.
#pragma once

#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {

constexpr int kTreeMaxRows = 128;    // query rows of an item at most

// bf16 calls with more than 16 rows and at most so many tiles (of 64 tokens x 16 rows) an SM run on the warp-level
// kernel too, 16 rows to an item: a tensor-memory item takes longer to begin and end.  24 rows over 777 tokens
// (1.4 tiles an SM) 13.2 us against 16.8, 64 rows over 777 (2.7) 14.8 against 18.3, over 4 x 300 (4.2)
// 15.8 against 25.0 (18.6 where the parts are joined by a launch), 32 rows over 4 x 777 (5.5) 21.2
// against 18.2, 128 rows over 777 (5.5) 21.3 against 19.6, 64 rows over 16 x 100 (6.7) 21.9 against 15.6.
constexpr int kTreeSmallWork = 4;

// Query rows of an item, in any kernel at most.
inline int tree_item_rows(int R) { return R <= 16 ? 16 : (R <= 64 ? 64 : kTreeMaxRows); }

// Words of shared memory that tree_part needs.
template <int NT>
constexpr int kTreeScan = 6 * (NT / 32) + 3;

struct TreeArgs {
    const void* q;
    int q_bf16;
    const void *k_pages, *v_pages;
    const int32_t *block_table, *seq_lens, *sel_ids, *sel_count;
    const uint32_t* mask;      // [B, Q, mask_words], null: a chain
    float* out;
    int B, Hq, Hkv, G, Q, R, D, N, bs, bs_shift, nb, nb_cap, num_pages, sel_stride, mask_words;
    int row_groups;            // items per unit
    int item_rows;             // query rows of an item at most
    int tile;                  // list positions per tile
    int min_per;               // tiles of a part at least
    int half_slack;            // a part may grow by twice as many tiles so that items begin with a part
    float scale_log2;
    float merge_scale;         // base-2 logits in a step of the kernel's maxima (part_m)
    int combine;               // shared items are added up by a launch of their own
    float *part_m, *part_l, *part_o;   // [2 * CTA + which][item_rows] ([D])
    int2* item_parts;          // combine: an item's first part and how many it has
    uint32_t* counters;        // [CTA] arrivals of the item that goes on behind this CTA's part; zero between calls
    uint32_t* err;

    // The kernels' EXT form (sa_shared.cu, sa_weigh.cu): a launch of its own joins the shares, so (m, l, o) are
    // left as they are, those of items in one part in row_m, row_l and `out`.  Only a kTreeAll item in one
    // part is done with.
    int pass;                  // kTreeAll, kTreePrefix, kTreeOwn or kTreeBoth
    int tensor;                // the tensor-core kernel's shares: relative to the rounded product of maximum and scale
    int seqs, groups;          // sequences of the batch, groups that share prefixes (B: units / Hkv)
    const int32_t *cu_seqs, *prefix_lens;
    int32_t *seq_prefix, *seq_group;     // [seqs]: shared tokens (-1: inactive) and group, by the prefix pass
    float *row_m, *row_l;      // [seqs * Q * Hq]: unscaled maximum and sum of rows in one part
    float2* stats;             // [seqs * Q * Hq]: kTreeAll: maximum and 1 / total of rows that are done
    float* scores;             // [unit][R][score_stride] unscaled scores, null: not kept
    long long score_stride;
    // kTreeBoth: where the own tokens' items go (the prefixes' to out, row_m, row_l, item_parts)
    float *own_out, *own_row_m, *own_row_l;
    int2* own_item_parts;
};

// What the units of an EXT launch are.
enum {
    kTreeAll = 0,              // (sequence, KV head): its whole context and its drafts
    kTreePrefix = 1,           // (group, KV head): the group's shared tokens, all its members' rows
    kTreeOwn = 2,              // (sequence, KV head): the context behind the shared tokens, and the drafts
    kTreeBoth = 3              // the units of both, groups first
};

// The list of a unit.
struct TreeUnit {
    int len;          // context tokens; -1: inactive
    int n_ctx;        // entries of the context (selection), or of everything without a selection
    int n_entries;
    int draft_blk;    // with a selection: the block of entry n_ctx
    // EXT only
    int b0;           // sequence of the unit's first query row
    int rows;         // query rows
    int table_row;    // sequence whose page table is read
    int from;         // tokens below it are not the unit's
    int first_blk;    // block of entry 0
    int drafts;       // drafts behind the context
    bool prefix;      // a group's shared tokens
};

// Shared tokens (-1: inactive) and group of sequence b.
__device__ __forceinline__ int2 tree_sequence(const TreeArgs& a, int b)
{
    int lo = 0, hi = a.groups;                               // the last group that begins at b or before
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_seqs[mid] <= b) lo = mid;
        else hi = mid;
    }
    const int b0 = a.cu_seqs[lo], b1 = a.cu_seqs[lo + 1];
    const int len = a.seq_lens != nullptr ? a.seq_lens[b] : a.N;
    const int n = b >= b0 && b < b1 ? a.prefix_lens[lo] : 0;
    bool bad = len < -1 || len > a.N;
    if (b >= b0 && b < b1) bad = bad || b0 < 0 || b1 > a.seqs || n < 0 || (len >= 0 && n > len);
    if (bad) raise_error(a.err, SPARSE_ATTN_ERR_LENGTH);
    return make_int2(bad || len < 0 ? -1 : n, lo);
}

// The unit of a launch that EXT gives other units, from the arrays that say so.
__device__ __forceinline__ TreeUnit tree_unit_ext(const TreeArgs& a, int u)
{
    TreeUnit t;
    int x = u / a.Hkv;
    t.len = -1;
    t.n_ctx = t.n_entries = t.draft_blk = 0;
    t.prefix = a.pass == kTreePrefix || (a.pass == kTreeBoth && x < a.groups);
    if (a.pass == kTreeBoth && !t.prefix) x -= a.groups;
    t.b0 = t.table_row = x;
    t.rows = a.R;
    t.from = t.first_blk = 0;
    t.drafts = a.Q;
    if (t.prefix) {
        const int b0 = a.cu_seqs[x], b1 = a.cu_seqs[x + 1], n = a.prefix_lens[x];
        if (b0 < 0 || b1 < b0 || b1 > a.seqs || n < 0 || n > a.N) {
            raise_error(a.err, SPARSE_ATTN_ERR_LENGTH);
            return t;
        }
        if (n == 0) return t;
        // the pages are those of the first member that holds the prefix
        int b = b0;
        if (a.seq_lens != nullptr)
            while (b < b1 && (a.seq_lens[b] < n || a.seq_lens[b] > a.N)) ++b;
        if (b == b1) return t;
        t.b0 = b0;
        t.table_row = b;
        t.rows = (b1 - b0) * a.R;
        t.drafts = 0;
        t.len = n;
        t.n_ctx = t.n_entries = (n + a.bs - 1) >> a.bs_shift;
        return t;
    }
    const int len = a.seq_lens != nullptr ? a.seq_lens[x] : a.N;
    if (a.pass != kTreeAll) {
        const int p = a.pass == kTreeOwn ? a.seq_prefix[x] : tree_sequence(a, x).x;
        if (p < 0) return t;                                 // reported where it was found
        t.from = p;
        t.first_blk = p >> a.bs_shift;
    } else if (len < 0 || len > a.N) {
        if (len != -1) raise_error(a.err, SPARSE_ATTN_ERR_LENGTH);
        return t;
    }
    t.len = len;
    t.n_ctx = t.n_entries = ((len + a.Q - 1) >> a.bs_shift) + 1 - t.first_blk;
    return t;
}

template <bool EXT = false>
__device__ __forceinline__ TreeUnit tree_unit(const TreeArgs& a, int u)
{
    if constexpr (EXT) return tree_unit_ext(a, u);
    TreeUnit t;
    const int b = u / a.Hkv;
    t.len = a.seq_lens != nullptr ? a.seq_lens[b] : a.N;
    t.n_ctx = t.n_entries = t.draft_blk = 0;
    if (t.len < 0 || t.len > a.N) {
        if (t.len != -1) raise_error(a.err, SPARSE_ATTN_ERR_LENGTH);
        t.len = -1;
        return t;
    }
    const int last = (t.len + a.Q - 1) >> a.bs_shift;       // the last block with a draft
    if (a.sel_ids == nullptr) {
        t.n_ctx = t.n_entries = last + 1;
        return t;
    }
    int count = a.sel_count[u];
    if (count < 0 || count > a.sel_stride) {
        raise_error(a.err, SPARSE_ATTN_ERR_SEL_COUNT);
        count = count < 0 ? 0 : a.sel_stride;
    }
    t.n_ctx = count;
    t.draft_blk = t.len >> a.bs_shift;
    t.n_entries = count + last - t.draft_blk + 1;
    return t;
}

template <bool EXT = false>
__device__ __forceinline__ int tree_tiles(const TreeArgs& a, const TreeUnit& t)
{
    if (t.len < 0) return 0;
    if constexpr (EXT) return (t.len + t.drafts - (t.first_blk << a.bs_shift) + a.tile - 1) / a.tile;
    const long long n = a.sel_ids == nullptr ? t.len + a.Q : (long long)t.n_entries << a.bs_shift;
    return int((n + a.tile - 1) / a.tile);
}

// Row groups of a unit.
template <bool EXT>
__device__ __forceinline__ int tree_row_groups(const TreeArgs& a, const TreeUnit& t)
{
    return EXT ? (t.rows + a.item_rows - 1) / a.item_rows : a.row_groups;
}

// The item behind `item`, of the unit t.
template <bool EXT>
__device__ __forceinline__ int tree_next_item(const TreeArgs& a, const TreeUnit& t, int item)
{
    if constexpr (EXT) {
        const int u = item / a.row_groups;
        if (t.len < 0 || item + 1 - u * a.row_groups >= tree_row_groups<true>(a, t)) return (u + 1) * a.row_groups;
    }
    return item + 1;
}

// Entry e of the list: the page's tile index (page * Hkv + KV head; -1 when there is none)
// and its first token.
template <bool EXT = false>
__device__ __forceinline__ int2 tree_entry(const TreeArgs& a, int u, const TreeUnit& t, int e)
{
    const int x = u / a.Hkv, kvh = u - x * a.Hkv, b = EXT ? t.table_row : x;
    int j = EXT ? t.first_blk + e : e;
    if (!EXT && a.sel_ids != nullptr) {
        if (e < t.n_ctx) {
            j = a.sel_ids[(long long)u * a.sel_stride + e];
            if (j < 0 || j >= a.nb) {
                raise_error(a.err, SPARSE_ATTN_ERR_SEL_ID);
                return make_int2(-1, 0);
            }
            if ((j << a.bs_shift) >= t.len) return make_int2(-1, 0);   // behind this sequence's context
        } else {
            j = t.draft_blk + e - t.n_ctx;
        }
    }
    const int page = a.block_table[(long long)b * a.nb_cap + j];
    if (page < 0 || page >= a.num_pages) {
        raise_error(a.err, SPARSE_ATTN_ERR_PAGE);
        return make_int2(-1, 0);
    }
    return make_int2(page * a.Hkv + kvh, j << a.bs_shift);
}

constexpr int kNoToken = INT32_MIN;  // first token of an entry without a page

// A row's view of the drafts: their bits, the first 64 at hand.
struct DraftView {
    const uint32_t* words;    // bit j of word j / 32; null: all of them
    uint64_t first;           // bits 0 .. 63
    int limit;                // drafts from here on are not seen
};

__device__ __forceinline__ DraftView draft_view(const uint32_t* words, int n_words, int limit)
{
    DraftView v{words, ~0ull, limit};
    if (words != nullptr) {
        v.first = words[0];
        if (n_words > 1) v.first |= uint64_t(words[1]) << 32;
    }
    return v;
}

// Bits d0 .. d0 + 7 of the view.
__device__ __forceinline__ uint32_t draft_bits8(const DraftView& w, int d0)
{
    if (d0 <= -8 || d0 >= w.limit) return 0u;
    uint32_t v;
    if (d0 < 0) {
        v = uint32_t(w.first) << -d0;
    } else if (d0 <= 56 || w.words == nullptr) {
        v = uint32_t(w.first >> min(d0, 32));                // no words: every bit is set
        if (d0 > 32 && w.words != nullptr) v = uint32_t(w.first >> d0);
    } else {
        const int x = d0 >> 5, s = d0 & 31;
        v = w.words[x] >> s;
        if (s > 24 && (x + 1) * 32 < w.limit) v |= w.words[x + 1] << (32 - s);
    }
    if (d0 + 8 > w.limit) v &= (1u << (w.limit - d0)) - 1u;
    return v & 0xffu;
}

// Which of the 8 list positions from p (a multiple of 8) a query with this view sees; e is
// their entry, `first` the entry's first token.
template <bool EXT = false>
__device__ __forceinline__ uint32_t tree_tokens8(const TreeArgs& a, const TreeUnit& un, int p, int e, int first,
                                                 const DraftView& view)
{
    if (first == kNoToken) return 0u;
    const int tok = first + (p & (a.bs - 1));
    if constexpr (EXT) {
        uint32_t bits = (1u << min(8, max(0, un.len - tok))) - 1u;
        bits &= ~((1u << min(8, max(0, un.from - tok))) - 1u);
        return bits | draft_bits8(view, tok - un.len);
    }
    const bool ctx = a.sel_ids == nullptr || e < un.n_ctx;
    uint32_t bits = 0u;
    if (ctx) bits = (1u << min(8, max(0, un.len - tok))) - 1u;
    if (a.sel_ids == nullptr || !ctx) bits |= draft_bits8(view, tok - un.len);
    return bits;
}

// This CTA's part [lo, hi) of the line of tiles and the item that holds tile lo.  The line is
// shorter than 2^31 tiles.
struct TreePart {
    int lo, hi;       // tiles of the line
    int start;        // first tile of `item`
    int item;
    int per;          // tiles of a part
    bool whole;       // the items that begin in the part belong to it to their ends
};

// Found by all threads (NT of them): as many warps as the units need count tiles, the others
// only keep step.  `s`: kTreeScan<NT> words of shared memory.
template <int NT, bool EXT = false>
__device__ TreePart tree_part(const TreeArgs& a, int* s)
{
    constexpr int W = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // EXT: the KV heads of a sequence or group are counted together (64 sequences x 8
    // heads behind 32K tokens 156 us for 160)
    const int units = EXT ? a.B : a.B * a.Hkv, ctas = gridDim.x;
    const int warps = min(W, (units + 31) / 32);
    const int ch = (units + warps * 32 - 1) / (warps * 32);    // units per counting thread, consecutive
    const int u0 = warp < warps ? min(units, tid * ch) : units, u1 = min(units, u0 + ch);
    struct Count {
        int tiles, groups;            // of an item, row groups (EXT: of all KV heads)
    };
    auto count = [&](int u) {
        const TreeUnit un = tree_unit<EXT>(a, EXT ? u * a.Hkv : u);
        return Count{tree_tiles<EXT>(a, un), tree_row_groups<EXT>(a, un) * (EXT ? a.Hkv : 1)};
    };
    const Count t_first = u0 < u1 ? count(u0) : Count{0, a.row_groups};
    auto tiles_of = [&](int u) { return u == u0 ? t_first : count(u); };
    int* s_sum = s;                   // [W] tiles
    int* s_parts = s + W;             // [3][W] parts at three lengths
    int* s_line = s + 4 * W;          // [W] stretches of the line
    int* s_longest = s + 5 * W;       // [W] tiles of the longest item
    int* s_found = s + 6 * W;         // item, start, end

    int tiles = 0;
    for (int u = u0; u < u1; ++u) {
        const Count n = tiles_of(u);
        tiles += EXT ? n.tiles * n.groups : n.tiles;
    }
    if (!EXT) tiles *= a.row_groups;
    if (warp < warps) {
        const int sum = __reduce_add_sync(kFullMask, tiles);
        if (lane == 0) s_sum[warp] = sum;
    }
    __syncthreads();
    int total = 0;
    for (int w = 0; w < warps; ++w) total += s_sum[w];
    int per = max(a.min_per, (total + ctas - 1) / ctas);
    // Items may begin with a part if the parts then suffice: at no cost, with half of the slack
    // added to a part, or with all of it.  Where items are too many for that and none is longer
    // than the slack, the parts take whole items, those that begin in them.
    int parts[3] = {0, 0, 0}, longest = 0;
    for (int u = u0; u < u1; ++u) {
        const Count n = tiles_of(u);
        const int t = n.tiles;
        longest = max(longest, t);
#pragma unroll
        for (int x = 0; x < 3; ++x)
            parts[x] += (t + per + x * a.half_slack - 1) / (per + x * a.half_slack) * (EXT ? n.groups : 1);
    }
    if (warp < warps) {
#pragma unroll
        for (int x = 0; x < 3; ++x) {
            if (!EXT) parts[x] *= a.row_groups;
            const int sum = __reduce_add_sync(kFullMask, parts[x]);
            if (lane == 0) s_parts[x * W + warp] = sum;
        }
        longest = __reduce_max_sync(kFullMask, longest);
        if (lane == 0) s_longest[warp] = longest;
    }
    __syncthreads();
    int all[3] = {0, 0, 0};
    for (int w = 0; w < warps; ++w) {
        longest = max(longest, s_longest[w]);
#pragma unroll
        for (int x = 0; x < 3; ++x) all[x] += s_parts[x * W + w];
    }
    int mine = tiles;
    bool aligned = false;
#pragma unroll
    for (int x = 2; x >= 0; --x) {
        if (all[x] > ctas) continue;
        aligned = true;
        mine = parts[x];
        total = all[x];
    }
    if (aligned) {
        per += (all[0] <= ctas ? 0 : (all[1] <= ctas ? 1 : 2)) * a.half_slack;
        mine *= per;
        total *= per;
    }
    int incl = mine;
    if (warp < warps) {
        incl = warp_inclusive_scan(mine, lane);
        if (lane == 31) s_line[warp] = incl;
    }
    __syncthreads();
    TreePart r;
    r.per = per;
    r.whole = !aligned && longest <= 2 * a.half_slack;
    r.lo = int(min((long long)total, (long long)blockIdx.x * per));
    r.hi = int(min((long long)total, (long long)r.lo + per));
    if (r.lo < r.hi && mine > 0) {
        int at = incl - mine;
        for (int w = 0; w < warp; ++w) at += s_line[w];
        if (r.lo >= at && r.lo < at + mine) {
            for (int u = u0; u < u1; ++u) {
                const Count n = tiles_of(u);
                const int t = n.tiles, groups = EXT ? n.groups : a.row_groups;
                const int len = aligned ? (t + per - 1) / per * per : t;      // the item's stretch of the line
                if (r.lo < at + len * groups) {
                    const int rg = (r.lo - at) / len;
                    const int next = r.whole && at + rg * len < r.lo;         // it began in an earlier part
                    s_found[0] = u * a.row_groups + rg + next;
                    if (EXT) {
                        const int per_head = groups / a.Hkv;
                        s_found[0] = (u * a.Hkv + (rg + next) / per_head) * a.row_groups + (rg + next) % per_head;
                    }
                    s_found[1] = at + (rg + next) * len;
                    s_found[2] = aligned ? at + rg * len + t : r.hi;
                    break;
                }
                at += len * groups;
            }
        }
    }
    __syncthreads();
    if (r.lo < r.hi) {
        r.item = s_found[0];
        r.start = s_found[1];
        r.hi = min(r.hi, s_found[2]);
        if (r.whole) r.lo = r.start;
    }
    if (r.whole) r.per = max(total, 1);                      // every item is one part
    __syncthreads();                                         // s may be used for something else
    return r;
}

// The output row of an item's query row r (query r / G, head r % G of the KV head's group).
__device__ __forceinline__ long long tree_out_row(const TreeArgs& a, int b, int kvh, int r)
{
    const int t = r / a.G, g = r - t * a.G;
    return ((long long)b * a.Q + t) * a.Hq + kvh * a.G + g;
}

// Partial slot of CTA `cta` for an item that starts at tile `start`: 0 when the item began in
// an earlier part, 1 when it begins in this one (and goes on in the next).
__device__ __forceinline__ int tree_slot(int cta, int per, int start)
{
    return 2 * cta + (start < (long long)cta * per ? 0 : 1);
}

// Barrier of the first NT threads of the CTA (barrier 2 is theirs).
template <int NT>
__device__ __forceinline__ void tree_sync()
{
    __syncwarp();
    asm volatile("bar.sync 2, %0;" ::"n"(NT) : "memory");
}

// What the combining launch has to know of an item, by the CTA that begins it (one thread).
__device__ __forceinline__ void tree_note_parts(const TreeArgs& a, int item, int start, int tiles, int per)
{
    const int c0 = start / per;
    a.item_parts[item] = make_int2(c0, (start + tiles - 1) / per - c0 + 1);
}

// An EXT row of an item in one part.
__device__ __forceinline__ void tree_note_row(const TreeArgs& a, const TreeUnit& un, long long row, bool done, float m,
                                              float l, float inv)
{
    if (done) {
        a.stats[row] = make_float2(m, inv);
    } else {
        const bool own = a.pass == kTreeBoth && !un.prefix;
        (own ? a.own_row_m : a.row_m)[row] = m;
        (own ? a.own_row_l : a.row_l)[row] = l;
    }
}

// The first part of an item and how many it has.
__device__ __forceinline__ int2 tree_parts(int start, int tiles, int per)
{
    const int c0 = start / per;
    return make_int2(c0, (start + tiles - 1) / per - c0 + 1);
}

// Where the parts of row group rg of an EXT unit are noted: row groups of one KV head in the order of
// their rows, a group of sequences beginning with one of its own.
__host__ __device__ __forceinline__ long long tree_notes_per_head(const TreeArgs& a, bool prefix, int item_rows)
{
    return prefix ? (long long)a.seqs * a.R / item_rows + a.groups + 1
                  : (long long)a.seqs * ((a.R + item_rows - 1) / item_rows);
}
__device__ __forceinline__ int2& tree_note(const TreeArgs& a, int u, const TreeUnit& un, int rg)
{
    const int x = u / a.Hkv, kvh = u - x * a.Hkv;
    const long long first = un.prefix ? (long long)un.b0 * a.R / a.item_rows + x
                                      : (long long)un.b0 * ((a.R + a.item_rows - 1) / a.item_rows);
    int2* notes = a.pass == kTreeBoth && !un.prefix ? a.own_item_parts : a.item_parts;
    return notes[kvh * tree_notes_per_head(a, un.prefix, a.item_rows) + first + rg];
}

// The weight of a share with maximum m and total l among shares whose largest maximum is M.  One that saw
// nothing has none; one whose scores are all NaN has a NaN total and no maximum either, and is kept.
__device__ __forceinline__ float tree_share(float m, float M, float l, float scale)
{
    return m == -INFINITY && l == 0.f ? 0.f : fast_exp2((m - M) * scale);
}

// The prefix pass: which group and how many shared tokens every sequence has, for the launches behind it;
// -1 where it is inactive.  By the last CTAs, which have the least to do when work is short.
__device__ __forceinline__ void tree_note_sequences(const TreeArgs& a, int threads)
{
    if (a.pass != kTreePrefix && a.pass != kTreeBoth) return;
    for (int b = (gridDim.x - 1 - blockIdx.x) * threads + threadIdx.x; b < a.seqs; b += gridDim.x * threads) {
        const int2 of = tree_sequence(a, b);
        a.seq_prefix[b] = of.x;
        a.seq_group[b] = of.y;
    }
}

// The weight of a share with maximum m and total l beside one whose maximum is M, unscaled both, and to which
// M itself is the reference.  Shares of the warp-level kernel are relative to m * scale exactly, those of
// the tensor-core one to the rounded product, which the difference takes into account; past 2^29 (in base-2
// logits) they are relative to m itself again, and so are the weights here.
__device__ __forceinline__ float share_weight(bool tensor, float m, float M, float l, float scale)
{
    if (m == -INFINITY && l == 0.f) return 0.f;
    const float rounded = __fmul_rn(m, scale);
    if (tensor && fabsf(rounded) < 536870912.f) return fast_exp2(-fmaf(M, scale, -rounded));
    return fast_exp2((m - M) * scale);
}

// Called by the CTA's first NT threads once its (m, l, o) of a shared item is written: counts the
// arrival at the counter of the item's first part (one item at most begins in a part and goes on
// behind it); the last one merges the parts c0 .. c1 and writes the output rows.  `s_w`: floats of
// shared memory free for use (at least as many as CTAs in the grid).
//   Two steps, so that no load waits for another one's result: a warp per row takes the parts'
// maxima and sums (lane = part) and leaves the parts' weights in shared memory, then a thread
// per four channels adds up its parts.
template <int NT>
__device__ void tree_arrive_and_merge(const TreeArgs& a, int item, int start, int tiles, int per, int* s_last,
                                      float* s_w, int n_w)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const int c0 = start / per, np = (start + tiles - 1) / per - c0 + 1;
    tree_sync<NT>();
    if (tid == 0) {
        const uint32_t before = atomic_add_acq_rel_u32(&a.counters[c0], 1u);
        *s_last = before + 1u == uint32_t(np);
        if (*s_last) a.counters[c0] = 0u;
    }
    tree_sync<NT>();
    const bool last = *s_last != 0;
    if (!last) return;                                      // the next item's barriers keep s_last
    const int u = item / a.row_groups, row0 = (item - u * a.row_groups) * a.item_rows;
    const int b = u / a.Hkv, kvh = u - b * a.Hkv;
    const int rows = min(a.item_rows, a.R - row0);
    const int vec = a.D / 4, batch = min(rows, n_w / (2 * np));
    float* s_l = s_w + batch * np;
    for (int r0 = 0; r0 < rows; r0 += batch) {
        const int n = min(batch, rows - r0);
        for (int i = tid; i < n * np; i += NT) {
            const int c = i / n, r = i - c * n;
            const long long at = (long long)tree_slot(c0 + c, per, start) * a.item_rows + r0 + r;
            s_w[r * np + c] = __ldcg(a.part_m + at);
            s_l[r * np + c] = __ldcg(a.part_l + at);
        }
        tree_sync<NT>();
        for (int r = tid >> 5; r < n; r += NT / 32) {
            float M = -INFINITY;
            for (int c = lane; c < np; c += 32) M = fmaxf(M, s_w[r * np + c]);
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, x));
            float den = 0.f;
            for (int c = lane; c < np; c += 32) {
                const float m = s_w[r * np + c];
                const float w = tree_share(m, M, s_l[r * np + c], a.merge_scale);
                s_w[r * np + c] = w;
                den = fmaf(w, s_l[r * np + c], den);
            }
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) den += __shfl_xor_sync(kFullMask, den, x);
            __syncwarp();
            const float inv = den == 0.f ? 0.f : 1.f / den;
            for (int c = lane; c < np; c += 32) s_w[r * np + c] *= inv;
        }
        tree_sync<NT>();
        for (int i = tid; i < n * vec; i += NT) {
            const int r = i / vec, d = (i - r * vec) * 4;
            float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < np; c += 8) {               // eight loads in flight
                float4 o[8];
                float w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    w[x] = c + x < np ? s_w[r * np + c + x] : 0.f;
                    o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (c + x < np)                         // without a weight too: it may hold infinities
                        o[x] = __ldcg(reinterpret_cast<const float4*>(
                            a.part_o + ((long long)tree_slot(c0 + c + x, per, start) * a.item_rows + r0 + r) * a.D + d));
                }
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    num.x = fmaf(o[x].x, w[x], num.x);
                    num.y = fmaf(o[x].y, w[x], num.y);
                    num.z = fmaf(o[x].z, w[x], num.z);
                    num.w = fmaf(o[x].w, w[x], num.w);
                }
            }
            *reinterpret_cast<float4*>(a.out + tree_out_row(a, b, kvh, row0 + r0 + r) * a.D + d) = num;
        }
        tree_sync<NT>();
    }
}

// Items whose parts hold this much are added up by a launch of their own (a warp per row, over
// the whole GPU) instead of by the CTA that arrives last, whose SM reads about 100 KB a
// microsecond; the second launch costs the host 2.5 us.  16 rows over 777 tokens (48 KB) 12.0 us
// against 16.8, over 300 (24 KB) 12.3 against 16.0, 64 rows over 8 x 777 (64 KB) 23.8 against 30.2.
// With few rows the launch has few warps, each with all the parts: 4 rows over 8K tokens (36 KB)
// 19.8 us against 18.2, 8 rows over 777 (24 KB) 11.4 against 13.4.
constexpr long long kTreeCombineBytes = 16 * 1024;
constexpr int kTreeCombineRows = 8;
void tree_choose_combine(TreeArgs& a, int ctas);
cudaError_t launch_tree_combine(const TreeArgs& a, cudaStream_t s);

// The tensor-core kernel (sa_tree_tc.cu): bf16 queries and K/V.
cudaError_t launch_tree_tc(TreeArgs a, cudaStream_t s);

// The EXT form (sa_tree_ext64.cu, sa_tree_ext128.cu, sa_tree_tc_ext.cu) for units of about `rows` query rows.
cudaError_t launch_tree_ext64(TreeArgs& a, bool kv_bf16, int rows, cudaStream_t s);
cudaError_t launch_tree_ext128(TreeArgs& a, bool kv_bf16, int rows, cudaStream_t s);
cudaError_t launch_tree_tc_ext(TreeArgs& a, int rows, cudaStream_t s);
// Whether the tensor-core kernel takes a launch with about so many rows a unit and `tiles` tiles of 64 tokens
// x 16 rows: kTreeSmallWork's rule, for 152 SMs.  Up to 32 rows it is for the long lists of prefixes:
// sequences' own tokens are fewer, and where scores are kept the warp-level kernel leaves them (20 rows over
// 4 x 32K tokens weighed in 155 us against 166, over 64 x 1000 in 102 against 156).
inline bool tree_ext_tensor(int pass, bool bf16, int rows, long long tiles)
{
    return bf16 && rows > (pass == kTreePrefix ? 16 : 32) && tiles > kTreeSmallWork * 152;
}
// Query rows of its items otherwise.
inline int tree_ext_item_rows(bool bf16, int rows) { return rows <= 16 ? 16 : (bf16 && rows <= 32 ? 32 : 64); }
inline cudaError_t launch_tree_ext(TreeArgs& a, bool kv_bf16, int rows, bool tensor, cudaStream_t s)
{
    if (tensor) return launch_tree_tc_ext(a, rows, s);
    return a.D == 128 ? launch_tree_ext128(a, kv_bf16, rows, s) : launch_tree_ext64(a, kv_bf16, rows, s);
}

// The sums of weights with the scores computed again (sa_weigh_tc.cu).
cudaError_t launch_weigh_tc(TreeArgs a, const float2* stats, float* weights, long long w_stride, cudaStream_t s);

// Joins the shares that EXT launches left and writes the output rows; `prefix` (null: none) has the group's
// tokens.  `stats`: [seqs * Q * Hq] (maximum, 1 / total), null: not wanted.
cudaError_t launch_tree_join(const TreeArgs& own, const TreeArgs* prefix, float2* stats, cudaStream_t s);

// Workspace of one EXT launch, which a call carves out of its own: notes, shares of items in several parts,
// and the maxima and sums of those in one.
struct TreeExtLayout {
    size_t item_parts, part_m, part_l, part_o, row_m, row_l, end;
};
TreeExtLayout tree_ext_layout(const Geometry& g, size_t at, int groups);
// The fields that every EXT launch of this problem has in common.
TreeArgs tree_ext_args(const Geometry& g, const TreeCall& c, char* ws, const TreeExtLayout& L);

}  // namespace sa
