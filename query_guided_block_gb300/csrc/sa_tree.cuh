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

constexpr int kTreeMaxCtas = 304;    // partial slots: two per CTA (the item a part begins in, the one it ends in)
constexpr int kTreeMaxRows = 128;    // query rows of an item at most

// Query rows of an item, in any kernel at most.
inline int tree_item_rows(int R) { return R <= 16 ? 16 : (R <= 64 ? 64 : kTreeMaxRows); }

// Words of shared memory that tree_part needs.
template <int NT>
constexpr int kTreeScan = NT / 32 + 3;

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
    int slack;                 // tiles that a part may grow by so that items begin with a part
    float scale_log2;
    float *part_m, *part_l, *part_o;   // [2 * CTA + which][item_rows] ([D])
    uint32_t *counters, *err;
};

// The list of a unit.
struct TreeUnit {
    int len;          // context tokens; -1: inactive
    int n_ctx;        // entries of the context (selection), or of everything without a selection
    int n_entries;
    int draft_blk;    // with a selection: the block of entry n_ctx
};

__device__ __forceinline__ TreeUnit tree_unit(const TreeArgs& a, int u)
{
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

__device__ __forceinline__ int tree_tiles(const TreeArgs& a, const TreeUnit& t)
{
    if (t.len < 0) return 0;
    const long long n = a.sel_ids == nullptr ? t.len + a.Q : (long long)t.n_entries << a.bs_shift;
    return int((n + a.tile - 1) / a.tile);
}

// Entry e of the list: the page's tile index (page * Hkv + KV head; -1 when there is none)
// and its first token.
__device__ __forceinline__ int2 tree_entry(const TreeArgs& a, int u, const TreeUnit& t, int e)
{
    const int b = u / a.Hkv, kvh = u - b * a.Hkv;
    int j = e;
    if (a.sel_ids != nullptr) {
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

// Bits d0 .. d0 + 7 of a draft mask (bit j of word j / 32), those in [0, limit).
__device__ __forceinline__ uint32_t mask_bits8(const uint32_t* words, int d0, int limit)
{
    if (d0 <= -8 || d0 >= limit) return 0u;
    uint32_t v;
    if (words == nullptr) {
        v = 0xffu;
        if (d0 < 0) v = (v << -d0) & 0xffu;
    } else if (d0 < 0) {
        v = words[0] << -d0;
    } else {
        const int w = d0 >> 5, s = d0 & 31;
        v = words[w] >> s;
        if (s > 24 && (w + 1) * 32 < limit) v |= words[w + 1] << (32 - s);
    }
    if (d0 + 8 > limit) v &= (1u << (limit - d0)) - 1u;
    return v & 0xffu;
}

// Which of the 8 list positions from p (a multiple of 8) a query with these mask words sees; e
// is their entry, `first` the entry's first token.
__device__ __forceinline__ uint32_t tree_tokens8(const TreeArgs& a, const TreeUnit& un, int p, int e, int first,
                                                 const uint32_t* words, int limit)
{
    if (first == kNoToken) return 0u;
    const int tok = first + (p & (a.bs - 1));
    const bool ctx = a.sel_ids == nullptr || e < un.n_ctx;
    uint32_t bits = 0u;
    if (ctx) bits = (1u << min(8, max(0, un.len - tok))) - 1u;
    if (a.sel_ids == nullptr || !ctx) bits |= mask_bits8(words, tok - un.len, limit);
    return bits;
}

// This CTA's part [lo, hi) of the line of tiles and the item that holds tile lo, found by all
// threads (NT of them, a multiple of 32).
struct TreePart {
    long long lo, hi;     // tiles of the line
    long long start;      // first tile of `item`
    int item;
    int per;              // tiles of a part
};

// Sums of v over the CTA's threads before this one (first) and over all of them.
template <int NT>
__device__ __forceinline__ void tree_scan(long long v, long long* s_scan, long long& before, long long& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long incl = v;
#pragma unroll
    for (int off = 1; off < kWarp; off <<= 1) {
        const long long t = __shfl_up_sync(kFullMask, incl, off);
        if (lane >= off) incl += t;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    before = incl - v;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    __syncthreads();
}

template <int NT>
__device__ TreePart tree_part(const TreeArgs& a, long long* s_scan /* [kTreeScan<NT>] shared */)
{
    const int units = a.B * a.Hkv, ctas = gridDim.x;
    // thread t owns units [t * ch, (t + 1) * ch)
    const int ch = (units + NT - 1) / NT;
    const int u0 = min(units, int(threadIdx.x) * ch), u1 = min(units, u0 + ch);
    const int t_first = u0 < u1 ? tree_tiles(a, tree_unit(a, u0)) : 0;
    auto tiles_of = [&](int u) { return u == u0 ? t_first : tree_tiles(a, tree_unit(a, u)); };
    long long mine = 0, before, total;
    for (int u = u0; u < u1; ++u) mine += tiles_of(u);
    mine *= a.row_groups;
    tree_scan<NT>(mine, s_scan, before, total);
    const long long share = (total + ctas - 1) / ctas;
    int per = int(share < a.min_per ? a.min_per : share);
    // items that begin with a part: at no cost, with half of the slack, then with all of it
    bool aligned = false;
    for (int more = 0; !aligned && more <= a.slack; more += max(1, a.slack / 2)) {
        const int p = per + more;
        long long parts = 0, parts_before, all_parts;
        for (int u = u0; u < u1; ++u) parts += (tiles_of(u) + p - 1) / p;
        parts *= a.row_groups;
        tree_scan<NT>(parts, s_scan, parts_before, all_parts);
        if (all_parts <= ctas) {
            aligned = true;
            per = p;
            mine = parts * p;
            before = parts_before * p;
            total = all_parts * p;
        }
    }
    TreePart r;
    r.per = per;
    r.lo = min(total, (long long)blockIdx.x * per);
    r.hi = min(total, r.lo + per);
    if (r.lo < r.hi && mine > 0 && r.lo >= before && r.lo < before + mine) {
        long long at = before;
        for (int u = u0; u < u1; ++u) {
            const int t = tiles_of(u);
            const int len = aligned ? (t + per - 1) / per * per : t;      // the item's stretch of the line
            const long long all = (long long)len * a.row_groups;
            if (r.lo < at + all) {
                const int rg = int((r.lo - at) / len);
                s_scan[NT / 32] = (long long)u * a.row_groups + rg;
                s_scan[NT / 32 + 1] = at + (long long)rg * len;
                s_scan[NT / 32 + 2] = aligned ? at + (long long)rg * len + t : r.hi;
                break;
            }
            at += all;
        }
    }
    __syncthreads();
    if (r.lo < r.hi) {
        r.item = int(s_scan[NT / 32]);
        r.start = s_scan[NT / 32 + 1];
        r.hi = min(r.hi, s_scan[NT / 32 + 2]);
    }
    __syncthreads();                                         // s_scan may be used for something else
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
__device__ __forceinline__ int tree_slot(int cta, int per, long long start)
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

// Called by the CTA's first NT threads once its (m, l, o) of a shared item is written: counts the
// arrival; the last one merges the parts c0 .. c1 and writes the output rows.  `s_w`: floats of
// shared memory free for use (at least as many as CTAs in the grid).
//   Two steps, so that no load waits for another one's result: a warp per row takes the parts'
// maxima and sums (lane = part) and leaves the parts' weights in shared memory, then a thread
// per four channels adds up its parts.
template <int NT>
__device__ void tree_arrive_and_merge(const TreeArgs& a, int item, long long start, int tiles, int per, int* s_last,
                                      float* s_w, int n_w)
{
    const int tid = threadIdx.x, lane = tid & 31;
    const int c0 = int(start / per), np = int((start + tiles - 1) / per) - c0 + 1;
    tree_sync<NT>();
    if (tid == 0) {
        const uint32_t before = atomic_add_acq_rel_u32(&a.counters[item], 1u);
        *s_last = before + 1u == uint32_t(np);
        if (*s_last) a.counters[item] = 0u;
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
                const float w = m == -INFINITY ? 0.f : fast_exp2(m - M);   // a part that saw nothing has no weight
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
                    if (w[x] != 0.f)
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

// The tensor-core kernel (sa_tree_tc.cu): bf16 queries and K/V.
cudaError_t launch_tree_tc(TreeArgs a, cudaStream_t s);

}  // namespace sa
