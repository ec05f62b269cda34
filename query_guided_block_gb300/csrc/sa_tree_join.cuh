// The join of the shares (m, l, o) that EXT launches of the draft-tree kernels leave (sa_shared.cu,
// sa_weigh.cu).
#pragma once

#include "sa_tree.cuh"

namespace sa {

constexpr int kJoinWarps = 4;
constexpr int kJoinThreads = 32 * kJoinWarps;

// One row's shares of a launch: rows of (m, l, o), the first one's and how many.
struct Shares {
    const float *m, *l, *o;
    int step, n;                   // step: rows of a slot
};

__device__ __forceinline__ Shares shares_of(const TreeArgs& a, int2 parts, int rr, long long out_row)
{
    if (parts.y <= 1) return Shares{a.row_m + out_row, a.row_l + out_row, a.out + out_row * a.D, 0, 1};
    // the first part of an item is the second slot of its CTA, the others are first slots
    const long long at = (2LL * parts.x + 1) * a.item_rows + rr;
    return Shares{a.part_m + at, a.part_l + at, a.part_o + at * a.D, a.item_rows, parts.y};
}
__device__ __forceinline__ long long share_row(int step, int c) { return c == 0 ? 0 : (2LL * c - 1) * step; }

// WPR warps to an output row: each has all the shares' maxima and totals (lane = share) and adds up every
// WPR-th share, eight loads on their way at once; their sums go through shared memory.  A small call waits
// for the chain of dependent loads (the sequence's group, notes, maxima, shares) and takes four warps a row,
// which leaves one round of shares; with many rows one warp has a row to itself (2048 rows of about 12
// shares 7.0 us, four warps a row 10.6).  Where the attention has finished the rows in one part, a warp looks
// eight rows' notes up and joins those that are left: from many rows on, since it joins them one by one (131072 rows,
// none left: 6.5 us, 97 with a warp a row; 16384 rows in split items 15 with a warp a row, 36 with one for 32).
template <int D, int WPR>
__device__ __forceinline__ void join_row(const TreeArgs& own, const TreeArgs& pre, int with_prefix, float2* stats, int row)
{
    __shared__ float4 s_num[WPR > 1 ? kJoinWarps : 1][D / 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % WPR;
    const int h = row % own.Hq, bt = row / own.Hq, b = bt / own.Q, t = bt - b * own.Q;
    const int kvh = h / own.G, r = t * own.G + h - kvh * own.G;
    const int rg = r / own.item_rows;
    const int2 own_parts = own.item_parts[kvh * tree_notes_per_head(own, false, own.item_rows) + (long long)b * own.row_groups + rg];
    float4* out = reinterpret_cast<float4*>(own.out + (long long)row * D) + lane;
    int from = 0, group = 0;
    bool active;
    if (with_prefix) {
        from = own.seq_prefix[b];
        group = own.seq_group[b];
        active = from >= 0;
    } else {
        const int len = own.seq_lens != nullptr ? own.seq_lens[b] : own.N;
        active = len >= 0 && len <= own.N;
    }
    // no output, or done already; the same for all warps of a row
    if (!active || (own.pass == kTreeAll && own_parts.y <= 1)) return;
    const Shares x0 = shares_of(own, own_parts, r - rg * own.item_rows, row);
    Shares x1 = x0;
    x1.n = 0;
    if (from > 0) {
        const int b0 = pre.cu_seqs[group];
        const int rp = (b - b0) * pre.R + r, rgp = rp / pre.item_rows;
        const long long note = kvh * tree_notes_per_head(pre, true, pre.item_rows) + (long long)b0 * pre.R / pre.item_rows + group + rgp;
        x1 = shares_of(pre, pre.item_parts[note], rp - rgp * pre.item_rows, row);
    }
    const float scale = own.scale_log2;
    const int n = x0.n + x1.n;
    auto share_m = [&](int c) {
        return __ldcg(c < x0.n ? x0.m + share_row(x0.step, c) : x1.m + share_row(x1.step, c - x0.n));
    };
    auto share_l = [&](int c) {
        return __ldcg(c < x0.n ? x0.l + share_row(x0.step, c) : x1.l + share_row(x1.step, c - x0.n));
    };
    constexpr int LOADS = 8;
    float4 o[LOADS];
    auto load = [&](int c0) {                                 // this warp's shares of c0 .. c0 + LOADS * WPR - 1
#pragma unroll
        for (int y = 0; y < LOADS; ++y) {
            const int c = c0 + y * WPR + sub;
            o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c < n && lane < D / 4)                        // without a weight too: it may hold infinities
                o[y] = __ldcg(reinterpret_cast<const float4*>(c < x0.n ? x0.o + share_row(x0.step, c) * D
                                                                       : x1.o + share_row(x1.step, c - x0.n) * D) + lane);
        }
    };
    load(0);                                                  // on their way beside the maxima
    float M = -INFINITY, m = -INFINITY, l = 0.f;              // m, l: of share `lane`
    if (lane < n) {
        m = share_m(lane);
        l = share_l(lane);
        M = m;
    }
    for (int c = 32 + lane; c < n; c += 32) M = fmaxf(M, share_m(c));
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, i));
    float den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < n; c0 += 32) {
        float w = 0.f;
        if (c0 + lane < n) {
            if (c0 > 0) {
                m = share_m(c0 + lane);
                l = share_l(c0 + lane);
            }
            w = share_weight(c0 + lane < x0.n ? own.tensor != 0 : pre.tensor != 0, m, M, l, scale);
            den = fmaf(w, l, den);
        }
        for (int c = c0; c < min(n, c0 + 32); c += LOADS * WPR) {
            if (c > 0) load(c);
#pragma unroll
            for (int y = 0; y < LOADS; ++y) {
                const float wc = __shfl_sync(kFullMask, w, (c + y * WPR + sub) & 31);
                if (c + y * WPR + sub >= n) continue;
                num.x = fmaf(o[y].x, wc, num.x);
                num.y = fmaf(o[y].y, wc, num.y);
                num.z = fmaf(o[y].z, wc, num.z);
                num.w = fmaf(o[y].w, wc, num.w);
            }
        }
    }
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) den += __shfl_xor_sync(kFullMask, den, i);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    if constexpr (WPR > 1) {
        if (lane < D / 4) s_num[warp][lane] = num;
        __syncthreads();
        if (sub == 0 && lane < D / 4) {
#pragma unroll
            for (int x = 1; x < WPR; ++x) {
                const float4 y = s_num[warp + x][lane];
                num = make_float4(num.x + y.x, num.y + y.y, num.z + y.z, num.w + y.w);
            }
        }
    }
    if (sub == 0 && lane < D / 4) *out = make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
    if (stats != nullptr && sub == 0 && lane == 0) stats[row] = make_float2(M, inv);
}

}  // namespace sa
