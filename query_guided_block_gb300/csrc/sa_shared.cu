// Attention of a batch whose groups of sequences share a long prefix, the prefix's keys and values read
// once a group:
//   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale q.k_t),
// over the prefix, the sequence's own context and the drafts it sees.  Sums over parts of the tokens
// add up once they are relative to one maximum, so the prefix is one launch, in which all the
// members' query rows are rows of one item, the own tokens are another, and a third joins the shares (m, l, o).
//
// The launches are the EXT form of the draft-tree kernels (sa_tree_kernel.cuh).
#include "sa_tree.cuh"

namespace sa {
namespace {

constexpr int kJoinWarps = 4;
constexpr int kJoinThreads = 32 * kJoinWarps;

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

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
__device__ __forceinline__ void join_row(const TreeArgs& own, const TreeArgs& pre, int with_prefix, float2* stats, int row);

constexpr int kJoinMany = 8;               // rows of a warp that looks for what is left

template <int D, int WPR>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const __grid_constant__ TreeArgs own,
                                                                 const __grid_constant__ TreeArgs pre, int with_prefix,
                                                                 float2* stats, int many)
{
    allow_dependents_early();
    grid_dependency_wait();   // the shares come from the previous kernels
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = own.seqs * own.Q * own.Hq;
    if (WPR == 1 && many) {
        const int first = (int(blockIdx.x) * kJoinWarps + warp) * kJoinMany, row = first + lane;
        bool left = false;
        if (lane < kJoinMany && row < rows) {
            const int h = row % own.Hq, bt = row / own.Hq, b = bt / own.Q, kvh = h / own.G;
            const int rg = ((bt - b * own.Q) * own.G + h - kvh * own.G) / own.item_rows;
            const int len = own.seq_lens != nullptr ? own.seq_lens[b] : own.N;
            if (len >= 0 && len <= own.N)
                left = own.item_parts[kvh * tree_notes_per_head(own, false, own.item_rows) + (long long)b * own.row_groups + rg].y > 1;
        }
        for (uint32_t todo = __ballot_sync(kFullMask, left); todo != 0u; todo &= todo - 1)
            join_row<D, WPR>(own, pre, with_prefix, stats, first + __ffs(todo) - 1);
        return;
    }
    const int row = int(blockIdx.x) * (kJoinWarps / WPR) + warp / WPR;
    if (row < rows) join_row<D, WPR>(own, pre, with_prefix, stats, row);       // whole warps, and whole CTAs with WPR = 4
}

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

template <int D, int WPR>
cudaError_t launch_join_t(const TreeArgs& own, const TreeArgs* prefix, float2* stats, cudaStream_t s)
{
    static_assert(WPR == 1 || WPR == kJoinWarps, "a CTA is one row or a row a warp");
    const long long rows = (long long)own.seqs * own.Q * own.Hq;
    const bool many = WPR == 1 && own.pass == kTreeAll && rows >= 256LL * num_sms();
    const long long per = kJoinWarps / WPR * (many ? kJoinMany : 1);
    return launch_after_previous(tree_join_kernel<D, WPR>, dim3(unsigned((rows + per - 1) / per)), dim3(kJoinThreads), 0, s, own,
                                 prefix != nullptr ? *prefix : own, int(prefix != nullptr), stats, int(many));
}

}  // namespace

cudaError_t launch_tree_join(const TreeArgs& own, const TreeArgs* prefix, float2* stats, cudaStream_t s)
{
    const bool few = (long long)own.seqs * own.Q * own.Hq <= 4LL * num_sms();
    if (own.D == 128) return few ? launch_join_t<128, kJoinWarps>(own, prefix, stats, s) : launch_join_t<128, 1>(own, prefix, stats, s);
    return few ? launch_join_t<64, kJoinWarps>(own, prefix, stats, s) : launch_join_t<64, 1>(own, prefix, stats, s);
}

TreeExtLayout tree_ext_layout(const Geometry& g, size_t at, int groups)
{
    TreeExtLayout L{};
    TreeArgs a{};
    a.seqs = g.B;
    a.groups = groups;
    a.R = g.Q * g.G;
    const size_t notes = size_t(g.Hkv) * size_t(tree_notes_per_head(a, groups > 0, 16));
    const size_t slots = 2 * size_t(kTreeMaxCtas) * kTreeMaxRows, rows = size_t(g.B) * g.Q * g.Hq;
    L.item_parts = at;
    L.part_m = align256(L.item_parts + notes * sizeof(int2));
    L.part_l = align256(L.part_m + slots * sizeof(float));
    L.part_o = align256(L.part_l + slots * sizeof(float));
    L.row_m = align256(L.part_o + slots * g.D * sizeof(float));
    L.row_l = align256(L.row_m + rows * sizeof(float));
    L.end = align256(L.row_l + rows * sizeof(float));
    return L;
}

TreeArgs tree_ext_args(const Geometry& g, const TreeCall& c, char* ws, const TreeExtLayout& L)
{
    TreeArgs a{};
    a.q = c.q;
    a.q_bf16 = g.q_bf16;
    a.k_pages = c.k_pages;
    a.v_pages = c.v_pages;
    a.block_table = c.block_table;
    a.seq_lens = c.seq_lens;
    a.mask = c.mask;
    a.out = c.out;
    a.B = a.seqs = g.B;
    a.Hq = g.Hq;
    a.Hkv = g.Hkv;
    a.G = g.G;
    a.Q = g.Q;
    a.R = g.Q * g.G;
    a.D = g.D;
    a.N = g.N;
    a.bs = g.bs;
    while ((1 << a.bs_shift) < g.bs) ++a.bs_shift;
    a.nb = g.nb;
    a.nb_cap = g.nb_cap;
    a.num_pages = g.num_pages;
    a.mask_words = (g.Q + 31) / 32;
    a.scale_log2 = g.scale_log2;
    a.merge_scale = g.scale_log2;
    a.combine = 1;
    a.item_parts = reinterpret_cast<int2*>(ws + L.item_parts);
    a.part_m = reinterpret_cast<float*>(ws + L.part_m);
    a.part_l = reinterpret_cast<float*>(ws + L.part_l);
    a.part_o = reinterpret_cast<float*>(ws + L.part_o);
    a.row_m = reinterpret_cast<float*>(ws + L.row_m);
    a.row_l = reinterpret_cast<float*>(ws + L.row_l);
    a.err = reinterpret_cast<uint32_t*>(ws);
    return a;
}

namespace {

struct SharedLayout {
    size_t seq_prefix, seq_group, prior;
    TreeExtLayout prefix, own;
};

SharedLayout shared_layout(const Geometry& g, int groups)
{
    SharedLayout L{};
    L.seq_prefix = kTreeWsFree;
    L.seq_group = align256(L.seq_prefix + size_t(g.B) * sizeof(int32_t));
    L.prior = align256(L.seq_group + size_t(g.B) * sizeof(int32_t));
    L.prefix = tree_ext_layout(g, align256(L.prior + size_t(g.B) * g.Q * g.Hq * g.D * sizeof(float)), groups);
    L.own = tree_ext_layout(g, L.prefix.end, 0);
    return L;
}

}  // namespace

size_t shared_workspace(const Geometry& g, int groups) { return shared_layout(g, groups).own.end; }

cudaError_t launch_shared(const Geometry& g, const TreeCall& c, int groups, const int32_t* cu_seqs, const int32_t* prefix_lens,
                          char* ws, cudaStream_t s)
{
    const SharedLayout L = shared_layout(g, groups);
    TreeArgs pre = tree_ext_args(g, c, ws, L.prefix);
    pre.pass = kTreePrefix;
    pre.B = pre.groups = groups;
    pre.cu_seqs = cu_seqs;
    pre.prefix_lens = prefix_lens;
    pre.seq_prefix = reinterpret_cast<int32_t*>(ws + L.seq_prefix);
    pre.seq_group = reinterpret_cast<int32_t*>(ws + L.seq_group);
    pre.out = reinterpret_cast<float*>(ws + L.prior);
    TreeArgs own = tree_ext_args(g, c, ws, L.own);
    own.pass = kTreeOwn;
    own.seq_prefix = pre.seq_prefix;
    own.seq_group = pre.seq_group;
    // What the launches go by: groups of even sizes; the prefixes and the rest are not known here, so each
    // launch is taken for the larger part of the contexts.
    const long long rows = (long long)(g.B > groups ? g.B : groups) * pre.R / groups;
    const long long tiles = (g.N + kTreeLeastTile - 1) / kTreeLeastTile;
    const int pre_rows = int(rows < 1024 ? rows : 1024);
    const long long pre_tiles = tiles * groups * g.Hkv * ((rows + 15) / 16), own_tiles = tiles * g.units() * ((own.R + 15) / 16);
    const bool bf16 = g.kv_bf16 && g.q_bf16;
    if (!tree_ext_tensor(kTreePrefix, bf16, pre_rows, pre_tiles) && !tree_ext_tensor(kTreeOwn, bf16, own.R, own_tiles) &&
        (bf16 || tree_ext_item_rows(bf16, pre_rows) == tree_ext_item_rows(bf16, own.R))) {
        // Both kinds on one line of work, in items of the own rows' size (more rows of bf16 are then few tiles):
        // 4 samples of a 777-token prompt 16.3 us, two launches 25.
        pre.pass = kTreeBoth;
        pre.B = groups + g.B;
        pre.own_out = own.out;
        pre.own_row_m = own.row_m;
        pre.own_row_l = own.row_l;
        pre.own_item_parts = own.item_parts;
        const cudaError_t e = launch_tree_ext(pre, g.kv_bf16, own.R, 0, s);
        if (e != cudaSuccess) return e;
        own.part_m = pre.part_m;
        own.part_l = pre.part_l;
        own.part_o = pre.part_o;
        own.item_rows = pre.item_rows;
        own.row_groups = (own.R + own.item_rows - 1) / own.item_rows;
        return launch_tree_join(own, &pre, nullptr, s);
    }
    cudaError_t e = launch_tree_ext(pre, g.kv_bf16, pre_rows, pre_tiles, s);
    if (e == cudaSuccess) e = launch_tree_ext(own, g.kv_bf16, own.R, own_tiles, s);
    return e == cudaSuccess ? launch_tree_join(own, &pre, nullptr, s) : e;
}

}  // namespace sa
