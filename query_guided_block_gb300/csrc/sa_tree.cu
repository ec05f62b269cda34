// Attention of a tree of drafted tokens over a paged cache: Q queries per sequence, each over
// the context (all of it or its KV head's selected blocks) and over the drafts its mask names.
//
// This file: the kernel for every type combination on warp-level matrix instructions, and
// the launcher.  Per 64-token tile of the unit's list (sa_tree.cuh) and warp of 16 query
// rows: S = Q K^T, the softmax with a running maximum and sum on the accumulator fragments,
// O += P V with the score fragments as the A operand.
//   bf16 K/V: mma.m16n8k16, fp32 accumulation.  P goes in as three bf16 parts cut off its 24
//     bits, which add up to it exactly (two would leave up to 2^-15 of every weight, more than
//     an fp32 softmax's own error), an fp32 query likewise.
//   fp32 K/V: mma.m16n8k8 on tf32 parts, x = hi + lo rounded to nearest (22 bits), the three
//     products that matter: each operand is off by at most 2^-22 of itself and lo lo, as much, is
//     left out.  Three parts would take six products for these three, which bound such calls.
//     (Measured error against 64 bits 3.5e-7 to 8e-7, a plain fp32 computation's 4.1e-7 to 5e-7.)
//     The channel (token) order inside a k-step is permuted alike on both sides, so that a thread's
//     two elements are neighbours in memory.
// The matrix unit rounds its running sum toward zero at every step, so a long chain drifts
// (measured: 1e-5 of the output after 8K tokens).  A tile's product is therefore summed from
// zero and joins the running O by one fused multiply-add, which carries the rescaling too.
// Weights are ex2.approx: 2^-22 of themselves, 0 below 2^-126 of the largest.
// Four warps: 4 x 16 rows over the same tokens, or with at most 16 rows 4 x 16 tokens over the
// same rows, their (m, l, o) joined at the item's end.
#include "sa_tree_kernel.cuh"

namespace sa {
namespace {

template <int D, bool KB, int NQ, int RW>
cudaError_t launch_tree_t(TreeArgs a, cudaStream_t s)
{
    using SH = TrShape<D, KB>;
    const size_t smem = 128 + size_t(SH::STAGES) * SH::STAGE + (KB ? 0 : size_t(16 * RW) * SH::Q_ROW * 4);
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(tree_kernel<D, KB, NQ, RW, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    });
    if (cfg != cudaSuccess) return cfg;
    a.tile = kTrTile;
    a.item_rows = 16 * RW;
    a.row_groups = (a.R + a.item_rows - 1) / a.item_rows;
    a.min_per = 2;
    a.half_slack = 4;
    int ctas = num_sms() * (2 * (smem + 10 * 1024) <= size_t(kSmemPerSm) ? 2 : 1);
    if (ctas > kTreeMaxCtas) ctas = kTreeMaxCtas;
    tree_choose_combine(a, ctas);
    const cudaError_t e = launch_after_previous(tree_kernel<D, KB, NQ, RW, false>, dim3(unsigned(ctas)), dim3(kTrThreads), smem, s, a);
    return e == cudaSuccess && a.combine ? launch_tree_combine(a, s) : e;
}

template <int D, bool KB, int NQ>
cudaError_t launch_tree_rows(const TreeArgs& a, cudaStream_t s)
{
    return a.R <= 16 ? launch_tree_t<D, KB, NQ, 1>(a, s) : launch_tree_t<D, KB, NQ, 4>(a, s);
}

// Adds up the parts of shared items: a warp per query row, a quarter of a float4 row per lane.
template <int D>
__global__ void __launch_bounds__(128) tree_combine_kernel(TreeArgs a)
{
    allow_dependents_early();
    grid_dependency_wait();   // the parts come from the previous kernel
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
    if (row >= a.B * a.Hkv * a.R) return;
    const int u = row / a.R, r = row - u * a.R, rg = r / a.item_rows, rr = r - rg * a.item_rows;
    const int b = u / a.Hkv, kvh = u - b * a.Hkv;
    const int len = a.seq_lens != nullptr ? a.seq_lens[b] : a.N;
    if (len < 0 || len > a.N) return;                         // inactive: no output
    const int2 at = a.item_parts[u * a.row_groups + rg];
    if (at.y <= 1) return;                                    // written whole
    // the first part of an item is the second slot of its CTA, the others are first slots
    auto slot = [&](int c) { return (long long)(2 * (at.x + c) + (c == 0 ? 1 : 0)) * a.item_rows + rr; };
    float M = -INFINITY;
    for (int c = lane; c < at.y; c += 32) M = fmaxf(M, __ldcg(a.part_m + slot(c)));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, x));
    float den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c0 = 0; c0 < at.y; c0 += 32) {
        float w = 0.f;
        if (c0 + lane < at.y) {
            const float m = __ldcg(a.part_m + slot(c0 + lane));
            const float l = __ldcg(a.part_l + slot(c0 + lane));
            w = tree_share(m, M, l, a.merge_scale);
            den = fmaf(w, l, den);
        }
        const int n = min(32, at.y - c0);
        for (int c = 0; c < n; c += 8) {
            float4 o[8];
            float wc[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                wc[x] = __shfl_sync(kFullMask, w, (c + x) & 31);
                o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (c + x < n && lane < D / 4)
                    o[x] = __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(c0 + c + x) * D) + lane);
            }
#pragma unroll
            for (int x = 0; x < 8; ++x) {
                const float wx = c + x < n ? wc[x] : 0.f;
                num.x = fmaf(o[x].x, wx, num.x);
                num.y = fmaf(o[x].y, wx, num.y);
                num.z = fmaf(o[x].z, wx, num.z);
                num.w = fmaf(o[x].w, wx, num.w);
            }
        }
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) den += __shfl_xor_sync(kFullMask, den, x);
    const float inv = den == 0.f ? 0.f : 1.f / den;
    if (lane < D / 4)
        reinterpret_cast<float4*>(a.out + tree_out_row(a, b, kvh, r) * D)[lane] =
            make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

}  // namespace

// Tokens that a sequence's queries meet at most, rounded up to whole selected blocks.
static long long tree_list(const TreeArgs& a)
{
    return a.sel_ids == nullptr ? (long long)a.N + a.Q : (long long)a.sel_stride * a.bs + a.Q + 2 * a.bs;
}

void tree_choose_combine(TreeArgs& a, int ctas)
{
    const long long items = (long long)a.B * a.Hkv * a.row_groups;
    const long long tiles = (tree_list(a) + a.tile - 1) / a.tile;    // of an item at most
    long long parts = tiles / a.min_per;
    if (parts > ctas / items) parts = ctas / items;
    // With more than half as many items as CTAs, those of equal length need no join unless they are
    // longer than a part and the slack that keeps them whole.
    const long long part = items <= ctas ? (items * tiles + ctas - 1) / ctas : 0;
    const bool joins = parts > 1 || tiles > part + 2 * a.half_slack;
    const int rows = a.R < a.item_rows ? a.R : a.item_rows;
    a.combine = joins && rows >= kTreeCombineRows && (parts > 2 ? parts : 2) * rows * a.D * 4 >= kTreeCombineBytes;
}

cudaError_t launch_tree_combine(const TreeArgs& a, cudaStream_t s)
{
    const unsigned grid = unsigned(((long long)a.B * a.Hkv * a.R + 3) / 4);
    return a.D == 128 ? launch_after_previous(tree_combine_kernel<128>, dim3(grid), dim3(128), 0, s, a)
                      : launch_after_previous(tree_combine_kernel<64>, dim3(grid), dim3(128), 0, s, a);
}

TreeLayout tree_layout(const Geometry& g)
{
    TreeLayout L{};
    const int R = g.Q * g.G;
    const size_t rows = size_t(tree_item_rows(R));
    const size_t slots = 2 * size_t(kTreeMaxCtas);
    L.counters = 256;
    const size_t items = size_t(g.units()) * ((R + 15) / 16);
    // the counters are what calls leave to each other: the same words whatever the problem
    L.item_parts = align256(L.counters + kTreeMaxCtas * sizeof(uint32_t));
    L.part_m = align256(L.item_parts + items * sizeof(int2));
    L.part_l = align256(L.part_m + slots * rows * sizeof(float));
    L.part_o = align256(L.part_l + slots * rows * sizeof(float));
    L.total = align256(L.part_o + slots * rows * g.D * sizeof(float));
    return L;
}

cudaError_t launch_tree(const Geometry& g, const TreeCall& c, char* ws, cudaStream_t s)
{
    const TreeLayout L = tree_layout(g);
    TreeArgs a{};
    a.q = c.q;
    a.q_bf16 = g.q_bf16;
    a.k_pages = c.k_pages;
    a.v_pages = c.v_pages;
    a.block_table = c.block_table;
    a.seq_lens = c.seq_lens;
    a.sel_ids = c.sel_ids;
    a.sel_count = c.sel_count;
    a.mask = c.mask;
    a.out = c.out;
    a.B = g.B;
    a.Hq = g.Hq;
    a.Hkv = g.Hkv;
    a.G = g.G;
    a.Q = g.Q;
    a.R = g.Q * g.G;
    a.D = g.D;
    a.N = g.N;
    a.bs = g.bs;
    a.bs_shift = 0;
    while ((1 << a.bs_shift) < g.bs) ++a.bs_shift;
    a.nb = g.nb;
    a.nb_cap = g.nb_cap;
    a.num_pages = g.num_pages;
    a.sel_stride = g.sel_stride;
    a.mask_words = (g.Q + 31) / 32;
    a.scale_log2 = g.scale_log2;
    a.merge_scale = g.scale_log2;
    a.part_m = reinterpret_cast<float*>(ws + L.part_m);
    a.part_l = reinterpret_cast<float*>(ws + L.part_l);
    a.part_o = reinterpret_cast<float*>(ws + L.part_o);
    a.counters = reinterpret_cast<uint32_t*>(ws + L.counters);
    a.item_parts = reinterpret_cast<int2*>(ws + L.item_parts);
    a.err = reinterpret_cast<uint32_t*>(ws);
    if (g.kv_bf16 && g.q_bf16) {
        const long long work = (long long)g.units() * ((a.R + 15) / 16) * ((tree_list(a) + kTrTile - 1) / kTrTile);
        if (a.R > 16 && work > (long long)kTreeSmallWork * num_sms()) return launch_tree_tc(a, s);
        return g.D == 128 ? launch_tree_t<128, true, 1, 1>(a, s) : launch_tree_t<64, true, 1, 1>(a, s);
    }
    if (g.kv_bf16) return g.D == 128 ? launch_tree_rows<128, true, 3>(a, s) : launch_tree_rows<64, true, 3>(a, s);
    return g.D == 128 ? launch_tree_rows<128, false, 1>(a, s) : launch_tree_rows<64, false, 1>(a, s);
}

}  // namespace sa
