// Attention of a batch whose groups of sequences share a long prefix, the prefix's keys and values read
// once a group:
//   out = sum_t w_t v_t / sum_t w_t,  w_t = exp(scale q.k_t),
// over the prefix, the sequence's own context and the drafts it sees.  Sums over parts of the tokens
// add up once they are relative to one maximum, so the prefix is one launch, in which all the
// members' query rows are rows of one item, the own tokens are another, and a third joins the shares (m, l, o).
// Where neither needs the tensor-core kernel, prefixes and own tokens are one launch.
//
// The launches are the EXT form of the draft-tree kernels (sa_tree_kernel.cuh).
#include "sa_tree_join.cuh"

namespace sa {
namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

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
    size_t seq_prefix, seq_group, cu_seqs, prior;
    TreeExtLayout prefix, own;
};

SharedLayout shared_layout(const Geometry& g, int groups)
{
    SharedLayout L{};
    L.seq_prefix = kTreeWsFree;
    L.seq_group = align256(L.seq_prefix + size_t(g.B) * sizeof(int32_t));
    L.cu_seqs = align256(L.seq_group + size_t(g.B) * sizeof(int32_t));
    L.prior = align256(L.cu_seqs + (size_t(groups) + 1) * sizeof(int32_t));
    L.prefix = tree_ext_layout(g, align256(L.prior + size_t(g.B) * g.Q * g.Hq * g.D * sizeof(float)), groups);
    L.own = tree_ext_layout(g, L.prefix.end, 0);
    return L;
}

// Groups out of order may overlap, up to every group being the whole batch.  The launches number the tiles of their
// items in 32 bits, which hold them as long as every sequence is in one group at most.  Whether they also hold the
// most that any cu_seqs can name:
bool any_groups_fit(const Geometry& g, int groups)
{
    const long long tiles = (long long)g.nb_cap * g.bs / kTreeLeastTile + 1, R = g.Q * g.G;
    const long long rows = ((long long)g.B * R + 15) / 16 * g.Hkv, own = (R + 15) / 16 * g.units();
    return double(tiles) * (double(groups) * double(rows) + double(own)) < double(INT32_MAX / 2);
}

// Where they do not, cu_seqs is looked over first, by one CTA: `to` becomes a copy or, with groups out of order,
// all 0, which leaves every sequence to itself.
constexpr int kOrderThreads = 1024;

__global__ void __launch_bounds__(kOrderThreads) order_kernel(const int32_t* cu_seqs, int groups, int32_t* to, uint32_t* err)
{
    allow_dependents_early();
    grid_dependency_wait();   // the groups may come from the previous kernel
    int bad = 0;
    for (int i = threadIdx.x; i < groups; i += kOrderThreads) bad |= cu_seqs[i] > cu_seqs[i + 1];
    bad = __syncthreads_or(bad);
    if (bad && threadIdx.x == 0) raise_error(err, SPARSE_ATTN_ERR_LENGTH);
    for (int i = threadIdx.x; i <= groups; i += kOrderThreads) to[i] = bad ? 0 : cu_seqs[i];
}

}  // namespace

size_t shared_workspace(const Geometry& g, int groups) { return shared_layout(g, groups).own.end; }

cudaError_t launch_shared(const Geometry& g, const TreeCall& c, int groups, const int32_t* cu_seqs, const int32_t* prefix_lens,
                          char* ws, cudaStream_t s)
{
    const SharedLayout L = shared_layout(g, groups);
    if (!any_groups_fit(g, groups)) {
        int32_t* to = reinterpret_cast<int32_t*>(ws + L.cu_seqs);
        const cudaError_t e = launch_after_previous(order_kernel, dim3(1), dim3(kOrderThreads), 0, s, cu_seqs, groups, to,
                                                    reinterpret_cast<uint32_t*>(ws));
        if (e != cudaSuccess) return e;
        cu_seqs = to;
    }
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
    const bool pre_tensor = tree_ext_tensor(kTreePrefix, bf16, pre_rows, pre_tiles);
    const bool own_tensor = tree_ext_tensor(kTreeOwn, bf16, own.R, own_tiles);
    if (!pre_tensor && !own_tensor && (bf16 || tree_ext_item_rows(bf16, pre_rows) == tree_ext_item_rows(bf16, own.R))) {
        // Both kinds on one line of work, in items of the own rows' size (more rows of bf16 are then few tiles):
        // 4 samples of a 777-token prompt 16.3 us, two launches 25.
        pre.pass = kTreeBoth;
        pre.B = groups + g.B;
        pre.own_out = own.out;
        pre.own_row_m = own.row_m;
        pre.own_row_l = own.row_l;
        pre.own_item_parts = own.item_parts;
        const cudaError_t e = launch_tree_ext(pre, g.kv_bf16, own.R, false, s);
        if (e != cudaSuccess) return e;
        own.part_m = pre.part_m;
        own.part_l = pre.part_l;
        own.part_o = pre.part_o;
        own.item_rows = pre.item_rows;
        own.row_groups = (own.R + own.item_rows - 1) / own.item_rows;
        return launch_tree_join(own, &pre, nullptr, s);
    }
    cudaError_t e = launch_tree_ext(pre, g.kv_bf16, pre_rows, pre_tensor, s);
    if (e == cudaSuccess) e = launch_tree_ext(own, g.kv_bf16, own.R, own_tensor, s);
    return e == cudaSuccess ? launch_tree_join(own, &pre, nullptr, s) : e;
}

}  // namespace sa
