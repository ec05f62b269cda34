// Attention that also adds up, for every cached token, the weight that the query rows of its KV head gave
// it:  weights[t] += sum_r exp(scale q_r.k_t) / sum_t' exp(scale q_r.k_t').
//
// A weight is known once its row's total is, after all keys.  The attention launch therefore leaves its
// scores (4 bytes a row and token, beside 2 D bytes of keys and as many of values), the joining launch
// every row's maximum and total, and a third launch turns the scores into weights: a thread has four
// tokens and adds up the rows in their order, so the sums do not depend on timing.  With many rows of
// bf16 the scores are computed again instead (sa_weigh_tc.cu).
#include "sa_tree_join.cuh"

namespace sa {
namespace {

constexpr int kWgThreads = 128;
constexpr int kWgTokens = 4 * kWgThreads;
constexpr int kWgRows = 256;                                 // rows whose maxima and totals are at hand
constexpr uint32_t kNotSeenScore = 0xffffffffu;              // as the attention launch marks it

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Adds what n rows give to the four tokens at `at` (their scores, a row `stride` floats from the next);
// s_row: the rows' maxima and 1 / totals.
__device__ __forceinline__ void add_rows(float (&sum)[4], const float* at, int n, long long stride, const float2* s_row, float scale)
{
    for (int r = 0; r < n; r += 4) {
        float4 x[4];
#pragma unroll
        for (int y = 0; y < 4; ++y)
            if (r + y < n) x[y] = __ldcs(reinterpret_cast<const float4*>(at + (r + y) * stride));
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            if (r + y >= n) break;
            const float2 st = s_row[r + y];
            if (st.y == 0.f) continue;                       // a row without a total
            const float s[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (__float_as_uint(s[e]) != kNotSeenScore) sum[e] = fmaf(fast_exp2((s[e] - st.x) * scale), st.y, sum[e]);
        }
    }
}

// The sums join the weights of tokens t .. t + 3; new tokens' are set.
__device__ __forceinline__ void store_weights(float* w, const float (&sum)[4], int t, int len, int end)
{
    if (t + 4 <= len) {
        const float4 old = *reinterpret_cast<const float4*>(w);
        *reinterpret_cast<float4*>(w) = make_float4(old.x + sum[0], old.y + sum[1], old.z + sum[2], old.w + sum[3]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (t + e < end) w[e] = t + e < len ? w[e] + sum[e] : sum[e];
    }
}

// CTA = (unit, every `chunks`th run of 512 tokens).
__global__ void __launch_bounds__(kWgThreads) weigh_kernel(TreeArgs a, const float2* stats, float* weights, long long w_stride,
                                                          int chunks)
{
    __shared__ float2 s_row[kWgRows];
    allow_dependents_early();
    grid_dependency_wait();   // scores, totals and weights come from previous kernels
    const int u = int(blockIdx.x) / chunks, b = u / a.Hkv, kvh = u - b * a.Hkv;
    const int len = a.seq_lens != nullptr ? a.seq_lens[b] : a.N;
    if (len < 0 || len > a.N) return;
    const int end = len + a.Q;
    for (int base = (int(blockIdx.x) - u * chunks) * kWgTokens; base < end; base += chunks * kWgTokens) {
        const int t = base + 4 * threadIdx.x;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r0 = 0; r0 < a.R; r0 += kWgRows) {
            const int n = min(kWgRows, a.R - r0);
            __syncthreads();
            for (int i = threadIdx.x; i < n; i += kWgThreads) s_row[i] = stats[tree_out_row(a, b, kvh, r0 + i)];
            __syncthreads();
            if (t < end) add_rows(sum, a.scores + ((long long)u * a.R + r0) * a.score_stride + t, n, a.score_stride, s_row, a.scale_log2);
        }
        store_weights(weights + u * w_stride + t, sum, t, len, end);
    }
}

// With few rows the join and the sums are one launch: the first CTAs are those of weigh_kernel, and find the
// rows' maxima and totals from the shares by themselves (a warp a row, lane = share), the others join rows.
// One token over 4096: 16.5 us, 18.8 in three launches;
// 32 rows over 32K tokens 87, 65 in three.
constexpr int kWgFew = 8;

template <int D, int WPR>
__global__ void __launch_bounds__(kJoinThreads) weigh_join_kernel(const __grid_constant__ TreeArgs a, float* weights,
                                                                  long long w_stride, int chunks, int weigh_ctas)
{
    static_assert(kWgThreads == kJoinThreads, "one launch");
    __shared__ float2 s_row[kWgFew];
    allow_dependents_early();
    grid_dependency_wait();   // scores, shares and weights come from previous kernels
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (int(blockIdx.x) >= weigh_ctas) {
        const int row = (int(blockIdx.x) - weigh_ctas) * (kJoinWarps / WPR) + warp / WPR;
        if (row < a.seqs * a.Q * a.Hq) join_row<D, WPR>(a, a, 0, nullptr, row);     // whole warps, and whole CTAs with WPR = 4
        return;
    }
    const int u = int(blockIdx.x) / chunks, b = u / a.Hkv, kvh = u - b * a.Hkv;
    const int len = a.seq_lens != nullptr ? a.seq_lens[b] : a.N;
    if (len < 0 || len > a.N) return;
    const int end = len + a.Q, first = (int(blockIdx.x) - u * chunks) * kWgTokens;
    if (first >= end) return;
    for (int r = warp; r < a.R; r += kJoinWarps) {
        const long long row = tree_out_row(a, b, kvh, r);
        const int rg = r / a.item_rows;
        const int2 parts = a.item_parts[kvh * tree_notes_per_head(a, false, a.item_rows) + (long long)b * a.row_groups + rg];
        float2 st;
        if (parts.y <= 1) {
            st = a.stats[row];
        } else {
            const Shares x = shares_of(a, parts, r - rg * a.item_rows, row);
            float M = -INFINITY, den = 0.f;
            for (int c = lane; c < x.n; c += 32) M = fmaxf(M, __ldcg(x.m + share_row(x.step, c)));
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, i));
            for (int c = lane; c < x.n; c += 32) {
                const float l = __ldcg(x.l + share_row(x.step, c));
                den = fmaf(share_weight(a.tensor != 0, __ldcg(x.m + share_row(x.step, c)), M, l, a.scale_log2), l, den);
            }
#pragma unroll
            for (int i = 16; i > 0; i >>= 1) den += __shfl_xor_sync(kFullMask, den, i);
            st = make_float2(M, den == 0.f ? 0.f : 1.f / den);
        }
        if (lane == 0) s_row[r] = st;
    }
    __syncthreads();
    for (int base = first; base < end; base += chunks * kWgTokens) {
        const int t = base + 4 * threadIdx.x;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        if (t < end) add_rows(sum, a.scores + (long long)u * a.R * a.score_stride + t, a.R, a.score_stride, s_row, a.scale_log2);
        store_weights(weights + u * w_stride + t, sum, t, len, end);
    }
}

template <int D, int WPR>
cudaError_t launch_weigh_join(const TreeArgs& a, float* weights, long long w_stride, int chunks, int units, cudaStream_t s)
{
    const long long rows = (long long)a.seqs * a.Q * a.Hq, per = kJoinWarps / WPR, weigh_ctas = (long long)chunks * units;
    return launch_after_previous(weigh_join_kernel<D, WPR>, dim3(unsigned(weigh_ctas + (rows + per - 1) / per)), dim3(kJoinThreads), 0,
                                 s, a, weights, w_stride, chunks, int(weigh_ctas));
}

struct WeighLayout {
    TreeExtLayout own;
    size_t stats, scores, end;
    long long stride;
};

// Tiles of 64 tokens x 16 rows.
long long weigh_tiles(const Geometry& g, long long tokens)
{
    return (long long)g.units() * ((g.Q * g.G + 15) / 16) * ((tokens + kTreeLeastTile - 1) / kTreeLeastTile);
}

size_t weigh_scores(const Geometry& g, long long tokens)     // bytes
{
    return size_t(g.units()) * g.Q * g.G * size_t((tokens + kTreeLeastTile - 1) / kTreeLeastTile * kTreeLeastTile) * sizeof(float);
}

// Scores are kept where the tensor-core kernels do not run.  Those also take 17 to 32 rows of bf16 whose scores
// would be more than this, which costs a few percent (see tree_ext_tensor).
constexpr size_t kWgMostScores = size_t(256) << 20;
bool weigh_tensor(const Geometry& g, long long tokens)
{
    const bool bf16 = g.kv_bf16 && g.q_bf16;
    const int rows = g.Q * g.G;
    return tree_ext_tensor(kTreeAll, bf16, rows, weigh_tiles(g, tokens)) ||
           (bf16 && rows > 16 && rows <= 32 && weigh_scores(g, tokens) > kWgMostScores);
}

WeighLayout weigh_layout(const Geometry& g, long long tokens)
{
    WeighLayout L{};
    L.own = tree_ext_layout(g, kTreeWsFree, 0);
    L.stride = (tokens + kTreeLeastTile - 1) / kTreeLeastTile * kTreeLeastTile;   // whole tiles are written
    L.stats = L.own.end;
    L.scores = align256(L.stats + size_t(g.B) * g.Q * g.Hq * sizeof(float2));
    size_t kept = weigh_scores(g, tokens);
    // with more tokens than that none are kept: then room for any fewer
    if (weigh_tensor(g, tokens)) kept = g.Q * g.G <= 32 ? kWgMostScores : size_t(kTreeSmallWork) * 152 * kTreeLeastTile * 16 * sizeof(float);
    L.end = align256(L.scores + kept);
    return L;
}

}  // namespace

size_t weigh_workspace(const Geometry& g, long long tokens) { return weigh_layout(g, tokens).end; }

cudaError_t launch_weigh(const Geometry& g, const TreeCall& c, float* weights, char* ws, cudaStream_t s)
{
    const WeighLayout L = weigh_layout(g, (long long)g.N + g.Q);
    TreeArgs a = tree_ext_args(g, c, ws, L.own);
    a.pass = kTreeAll;
    float2* stats = reinterpret_cast<float2*>(ws + L.stats);
    a.stats = stats;
    const long long tokens = (long long)g.N + g.Q, w_stride = (long long)g.nb_cap * g.bs;
    const bool tensor = weigh_tensor(g, tokens);
    if (!tensor) {
        a.scores = reinterpret_cast<float*>(ws + L.scores);
        a.score_stride = L.stride;
    }
    cudaError_t e = launch_tree_ext(a, g.kv_bf16, a.R, tensor, s);
    if (e != cudaSuccess) return e;
    long long chunks = (tokens + kWgTokens - 1) / kWgTokens;
    const long long most = (8LL * num_sms() + g.units() - 1) / g.units() * 4;   // more would only start and end
    if (chunks > most) chunks = most;
    const long long rows = (long long)g.B * g.Q * g.Hq;
    if (!tensor && a.R <= kWgFew && rows < 64LL * num_sms()) {
        if (rows <= 4LL * num_sms())
            return g.D == 128 ? launch_weigh_join<128, kJoinWarps>(a, weights, w_stride, int(chunks), g.units(), s)
                              : launch_weigh_join<64, kJoinWarps>(a, weights, w_stride, int(chunks), g.units(), s);
        return g.D == 128 ? launch_weigh_join<128, 1>(a, weights, w_stride, int(chunks), g.units(), s)
                          : launch_weigh_join<64, 1>(a, weights, w_stride, int(chunks), g.units(), s);
    }
    e = launch_tree_join(a, nullptr, stats, s);
    if (e != cudaSuccess) return e;
    if (tensor) return launch_weigh_tc(a, stats, weights, w_stride, s);
    return launch_after_previous(weigh_kernel, dim3(unsigned(chunks * g.units())), dim3(kWgThreads), 0, s, a,
                                 (const float2*)stats, weights, w_stride, int(chunks));
}

}  // namespace sa
