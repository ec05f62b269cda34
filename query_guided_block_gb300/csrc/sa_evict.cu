// Eviction from the paged cache by accumulated attention weight: for each (sequence, KV head) unit the
// first `sinks` tokens, the last `recent` ones and of the others those with the largest weights stay, in
// their order, in new pages.
//
// Two launches.  The first finds the kept tokens of a unit, by a thread-block cluster: the weights as
// keys of the same order, 32 bits, in shared memory; three histograms of 11, 11 and 10 bits, added up
// over the cluster, narrow the key of the last kept token down; tokens above it stay, of those equal to
// it as many as there is room for, lowest index first.  A kept token's place is the number of kept
// ones before it, which two ballots a warp give.  The second launch moves rows: K and V of 64 kept
// tokens a CTA, every load on its way before the first store, with their weights and their blocks' box.
// Bytes: 4 a cached token, then each kept row once in and once out.
#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvCache = 45056;            // keys of a CTA in shared memory; the rest is read again
constexpr int kEvMaxCluster = 8;
constexpr int kEvRun = 64;                 // kept tokens of a moving CTA when blocks are smaller

struct EvictArgs {
    const int32_t *seq_lens, *keep_lens, *block_table, *new_table;
    float* weights;                        // [units, w_stride]
    float* kept_weights;                   // [units, keep] workspace
    int32_t *kept_ids, *new_lens;          // [units, keep], [B]
    char *k_pages, *v_pages, *kmin, *kmax;
    uint32_t* err;
    long long w_stride;
    int B, Hkv, N, keep, sinks, recent, bs, nb_cap, nb_new, num_pages, row_bytes;
    int cluster, cache, run;
};

// Tokens of sequence b and how many of them stay; false: nothing of it is touched.
__device__ __forceinline__ bool evict_counts(const EvictArgs& a, int b, int& len, int& kept)
{
    len = a.seq_lens != nullptr ? a.seq_lens[b] : a.N;
    const int k = a.keep_lens != nullptr ? a.keep_lens[b] : a.keep;
    if (len == -1 || k == -1) return false;
    if (len < 0 || len > a.N || k < a.sinks + a.recent || k > a.keep) {
        raise_error(a.err, SPARSE_ATTN_ERR_LENGTH);
        return false;
    }
    kept = min(len, k);
    return true;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

__global__ void __launch_bounds__(kEvThreads, 1) evict_select_kernel(EvictArgs a)
{
    extern __shared__ uint32_t s_key[];
    __shared__ uint32_t s_hist[3][2048];
    __shared__ int s_warp[2][kEvWarps];
    __shared__ uint32_t s_total[2];        // kept for sure and equal to the last key, of this CTA
    __shared__ uint32_t s_found[2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int C = a.cluster, rank = int(cluster_ctarank());
    const int u = int(blockIdx.x) / C, b = u / a.Hkv;
    allow_dependents_early();
    grid_dependency_wait();   // lengths and weights may come from the previous kernel

    int n, kept;
    if (!evict_counts(a, b, n, kept)) return;                  // the whole cluster
    const float* w = a.weights + u * a.w_stride;
    int32_t* ids = a.kept_ids + (long long)u * a.keep;
    float* vals = a.kept_weights + (long long)u * a.keep;
    const int per = ((n + C - 1) / C + kEvThreads - 1) / kEvThreads * kEvThreads;   // tokens of a CTA
    const int i0 = min(n, rank * per), i1 = min(n, i0 + per);
    if (kept == n) {                                           // all of them
        for (int i = i0 + tid; i < i1; i += kEvThreads) {
            ids[i] = i;
            vals[i] = w[i];
        }
        return;
    }
    if (kept == 0) return;
    // Keys in the order of the weights; tokens that stay in any case are above all others.
    auto make_key = [&](int i) -> uint32_t {
        if (i < a.sinks || i >= n - a.recent) return 0xffffffffu;
        return min(order_key(w[i] + 0.f), 0xfffffffeu);        // + 0: no negative zero
    };
    auto key = [&](int i) { return i - i0 < a.cache ? s_key[i - i0] : make_key(i); };

    for (int i = tid; i < 3 * 2048; i += kEvThreads) (&s_hist[0][0])[i] = 0u;
    __syncthreads();
    for (int i = i0 + tid; i < i1; i += kEvThreads) {
        const uint32_t k = make_key(i);
        if (i - i0 < a.cache) s_key[i - i0] = k;
        atomicAdd(&s_hist[0][k >> 21], 1u);
    }
    uint32_t prefix = 0u;                                      // the last kept key's bits so far
    uint32_t room = uint32_t(kept);                            // tokens to take among those with these bits
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        if (pass > 0) {
            const int above = pass == 1 ? 21 : 10;
            for (int i = i0 + tid; i < i1; i += kEvThreads) {
                const uint32_t k = key(i);
                if ((k >> above) == (prefix >> above)) atomicAdd(&s_hist[pass][(k >> shift) & (pass == 1 ? 2047u : 1023u)], 1u);
            }
        }
        if (C > 1) cluster_sync_all();
        else __syncthreads();
        // from the largest digit down, four to a thread
        uint32_t h[4], sum = 0u;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int bin = 2047 - 4 * tid - x;
            h[x] = 0u;
            if (C == 1) h[x] = s_hist[pass][bin];
            else
                for (int r = 0; r < C; ++r) h[x] += ld_cluster_u32(cluster_map(smem_u32(&s_hist[pass][bin]), uint32_t(r)));
            sum += h[x];
        }
        const uint32_t incl = uint32_t(warp_inclusive_scan(int(sum), lane));
        if (lane == 31) s_warp[0][warp] = int(incl);
        __syncthreads();
        uint32_t at = incl - sum;
        for (int x = 0; x < warp; ++x) at += uint32_t(s_warp[0][x]);
        if (at < room && room <= at + sum) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                if (at < room && room <= at + h[x]) {
                    s_found[0] = uint32_t(2047 - 4 * tid - x);
                    s_found[1] = room - at;
                }
                at += h[x];
            }
        }
        __syncthreads();
        prefix |= s_found[0] << shift;
        room = s_found[1];
        __syncthreads();                                       // before s_warp and s_found are used again
    }
    // tokens with a key above `prefix` stay, and the first `room` of those equal to it
    const int seg = per / kEvWarps, w0 = min(i1, i0 + warp * seg), w1 = min(i1, w0 + seg);
    int gt = 0, eq = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t k = key(i);
        gt += k > prefix;
        eq += k == prefix;
    }
    gt = __reduce_add_sync(kFullMask, gt);
    eq = __reduce_add_sync(kFullMask, eq);
    if (lane == 0) {
        s_warp[0][warp] = gt;
        s_warp[1][warp] = eq;
    }
    __syncthreads();
    if (tid < 2) {
        uint32_t all = 0u;
        for (int x = 0; x < kEvWarps; ++x) all += uint32_t(s_warp[tid][x]);
        s_total[tid] = all;
    }
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    uint32_t gt_at = 0u, eq_at = 0u;
    for (int r = 0; r < rank; ++r) {
        gt_at += ld_cluster_u32(cluster_map(smem_u32(&s_total[0]), uint32_t(r)));
        eq_at += ld_cluster_u32(cluster_map(smem_u32(&s_total[1]), uint32_t(r)));
    }
    for (int x = 0; x < warp; ++x) {
        gt_at += uint32_t(s_warp[0][x]);
        eq_at += uint32_t(s_warp[1][x]);
    }
    for (int base = w0; base < w1; base += 32) {
        const int i = base + lane;
        const uint32_t k = i < w1 ? key(i) : 0u;
        const bool is_gt = i < w1 && k > prefix, is_eq = i < w1 && k == prefix;
        const uint32_t bg = __ballot_sync(kFullMask, is_gt), be = __ballot_sync(kFullMask, is_eq);
        const uint32_t g = gt_at + __popc(bg & lanemask_lt()), e = eq_at + __popc(be & lanemask_lt());
        if (is_gt || (is_eq && e < room)) {
            const uint32_t pos = g + min(e, room);
            ids[pos] = i;
            vals[pos] = w[i];
        }
        gt_at += __popc(bg);
        eq_at += __popc(be);
    }
    if (C > 1) cluster_sync_all();                             // others may still read this CTA's totals
}

// CTA = (unit, run of kept tokens): whole blocks of the new pages.
constexpr int kMvThreads = 256;
constexpr int kMvBatch = 4;                // rows of K and of V a thread has on their way

template <bool KB>
__global__ void __launch_bounds__(kMvThreads) evict_move_kernel(EvictArgs a)
{
    extern __shared__ __align__(16) uint4 s_rows[];            // [run][row], the moved keys, when there is a box
    __shared__ long long s_src[128], s_dst[128];               // byte offsets of the rows, -1: none
    const int tid = threadIdx.x;
    allow_dependents_early();
    grid_dependency_wait();   // the kept tokens come from the previous kernel

    const int chunks = (a.keep + a.run - 1) / a.run;
    const int u = int(blockIdx.x) / chunks, chunk = int(blockIdx.x) - u * chunks;
    const int b = u / a.Hkv, kvh = u - b * a.Hkv;
    int len, kept = 0;
    const bool active = evict_counts(a, b, len, kept);
    if (chunk == 0 && kvh == 0 && tid == 0) a.new_lens[b] = active ? kept : len;
    const int t0 = chunk * a.run, n = active ? min(a.run, kept - t0) : 0;
    if (n <= 0) return;
    if (tid < n) {
        const long long at = (long long)u * a.keep + t0 + tid;
        const int t = a.kept_ids[at];
        a.weights[u * a.w_stride + t0 + tid] = a.kept_weights[at];
        const int sp = a.block_table[(long long)b * a.nb_cap + t / a.bs];
        const int dp = a.new_table[(long long)b * a.nb_new + (t0 + tid) / a.bs];
        const bool ok = sp >= 0 && sp < a.num_pages && dp >= 0 && dp < a.num_pages;
        if (!ok) raise_error(a.err, SPARSE_ATTN_ERR_PAGE);
        s_src[tid] = ok ? (((long long)sp * a.Hkv + kvh) * a.bs + t % a.bs) * a.row_bytes : -1;
        s_dst[tid] = ok ? (((long long)dp * a.Hkv + kvh) * a.bs + (t0 + tid) % a.bs) * a.row_bytes : -1;
    }
    __syncthreads();
    const int CPR = a.row_bytes / 16, c_shift = __ffs(CPR) - 1;   // 16-byte chunks of a row: 8, 16 or 32
    const int c = tid & (CPR - 1), step = kMvThreads >> c_shift;
    for (int r0 = tid >> c_shift; r0 < n; r0 += step * kMvBatch) {
        uint4 k[kMvBatch], v[kMvBatch];
#pragma unroll
        for (int x = 0; x < kMvBatch; ++x) {
            const int r = r0 + x * step;
            if (r >= n || s_src[r] < 0) continue;
            k[x] = __ldcs(reinterpret_cast<const uint4*>(a.k_pages + s_src[r]) + c);
            v[x] = __ldcs(reinterpret_cast<const uint4*>(a.v_pages + s_src[r]) + c);
        }
#pragma unroll
        for (int x = 0; x < kMvBatch; ++x) {
            const int r = r0 + x * step;
            if (r >= n || s_src[r] < 0) continue;
            *(reinterpret_cast<uint4*>(a.k_pages + s_dst[r]) + c) = k[x];
            *(reinterpret_cast<uint4*>(a.v_pages + s_dst[r]) + c) = v[x];
            if (a.kmin != nullptr) s_rows[(r << c_shift) + c] = k[x];
        }
    }
    if (a.kmin == nullptr) return;
    __syncthreads();
    constexpr int EPL = KB ? 8 : 4;
    const int blks = (n + a.bs - 1) / a.bs, blk0 = t0 / a.bs;
    for (int it = tid; it < blks * CPR; it += kMvThreads) {
        const int j = it >> c_shift, cc = it & (CPR - 1), ra = j * a.bs, rb = min(n, ra + a.bs);
        float lo[EPL], hi[EPL];
#pragma unroll
        for (int e = 0; e < EPL; ++e) {
            lo[e] = INFINITY;
            hi[e] = -INFINITY;
        }
#pragma unroll 4
        for (int r = ra; r < rb; ++r) {
            if (s_src[r] < 0) continue;
            float f[EPL];
            unpack16<KB>(s_rows[(r << c_shift) + cc], f);
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                lo[e] = fminf(lo[e], f[e]);
                hi[e] = fmaxf(hi[e], f[e]);
            }
        }
        const long long box = (((long long)b * a.Hkv + kvh) * a.nb_cap + blk0 + j) * a.row_bytes + cc * 16;
        uint4* pmin = reinterpret_cast<uint4*>(a.kmin + box);
        uint4* pmax = reinterpret_cast<uint4*>(a.kmax + box);
        if constexpr (KB) {
            *pmin = make_uint4(pack_bf16x2(lo[0], lo[1]), pack_bf16x2(lo[2], lo[3]), pack_bf16x2(lo[4], lo[5]),
                               pack_bf16x2(lo[6], lo[7]));
            *pmax = make_uint4(pack_bf16x2(hi[0], hi[1]), pack_bf16x2(hi[2], hi[3]), pack_bf16x2(hi[4], hi[5]),
                               pack_bf16x2(hi[6], hi[7]));
        } else {
            *pmin = make_uint4(__float_as_uint(lo[0]), __float_as_uint(lo[1]), __float_as_uint(lo[2]), __float_as_uint(lo[3]));
            *pmax = make_uint4(__float_as_uint(hi[0]), __float_as_uint(hi[1]), __float_as_uint(hi[2]), __float_as_uint(hi[3]));
        }
    }
}

template <bool KB>
cudaError_t launch_move(const EvictArgs& a, unsigned grid, cudaStream_t s)
{
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(evict_move_kernel<KB>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 512);
    });
    if (cfg != cudaSuccess) return cfg;
    return launch_after_previous(evict_move_kernel<KB>, dim3(grid), dim3(kMvThreads),
                                 a.kmin != nullptr ? size_t(a.run) * a.row_bytes : 0, s, a);
}

}  // namespace

size_t evict_workspace(const Geometry& g, int keep) { return kTreeWsFree + size_t(g.units()) * keep * sizeof(float); }

cudaError_t launch_evict(const Geometry& g, const EvictCall& c, char* ws, cudaStream_t s)
{
    EvictArgs a{};
    a.seq_lens = c.seq_lens;
    a.keep_lens = c.keep_lens;
    a.block_table = c.block_table;
    a.new_table = c.new_table;
    a.weights = c.weights;
    a.kept_weights = reinterpret_cast<float*>(ws + kTreeWsFree);
    a.kept_ids = c.kept_ids;
    a.new_lens = c.new_lens;
    a.k_pages = static_cast<char*>(c.k_pages);
    a.v_pages = static_cast<char*>(c.v_pages);
    a.kmin = static_cast<char*>(c.kmin);
    a.kmax = static_cast<char*>(c.kmax);
    a.err = reinterpret_cast<uint32_t*>(ws);
    a.w_stride = (long long)g.nb_cap * g.bs;
    a.B = g.B;
    a.Hkv = g.Hkv;
    a.N = g.N;
    a.keep = c.keep;
    a.sinks = c.sinks;
    a.recent = c.recent;
    a.bs = g.bs;
    a.nb_cap = g.nb_cap;
    a.nb_new = (c.keep + g.bs - 1) / g.bs;
    a.num_pages = g.num_pages;
    a.row_bytes = g.D * (g.kv_bf16 ? 2 : 4);
    a.run = g.bs > kEvRun ? g.bs : kEvRun;
    // CTAs of a unit: as many as the SMs allow, each with some thousand tokens
    a.cluster = 1;
    while (a.cluster < kEvMaxCluster && 2LL * a.cluster * g.units() <= num_sms() && g.N / (2 * a.cluster) >= 2048) a.cluster *= 2;
    const int per = ((g.N + a.cluster - 1) / a.cluster + kEvThreads - 1) / kEvThreads * kEvThreads;
    a.cache = per < kEvCache ? per : kEvCache;
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvCache * 4);
    });
    if (cfg != cudaSuccess) return cfg;
    const cudaError_t e = launch_clusters_after_previous(evict_select_kernel, dim3(unsigned(g.units()) * unsigned(a.cluster)),
                                                         dim3(kEvThreads), size_t(a.cache) * 4, unsigned(a.cluster), s, a);
    if (e != cudaSuccess) return e;
    const unsigned grid = unsigned(g.units()) * unsigned((c.keep + a.run - 1) / a.run);
    return g.kv_bf16 ? launch_move<true>(a, grid, s) : launch_move<false>(a, grid, s);
}

}  // namespace sa
