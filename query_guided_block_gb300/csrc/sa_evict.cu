// Eviction from the paged cache by accumulated attention weight: for each (sequence, KV head) unit the
// first `sinks` tokens, the last `recent` ones and of the others those with the largest weights stay, in
// their order, in new pages.
//
// Two launches.  The first finds the kept tokens of a unit, by a thread-block cluster: the weights as
// keys of the same order, 32 bits, in shared memory; three histograms of 11, 11 and 10 bits, added up
// over the cluster, narrow the key of the last kept token down; tokens above it stay, of those equal to
// it as many as there is room for, lowest index first.  A kept token's place is the number of kept
// ones before it, which a scan over each warp's tokens gives.  The second launch moves rows: K and V of 64 kept
// tokens a CTA, every load on its way before the first store, with their weights and their blocks' box.
// Bytes: 4 a cached token, then each kept row once in and once out.
//
// 16 contexts of up to 32K tokens down to 8K, 8 heads of 128 (1.1 GB): 207 us, 5.3 TB/s; the first launch 26 us
// of it (loads with the first counts 10, digits 5, places 8), the second 179 of 162 for its bytes.  8 units of 128K
// tokens: 49 us, 26 in the first launch, by clusters of 8 (loads and first counts 6, digits 8: two barriers of
// the cluster and a round of remote reads each; places 6).  8 units of 8K tokens: 13.6 us, 10 in the first launch, a
// CTA a unit (lengths 1, loads and first counts 3, digits 3, places 3).  (Rows brought in by bulk copies of 256 bytes: 908 us,
// 65 ns a copy.)
#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kEvThreads = 1024;
constexpr int kEvWarps = kEvThreads / 32;   // a lane for each
constexpr int kEvCache = 47104;            // keys of a CTA in shared memory; the rest is read again
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

// Tokens of each of C CTAs: four to a lane and whole warps.
__host__ __device__ __forceinline__ int ev_slice(int n, int C)
{
    const int unit = 4 * kEvThreads;
    return ((n + C - 1) / C + unit - 1) / unit * unit;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__global__ void __launch_bounds__(kEvThreads, 1) evict_select_kernel(EvictArgs a)
{
    extern __shared__ __align__(16) uint32_t s_key[];
    __shared__ uint32_t s_hist[3][2048], s_sum[2048];         // of this CTA, of the cluster
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
    const int per = ev_slice(n, C);                            // tokens of a CTA
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
    auto make_key = [&](int i, float x) -> uint32_t {
        if (i < a.sinks || i >= n - a.recent) return 0xffffffffu;
        return min(order_key(x + 0.f), 0xfffffffeu);           // + 0: no negative zero
    };
    // Calls f(first index, its four keys) for this thread's tokens, four consecutive ones at a time (behind
    // i1: 0, below every key); the first time from memory into shared memory.
    auto each4 = [&](int from, int to, int stride, auto f) {
        for (int i = from; i < to; i += stride) {
            uint4 k;
            if (i - i0 + 4 <= a.cache) {
                k = *reinterpret_cast<const uint4*>(s_key + (i - i0));
            } else {
                const float4 x = *reinterpret_cast<const float4*>(w + i);
                k.x = make_key(i, x.x);
                k.y = i + 1 < i1 ? make_key(i + 1, x.y) : 0u;
                k.z = i + 2 < i1 ? make_key(i + 2, x.z) : 0u;
                k.w = i + 3 < i1 ? make_key(i + 3, x.w) : 0u;
            }
            f(i, k);
        }
    };
    // Counts one more of a digit; a warp's lanes that have its first lane's are counted together, so that many
    // equal weights (zeros) do not queue up.
    auto count = [&](uint32_t* hist, bool have, uint32_t digit) {
        const uint32_t live = __ballot_sync(kFullMask, have);
        if (live == 0u) return;
        const int lead = __ffs(live) - 1;
        const uint32_t first = __shfl_sync(kFullMask, digit, lead);
        const uint32_t same = __ballot_sync(kFullMask, have && digit == first);
        if (lane == lead) atomicAdd(&hist[first], uint32_t(__popc(same)));
        else if (have && digit != first) atomicAdd(&hist[digit], 1u);
    };

    for (int i = tid; i < 3 * 2048; i += kEvThreads) (&s_hist[0][0])[i] = 0u;
    __syncthreads();
    constexpr int LOADS = 4;                                   // 16-byte loads a thread has on their way
    for (int base = i0; base < i1; base += 4 * kEvThreads * LOADS) {
        float4 x[LOADS];
#pragma unroll
        for (int y = 0; y < LOADS; ++y) {
            const int i = base + 4 * (y * kEvThreads + tid);
            if (i < i1) x[y] = *reinterpret_cast<const float4*>(w + i);      // the row goes on to a multiple of 8
        }
#pragma unroll
        for (int y = 0; y < LOADS; ++y) {
            const int i = base + 4 * (y * kEvThreads + tid);
            const float e[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
            uint32_t k[4];
#pragma unroll
            for (int z = 0; z < 4; ++z) {
                k[z] = i + z < i1 ? make_key(i + z, e[z]) : 0u;
                count(s_hist[0], i + z < i1, k[z] >> 21);
            }
            if (i < i1 && i - i0 + 4 <= a.cache) *reinterpret_cast<uint4*>(s_key + (i - i0)) = make_uint4(k[0], k[1], k[2], k[3]);
        }
    }
    uint32_t prefix = 0u;                                      // the last kept key's bits so far
    uint32_t room = uint32_t(kept);                            // tokens to take among those with these bits
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        if (pass > 0) {
            const int above = pass == 1 ? 21 : 10;
            each4(i0 + 4 * tid, i1, 4 * kEvThreads, [&](int i, uint4 k) {
                const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (i + z < i1 && (e[z] >> above) == (prefix >> above))
                        atomicAdd(&s_hist[pass][(e[z] >> shift) & (pass == 1 ? 2047u : 1023u)], 1u);
            });
        }
        if (C > 1) cluster_sync_all();
        else __syncthreads();
        const uint32_t* totals = s_hist[pass];
        if (C > 1) {                                           // every CTA adds up its share of the bins and tells the others
            const int share = 2048 / C;
            for (int x = tid; x < share; x += kEvThreads) {
                const int bin = rank * share + x;
                const uint32_t at = smem_u32(&s_hist[pass][bin]), to = smem_u32(&s_sum[bin]);
                uint32_t of[kEvMaxCluster], all = 0u;
#pragma unroll
                for (int r = 0; r < kEvMaxCluster; ++r) of[r] = ld_cluster_u32(cluster_map(at, uint32_t(r < C ? r : rank)));
#pragma unroll
                for (int r = 0; r < kEvMaxCluster; ++r) all += r < C ? of[r] : 0u;
                for (int r = 0; r < C; ++r) st_cluster_u32(cluster_map(to, uint32_t(r)), all);
            }
            cluster_sync_all();
            totals = s_sum;                                    // read before the next pass's first barrier
        }
        // from the largest digit down, two to a thread
        uint32_t h[2], sum = 0u;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            h[x] = totals[2047 - 2 * tid - x];
            sum += h[x];
        }
        const uint32_t incl = uint32_t(warp_inclusive_scan(int(sum), lane));
        if (lane == 31) s_warp[0][warp] = int(incl);
        __syncthreads();
        const uint32_t at_warp = __reduce_add_sync(kFullMask, lane < warp ? uint32_t(s_warp[0][lane]) : 0u);
        uint32_t at = at_warp + incl - sum;
        if (at < room && room <= at + sum) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                if (at < room && room <= at + h[x]) {
                    s_found[0] = uint32_t(2047 - 2 * tid - x);
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
    each4(w0 + 4 * lane, w1, 128, [&](int i, uint4 k) {
        const uint32_t e[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            gt += i + z < w1 && e[z] > prefix;
            eq += i + z < w1 && e[z] == prefix;
        }
    });
    gt = __reduce_add_sync(kFullMask, gt);
    eq = __reduce_add_sync(kFullMask, eq);
    if (lane == 0) {
        s_warp[0][warp] = gt;
        s_warp[1][warp] = eq;
    }
    __syncthreads();
    if (warp < 2) {
        const uint32_t all = __reduce_add_sync(kFullMask, uint32_t(s_warp[warp][lane]));
        if (lane == 0) s_total[warp] = all;
    }
    if (C > 1) cluster_sync_all();
    else __syncthreads();
    uint32_t gt_at = lane < warp ? uint32_t(s_warp[0][lane]) : 0u, eq_at = lane < warp ? uint32_t(s_warp[1][lane]) : 0u;
    if (lane < rank) {                                         // the CTAs before this one
        gt_at += ld_cluster_u32(cluster_map(smem_u32(&s_total[0]), uint32_t(lane)));
        eq_at += ld_cluster_u32(cluster_map(smem_u32(&s_total[1]), uint32_t(lane)));
    }
    gt_at = __reduce_add_sync(kFullMask, gt_at);
    eq_at = __reduce_add_sync(kFullMask, eq_at);
    for (int base = w0; base < w1; base += 128) {              // four consecutive tokens a lane
        uint4 k4 = make_uint4(0u, 0u, 0u, 0u);
        const int i = base + 4 * lane;
        each4(i, min(w1, i + 1), 4, [&](int, uint4 k) { k4 = k; });
        const uint32_t e[4] = {k4.x, k4.y, k4.z, k4.w};
        int more = 0, equal = 0;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            more += i + z < w1 && e[z] > prefix;
            equal += i + z < w1 && e[z] == prefix;
        }
        const int both = warp_inclusive_scan(more << 16 | equal, lane);
        const int all = __shfl_sync(kFullMask, both, 31);
        uint32_t g = gt_at + (both >> 16) - more, q = eq_at + (both & 0xffff) - equal;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            if (i + z >= w1) break;
            const bool is_gt = e[z] > prefix, is_eq = e[z] == prefix;
            if (is_gt || (is_eq && q < room)) {
                const uint32_t pos = g + min(q, room);
                ids[pos] = i + z;
                // the weight, from its key; of those that stay in any case from memory
                vals[pos] = e[z] == 0xffffffffu ? w[i + z] : __uint_as_float((e[z] & 0x80000000u) ? e[z] ^ 0x80000000u : ~e[z]);
            }
            g += is_gt;
            q += is_eq;
        }
        gt_at += uint32_t(all >> 16);
        eq_at += uint32_t(all & 0xffff);
    }
    if (C > 1) cluster_sync_all();                             // others may still read this CTA's totals
}

// The minimum and maximum of 16 bytes of channels over rows.
template <bool KB>
struct Box {
    static constexpr int N = KB ? 8 : 4;
    float lo[N], hi[N];
    __device__ __forceinline__ Box()
    {
#pragma unroll
        for (int e = 0; e < N; ++e) {
            lo[e] = INFINITY;
            hi[e] = -INFINITY;
        }
    }
    __device__ __forceinline__ void join(const uint4& low, const uint4& high)
    {
        float f[N], g[N];
        unpack16<KB>(low, f);
        unpack16<KB>(high, g);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            lo[e] = fminf(lo[e], f[e]);
            hi[e] = fmaxf(hi[e], g[e]);
        }
    }
    __device__ __forceinline__ void join(const uint4& v) { join(v, v); }
    static __device__ __forceinline__ uint4 stored(const float (&f)[N])
    {
        if constexpr (KB)
            return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        else
            return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
    __device__ __forceinline__ uint4 low() const { return stored(lo); }
    __device__ __forceinline__ uint4 high() const { return stored(hi); }
};

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
    // The box: of eight rows a thread, then of a block's eights.  (A thread for all 64 rows of a block: 205 us
    // for 16 x 8K tokens of 8 heads, so 179, 162 without a box.)
    __syncthreads();
    uint4* s_part = s_rows + (a.run << c_shift);               // [eight][chunk][lowest, highest]
    for (int it = tid; it < (n + 7) / 8 * CPR; it += kMvThreads) {
        const int ra = (it >> c_shift) * 8, rb = min(n, ra + 8);
        Box<KB> box;
        for (int r = ra; r < rb; ++r)
            if (s_src[r] >= 0) box.join(s_rows[(r << c_shift) + (it & (CPR - 1))]);
        s_part[2 * it] = box.low();
        s_part[2 * it + 1] = box.high();
    }
    __syncthreads();
    const int blks = (n + a.bs - 1) / a.bs, blk0 = t0 / a.bs;
    for (int it = tid; it < blks * CPR; it += kMvThreads) {
        const int j = it >> c_shift, cc = it & (CPR - 1), ea = j * a.bs / 8, eb = (min(n, (j + 1) * a.bs) + 7) / 8;
        Box<KB> box;
        for (int e = ea; e < eb; ++e) box.join(s_part[2 * ((e << c_shift) + cc)], s_part[2 * ((e << c_shift) + cc) + 1]);
        const long long at = ((long long)u * a.nb_cap + blk0 + j) * a.row_bytes + cc * 16;
        *reinterpret_cast<uint4*>(a.kmin + at) = box.low();
        *reinterpret_cast<uint4*>(a.kmax + at) = box.high();
    }
}

template <bool KB>
cudaError_t launch_move(const EvictArgs& a, unsigned grid, cudaStream_t s)
{
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(evict_move_kernel<KB>, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 * 512 * 5 / 4);
    });
    if (cfg != cudaSuccess) return cfg;
    return launch_after_previous(evict_move_kernel<KB>, dim3(grid), dim3(kMvThreads),
                                 a.kmin != nullptr ? size_t(a.run) * a.row_bytes * 5 / 4 : 0, s, a);
}

// Behind an eviction: the page table, the lengths and the weights of the sequences that moved.  The first launch counts
// for each page the contexts that read it and writes down which sequences moved, from the old lengths; the
// second overwrites them.  The counts are in a hash table, whose size goes by the page table's and not by the
// pool's, with open addressing: it is half empty at least, so a search ends.  Bytes: the page table twice, the hash
// table, the weights behind the kept tokens once.  Up to 64 contexts 5 to 8 us, which are the three steps' starts; 256 x
// 32K tokens of 8 heads (235 MB of zeros) 46 us, the zeros' time (a CTA a row of weights: one context of 128K 11.7 us
// for 5.2).
constexpr int kAdThreads = 256;
constexpr int kAdRun = 4096;               // weights of a CTA at a time

struct Reader {
    int page;              // -1: free
    int count;             // contexts that read it, less one
};

struct AdoptArgs {
    AdoptCall c;
    Reader* readers;                       // [2^readers_log2], all bits set before
    int32_t *was, *moved;                  // [B] old length (-1: no context), [B]
    long long w_stride;
    int B, Hkv, N, bs, nb_cap, num_pages, table_ctas, w_runs, readers_log2;
};

__device__ __forceinline__ unsigned reader_place(const AdoptArgs& a, int page)
{
    return (unsigned(page) * 2654435769u) >> (32 - a.readers_log2);        // 2^32 over the golden ratio
}

__global__ void __launch_bounds__(kAdThreads) adopt_count_kernel(AdoptArgs a)
{
    allow_dependents_early();
    grid_dependency_wait();   // lengths and pages may come from the previous kernel
    const long long entries = (long long)a.B * a.nb_cap, step = (long long)gridDim.x * kAdThreads;
    for (long long i = (long long)blockIdx.x * kAdThreads + threadIdx.x; i < entries; i += step) {
        const int b = int(i / a.nb_cap), j = int(i - (long long)b * a.nb_cap), len = a.c.seq_lens[b];
        const bool active = len >= 0 && len <= a.N;
        if (j == 0) {
            const int k = a.c.keep_lens != nullptr ? a.c.keep_lens[b] : a.c.keep;
            a.was[b] = active ? len : -1;
            a.moved[b] = active && k >= a.c.sinks + a.c.recent && k <= a.c.keep;
        }
        if (!active || (long long)j * a.bs >= len) continue;
        const int page = a.c.block_table[i];
        if (page < 0 || page >= a.num_pages) continue;
        const unsigned size = 1u << a.readers_log2;
        unsigned at = reader_place(a, page);
        for (unsigned n = 0; n < size; ++n, at = (at + 1) & (size - 1)) {
            const int there = atomicCAS(&a.readers[at].page, -1, page);
            if (there != -1 && there != page) continue;
            atomicAdd(&a.readers[at].count, 1);
            break;
        }
    }
}

// The first table_ctas CTAs write the table and the lengths, the others the weights.
__global__ void __launch_bounds__(kAdThreads) adopt_kernel(AdoptArgs a)
{
    allow_dependents_early();
    grid_dependency_wait();   // counts and old lengths come from the previous kernel
    const int tid = threadIdx.x;
    if (int(blockIdx.x) >= a.table_ctas) {
        const int first = int(blockIdx.x) - a.table_ctas, ctas = int(gridDim.x) - a.table_ctas;
        for (long long it = first; it < (long long)a.B * a.Hkv * a.w_runs; it += ctas) {
            const int u = int(it / a.w_runs), t0 = int(it - (long long)u * a.w_runs) * kAdRun, b = u / a.Hkv;
            if (a.moved[b] == 0) continue;
            float* w = a.c.weights + u * a.w_stride;           // a row is whole 16 bytes
            const int from = max(t0, a.c.new_lens[b]), to = min(int(a.w_stride), t0 + kAdRun), up = min((from + 3) & ~3, to);
            if (tid < up - from) w[from + tid] = 0.f;
            for (int t = up + 4 * tid; t < to; t += 4 * kAdThreads) *reinterpret_cast<float4*>(w + t) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        return;
    }
    auto readers = [&](int page) {
        const unsigned size = 1u << a.readers_log2;
        unsigned at = reader_place(a, page);
        for (unsigned n = 0; n < size && a.readers[at].page != -1; ++n, at = (at + 1) & (size - 1))
            if (a.readers[at].page == page) return a.readers[at].count + 1;
        return 0;
    };
    const long long entries = (long long)a.B * a.nb_cap, step = (long long)a.table_ctas * kAdThreads;
    for (long long i = (long long)blockIdx.x * kAdThreads + tid; i < entries; i += step) {
        const int b = int(i / a.nb_cap), j = int(i - (long long)b * a.nb_cap);
        if (a.moved[b] == 0) continue;
        if (j == 0) a.c.seq_lens[b] = a.c.new_lens[b];
        if (j < a.c.new_width) {
            a.c.block_table[i] = a.c.new_table[(long long)b * a.c.new_width + j];
        } else {
            const int page = a.c.block_table[i], own = (long long)j * a.bs < a.was[b];
            if (page >= 0 && page < a.num_pages && readers(page) > own) a.c.block_table[i] = -1;
        }
    }
}

struct EvictLayout {
    size_t kept_weights, readers, was, moved, end;
    int readers_log2;
};

EvictLayout evict_layout(const Geometry& g, int keep)
{
    auto align256 = [](size_t x) { return (x + 255) & ~size_t(255); };
    EvictLayout L{};
    L.kept_weights = kTreeWsFree;
    L.readers = align256(L.kept_weights + size_t(g.units()) * keep * sizeof(float));
    L.readers_log2 = 1;
    while ((1LL << L.readers_log2) < 2LL * g.B * g.nb_cap) ++L.readers_log2;
    L.was = L.readers + align256((sizeof(Reader)) << L.readers_log2);
    L.moved = L.was + align256(size_t(g.B) * sizeof(int32_t));
    L.end = L.moved + align256(size_t(g.B) * sizeof(int32_t));
    return L;
}

}  // namespace

size_t evict_workspace(const Geometry& g, int keep) { return evict_layout(g, keep).end; }

cudaError_t launch_adopt(const Geometry& g, const AdoptCall& c, char* ws, cudaStream_t s)
{
    const EvictLayout L = evict_layout(g, c.keep);
    AdoptArgs a{};
    a.c = c;
    a.readers = reinterpret_cast<Reader*>(ws + L.readers);
    a.readers_log2 = L.readers_log2;
    a.was = reinterpret_cast<int32_t*>(ws + L.was);
    a.moved = reinterpret_cast<int32_t*>(ws + L.moved);
    a.w_stride = (long long)g.nb_cap * g.bs;
    a.B = g.B;
    a.Hkv = g.Hkv;
    a.N = g.N;
    a.bs = g.bs;
    a.nb_cap = g.nb_cap;
    a.num_pages = g.num_pages;
    const long long entries = (long long)g.B * g.nb_cap, ctas = (entries + kAdThreads - 1) / kAdThreads, most = 4LL * num_sms();
    a.table_ctas = int(ctas < most ? ctas : most);
    a.w_runs = int((a.w_stride + kAdRun - 1) / kAdRun);
    const long long runs = (long long)g.units() * a.w_runs;
    const int weight_ctas = c.weights == nullptr ? 0 : int(runs < most ? runs : most);
    cudaError_t e = cudaMemsetAsync(a.readers, 0xff, sizeof(Reader) << L.readers_log2, s);
    if (e != cudaSuccess) return e;
    e = launch_after_previous(adopt_count_kernel, dim3(unsigned(a.table_ctas)), dim3(kAdThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_after_previous(adopt_kernel, dim3(unsigned(a.table_ctas + weight_ctas)), dim3(kAdThreads), 0, s, a);
}

cudaError_t launch_evict(const Geometry& g, const EvictCall& c, char* ws, cudaStream_t s)
{
    EvictArgs a{};
    a.seq_lens = c.seq_lens;
    a.keep_lens = c.keep_lens;
    a.block_table = c.block_table;
    a.new_table = c.new_table;
    a.weights = c.weights;
    a.kept_weights = reinterpret_cast<float*>(ws + evict_layout(g, c.keep).kept_weights);
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
    // CTAs of a unit: one up to 16K tokens, beyond that as many as the SMs allow, each with 4096 at least.  8 units
    // of 8K tokens: one CTA 10.0 us, two 12.9; of 16K: 14.7, four 14.2; of 32K: 25, eight 14.5; of 128K: 111, eight 26.
    a.cluster = 1;
    while (g.N > 16384 && a.cluster < kEvMaxCluster && 2LL * a.cluster * g.units() <= num_sms() && g.N / (2 * a.cluster) >= 4096)
        a.cluster *= 2;
    const int per = ev_slice(g.N, a.cluster);
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
