// The sums of attention weights on the fifth-generation tensor cores (bf16, many query rows): the scores
// are computed again instead of kept, which costs the keys once more (2 D bytes a token) where 4 bytes a
// row and token written and read would be several times that.
//
// Per tile of 128 tokens: S^T = K Q^T (tcgen05.mma, M = the tile's tokens, N = up to 256 query rows), so that a
// thread owns a token and adds up exp2((s - m_r) scale) / l_r over the rows r in registers, the rows' maxima and
// reciprocal totals being broadcast from shared memory.  Four groups of four warps take a quarter of the rows
// each; their sums meet in shared memory.  Rows past 256 are further passes over the same tiles.
//
// Roles: warps 0-15 the sums, warp 16 resolves pages and brings K by TMA into a ring, warp 17 issues the
// products into one of two score tiles in tensor memory.  No wait is without a limit.
#include "sa_tree_tc_kernel.cuh"

namespace sa {
namespace {

constexpr int kWtGroups = 4;             // of four warps, each with a quarter of the rows
constexpr int kWtSum = 128 * kWtGroups;
constexpr int kWtThreads = kWtSum + 64;
constexpr int kWtRows = 256;               // query rows of a pass

template <int D>
struct WtShape {
    static constexpr int HALVES = D / 64;
    static constexpr int HALF = kTcTile * 128;              // 128 tokens x 64 bf16
    static constexpr int UNIT = HALVES * HALF;
    static constexpr int Q_HALF = kWtRows * 128;
    static constexpr int Q_TILE = HALVES * Q_HALF;
    static constexpr int STAGES = D == 128 ? 4 : 8;
    // Tiles whose entries are remembered: the producer is at most STAGES tiles past the last one whose product
    // is done, and the sums are at most two behind that.
    static constexpr int INFO = STAGES + 4;
    static constexpr int OFF_RING = Q_TILE;
    static constexpr int OFF_SHARED = OFF_RING + STAGES * UNIT;
};

template <int D>
struct WtShared {
    uint64_t full[WtShape<D>::STAGES], empty[WtShape<D>::STAGES], s_full[2], s_read[2];
    float m[kWtRows], inv[kWtRows];             // of the pass's rows
    float part[2][kWtGroups - 1][kTcTile];      // sums of the groups behind the first, tile mod 2
    int scan[kTreeScan<kWtThreads>];
    uint32_t pages[WtShape<D>::INFO];           // entries of a tile that have a page
    uint32_t tmem;
    int dead;                                   // a bounded wait ran out: no more waiting
};
template <int D>
constexpr size_t wt_smem()
{
    static_assert(WtShape<D>::OFF_SHARED + sizeof(WtShared<D>) <= 227 * 1024, "shared memory of a CTA");
    return WtShape<D>::OFF_SHARED + sizeof(WtShared<D>);
}

template <int D>
__global__ void __launch_bounds__(kWtThreads, 1)
    weigh_tc_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ CUtensorMap kmap, const float2* stats,
                    float* weights, long long w_stride)
{
    using SH = WtShape<D>;
    extern __shared__ __align__(1024) unsigned char smem[];        // swizzle atoms: 1024-byte aligned
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_u32(smem);
    WtShared<D>& sh = *reinterpret_cast<WtShared<D>*>(smem + SH::OFF_SHARED);
    if ((base & 1023u) != 0u) {                                    // the alignment above is not kept: no result
        if (tid == 0) raise_error(a.err, SPARSE_ATTN_ERR_CAPACITY);
        return;
    }
    allow_dependents_early();
    if (warp == 0) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < SH::STAGES; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.s_read[s], kWtSum);
        }
        sh.dead = 0;
        fence_mbar_init();
    }
    grid_dependency_wait();   // totals, weights, queries and pages may come from previous kernels
    tc_fence_before_sync();
    const TreePart part = tree_part<kWtThreads, true>(a, sh.scan);  // synchronises the CTA
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const int passes = (a.R + kWtRows - 1) / kWtRows;
    int lo = part.lo, start = part.start, item = part.item;
    uint32_t tile0 = 0;                                            // tiles of earlier passes
    TcSegment g;

    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return;
        if (*reinterpret_cast<volatile int*>(&sh.dead) != 0) return;
        if (!mbar_wait_bounded(bar, parity, kWaitCycles)) {
            *reinterpret_cast<volatile int*>(&sh.dead) = 1;
            raise_error(a.err, SPARSE_ATTN_ERR_TIMEOUT);
        }
    };
    // columns of a pass: its rows, whole 16s for each group of warps
    auto columns = [&](int pass) { return (min(kWtRows, a.R - pass * kWtRows) + 16 * kWtGroups - 1) / (16 * kWtGroups) * (16 * kWtGroups); };

    while (tc_next<true>(a, part, lo, start, item, g)) {
        const int ntl = g.t1 - g.t0;
        for (int pass = 0; pass < passes; ++pass, tile0 += ntl) {
            if (warp == kWtSum / 32) {
                // ---- producer -----------------------------------------------------------------
                const int n_e = a.bs >= kTcTile ? 1 : kTcTile >> a.bs_shift;   // entries of a tile
                const int per_batch = 32 / n_e;                    // tiles whose entries one batch holds
                const int e_base = (g.t0 * kTcTile) >> a.bs_shift;
                auto resolve = [&](int batch) -> int {
                    const int e = e_base + batch * 32 + lane;
                    return e < g.un.n_entries && batch * 32 + lane < ntl * n_e ? tree_entry<true>(a, g.u, g.un, e).x : -1;
                };
                int cur = resolve(0), nxt = resolve(1);
                for (int i = 0; i < ntl; ++i) {
                    const int at = i % per_batch;
                    if (i > 0 && at == 0) {
                        cur = nxt;
                        nxt = resolve(i / per_batch + 1);
                    }
                    const int page = __shfl_sync(kFullMask, cur, (at * n_e + lane) & 31);
                    const uint32_t ok = __ballot_sync(kFullMask, lane < n_e && page >= 0);
                    const uint32_t n = tile0 + i, st = n % SH::STAGES;
                    if (n >= SH::STAGES) wait(&sh.empty[st], (n / SH::STAGES - 1) & 1u);
                    // start no more copies; the warp decides together
                    if (__any_sync(kFullMask, *reinterpret_cast<volatile int*>(&sh.dead) != 0)) continue;
                    if (lane == 0) {
                        sh.pages[n % SH::INFO] = ok;               // before the arrival that the sums wait for, through the product
                        mbar_arrive_expect_tx(&sh.full[st], __popc(ok) * uint32_t(a.bs * 128 * SH::HALVES));
                    }
                    __syncwarp();
                    if (lane < n_e && page >= 0) {
                        const uint32_t dst = base + SH::OFF_RING + st * SH::UNIT + lane * a.bs * 128;
#pragma unroll
                        for (int h = 0; h < SH::HALVES; ++h) tma_load_3d(dst + h * SH::HALF, &kmap, h * 64, 0, page, &sh.full[st]);
                    }
                }
            } else if (warp == kWtSum / 32 + 1) {
                // ---- scores -------------------------------------------------------------------
                bar_sync(1, kWtSum + 32);                          // queries staged
                if (lane == 0) {
                    const uint32_t idesc = idesc_bf16_f32(kTcTile, columns(pass), false);
                    const uint64_t q_desc = smem_desc_sw128(base, 16, 1024);
                    const uint64_t k_desc0 = smem_desc_sw128(base + SH::OFF_RING, 16, 1024);
                    for (int i = 0; i < ntl; ++i) {
                        const uint32_t n = tile0 + i, s = n & 1u, st = n % SH::STAGES;
                        if (n >= 2) wait(&sh.s_read[s], ((n - 2) >> 1) & 1u);
                        wait(&sh.full[st], (n / SH::STAGES) & 1u);
                        tc_fence_after_sync();
                        const uint64_t kd = k_desc0 + uint64_t((st * SH::UNIT) >> 4);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k)
                            umma_bf16(tmem + s * kWtRows, kd + uint32_t(((k >> 2) * SH::HALF + (k & 3) * 32) >> 4),
                                      q_desc + uint32_t(((k >> 2) * SH::Q_HALF + (k & 3) * 32) >> 4), idesc, k > 0 ? 1u : 0u);
                        umma_commit(&sh.s_full[s]);
                        umma_commit(&sh.empty[st]);
                    }
                }
                __syncwarp();
            } else {
                // ---- the sums: thread = token, group = a quarter of the rows -----------------------------
                const int cols = columns(pass), rows = min(kWtRows, a.R - pass * kWtRows);
                {
                    constexpr int CPR = D / 8;                     // 16-byte chunks of a row
                    bar_sync(2, kWtSum);                           // the pass before is done with the queries and totals
                    for (int i = tid; i < cols * CPR; i += kWtSum) {
                        const int r = i / CPR, c = i % CPR;
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (r < rows)
                            v = *(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                 tree_out_row(a, g.b, g.kvh, pass * kWtRows + r) * D) + c);
                        *reinterpret_cast<uint4*>(smem + (c >> 3) * SH::Q_HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
                    }
                    if (tid < cols) {                              // a row without a total weighs nothing: exp2(-inf)
                        const float2 st = tid < rows ? stats[tree_out_row(a, g.b, g.kvh, pass * kWtRows + tid)]
                                                     : make_float2(0.f, 0.f);
                        sh.m[tid] = st.y != 0.f ? -st.x : -INFINITY;
                        sh.inv[tid] = st.y;
                    }
                    fence_proxy_async_smem();                      // before the tensor core uses this memory
                }
                bar_sync(1, kWtSum + 32);
                const int h = warp >> 2, token = 32 * (warp & 3) + lane;
                const int c0 = h * (cols / kWtGroups), c1 = c0 + cols / kWtGroups;
                const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
                const F2 scale2 = make_f2(a.scale_log2, a.scale_log2);
                for (int i = 0; i < ntl; ++i) {
                    const uint32_t n = tile0 + i, s = n & 1u;
                    const int t = (g.t0 + i) * kTcTile + token;
                    float* w = weights + g.u * w_stride + t;
                    float old = 0.f;
                    if (h == 0 && t < g.un.len + (pass > 0 ? a.Q : 0)) old = *w;
                    wait(&sh.s_full[s], (n >> 1) & 1u);
                    __syncwarp();
                    tc_fence_after_sync();
                    // query rows from `first` on see the token
                    const bool there = (sh.pages[n % SH::INFO] >> (token >> a.bs_shift)) & 1u;
                    const int first = !there || t >= g.un.len + a.Q ? INT32_MAX : max(0, t - g.un.len) * a.G - pass * kWtRows;
                    const bool all = (__all_sync(kFullMask, first <= 0)) != 0;
                    F2 sum_a = make_f2(0.f, 0.f), sum_b = make_f2(0.f, 0.f);
                    for (int c = c0; c < c1; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(tmem + s * kWtRows + c + lanes, v);
                        tmem_wait_ld16(v);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 m = *reinterpret_cast<const float4*>(sh.m + c + j);
                            const float4 l = *reinterpret_cast<const float4*>(sh.inv + c + j);
                            F2 x = mul2(add2(make_f2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), make_f2(m.x, m.y)), scale2);
                            F2 y = mul2(add2(make_f2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), make_f2(m.z, m.w)), scale2);
                            x = make_f2(fast_exp2(x.f.x), fast_exp2(x.f.y));
                            y = make_f2(fast_exp2(y.f.x), fast_exp2(y.f.y));
                            if (!all) {
                                if (c + j < first) x.f.x = 0.f;
                                if (c + j + 1 < first) x.f.y = 0.f;
                                if (c + j + 2 < first) y.f.x = 0.f;
                                if (c + j + 3 < first) y.f.y = 0.f;
                            }
                            sum_a = fma2(x, make_f2(l.x, l.y), sum_a);
                            sum_b = fma2(y, make_f2(l.z, l.w), sum_b);
                        }
                    }
                    tc_fence_before_sync();
                    mbar_arrive(&sh.s_read[s]);
                    const F2 sum2 = add2(sum_a, sum_b);
                    float sum = sum2.f.x + sum2.f.y;
                    if (h > 0) sh.part[s][h - 1][token] = sum;
                    bar_sync(2, kWtSum);
                    if (h == 0 && t < g.un.len + a.Q) {
#pragma unroll
                        for (int x = 0; x < kWtGroups - 1; ++x) sum += sh.part[s][x][token];
                        *w = old + sum;
                    }
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    if (sh.dead != 0) {
        // a wait ran out: leave copies that may still be on their way the time to land
        const long long t = clock64();
        while (clock64() - t < 4000000LL) {
        }
    }
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch_t(const TreeArgs& a, const float2* stats, float* weights, long long w_stride, cudaStream_t s)
{
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(weigh_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(wt_smem<D>()));
    });
    if (cfg != cudaSuccess) return cfg;
    CUtensorMap kmap;
    const cudaError_t e = encode_tree_map(&kmap, a.k_pages, D, a.bs, (long long)a.num_pages * a.Hkv);
    if (e != cudaSuccess) return e;
    const int ctas = num_sms() < kTreeMaxCtas ? num_sms() : kTreeMaxCtas;
    return launch_after_previous(weigh_tc_kernel<D>, dim3(unsigned(ctas)), dim3(kWtThreads), wt_smem<D>(), s, a, kmap, stats,
                                 weights, w_stride);
}

}  // namespace

cudaError_t launch_weigh_tc(TreeArgs a, const float2* stats, float* weights, long long w_stride, cudaStream_t s)
{
    a.tile = kTcTile;
    a.item_rows = a.R;             // an item is a unit
    a.row_groups = 1;
    a.min_per = 1;
    a.half_slack = 1;
    return a.D == 128 ? launch_t<128>(a, stats, weights, w_stride, s) : launch_t<64>(a, stats, weights, w_stride, s);
}

}  // namespace sa
