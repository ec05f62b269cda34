// Draft-tree attention on the fifth-generation tensor cores (bf16 queries and K/V).
//
// A CTA holds one or two tiles of 128 query rows of a (sequence, KV head) unit and walks the
// unit's list (sa_tree.cuh) in tiles of 128 tokens.  Two slots work side by side, each with a
// score tile and an output tile in tensor memory (all 512 columns) and a warpgroup of its own:
// with one row tile the slots take the even and the odd token tiles (their results are joined
// at the item's end), with two row tiles each slot keeps one of them and both use every K/V
// tile.  While one slot's softmax runs, the other's products keep the tensor core busy.
//
// Roles (12 warps):
//   warp 8      resolves the list's entries 32 at a time and brings K and V by TMA, one box
//               of 64 channels x one block per entry and channel half, into a ring of K and
//               V units that it refills as the products release them;
//   warps 9, 10 one thread each: S = Q K^T, then O = P V for one slot (tcgen05.mma);
//   warps 0-3, 4-7  the slots' softmax: a thread owns one query row.  Reads S, takes the
//               maximum, writes P, then adds the finished O tile to its row in registers.
//
// Precision.  The output is fp32, so P goes into the product as three bf16 parts that hold
// its 24 bits exactly: two of them overwrite S in tensor memory (A operands there), the third
// goes through shared memory.  The tensor core rounds its running sum toward zero at every
// step (measured: the drift of a sum kept over 8K tokens is 1e-5), so O starts from zero in
// every tile and the rows add it up in registers by one FMA, which carries the softmax's
// rescaling as well.
//
// Per 128 tokens and row tile the tensor core does 4 x 128 x 128 x D multiply-adds (one for S,
// three for P V), about 2050 cycles at D = 128; the 64 KB of K and V arrive in about 2800
// cycles at the SM's share of the HBM bandwidth, so one row tile is bound by memory and
// two row tiles by the tensor core.
#include "sa_tcgen05.cuh"
#include "sa_tree.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

namespace sa {
namespace {

constexpr int kTcThreads = 384;
constexpr int kTcTile = 128;
constexpr int kTcInfo = 8;           // tiles whose entries are remembered (more than the ring holds)
constexpr int kNoToken = INT32_MIN;

template <int D, int RT>
struct TcShape {
    static constexpr int HALVES = D / 64;
    static constexpr int HALF = kTcTile * 128;              // 128 rows x 64 bf16
    static constexpr int UNIT = HALVES * HALF;              // K or V of a tile
    static constexpr int Q_TILE = HALVES * HALF;
    static constexpr int P_TILE = 2 * HALF;                 // 128 rows x 128 tokens
    static constexpr int UNITS = D == 128 ? (RT == 1 ? 4 : 3) : 8;
    static constexpr int OFF_P = RT * Q_TILE;
    static constexpr int OFF_RING = OFF_P + 2 * P_TILE;
    static constexpr size_t SMEM = 1024 + size_t(OFF_RING) + size_t(UNITS) * UNIT;
    static_assert(SMEM <= 227 * 1024 - 2000, "dynamic and static shared memory of one CTA");
    static_assert(size_t(UNITS) * UNIT >= size_t(kTcTile) * D * 4, "the joined rows go through the ring");
};

__device__ __forceinline__ void bar_sync(int id, int threads)
{
    __syncwarp();
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// D (tensor memory) = A (tensor memory) * B (+ D when accumulate != 0).
__device__ __forceinline__ void umma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr)
{
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
    return r;
}

// A pair of fp32 cut to bf16 (the upper halves of the words; the first in the low half), the
// remainders left behind.
__device__ __forceinline__ uint32_t cut_bf16x2(float& x, float& y)
{
    const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
    x -= __uint_as_float(ux & 0xffff0000u);
    y -= __uint_as_float(uy & 0xffff0000u);
    return __byte_perm(ux, uy, 0x7632);
}

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

// Register shares: the CTA starts with 12 warps x 168; the softmax threads hold an output row.
constexpr int kTcRegsFew = 88, kTcRegsMany = 208;
static_assert(kTcRegsFew * 128 + kTcRegsMany * 256 <= 168 * kTcThreads, "no more registers than the launch got");

struct TcShared {
    uint64_t full[8], empty[8], s_full[2], o_full[2], p_ready[2];
    uint32_t tmem;
    int dead;                                   // a bounded wait ran out: no more waiting
    int last;
    uint32_t bad[2][4];
    uint32_t any[kTreeMaxDrafts / 32];
    int2 entry[kTcInfo][16];
    int masked[kTcInfo];
};

// One item's share of this CTA's part: tiles [t0, t1) of the item's list.
struct TcSegment {
    int u, b, kvh, item, row0, t0, t1, tiles;
    long long start;
    TreeUnit un;
};

__device__ __forceinline__ bool tc_next(const TreeArgs& a, const TreePart& part, long long& lo, long long& start,
                                        int& item, TcSegment& g)
{
    while (lo < part.hi) {
        g.u = item / a.row_groups;
        g.un = tree_unit(a, g.u);
        g.tiles = tree_tiles(a, g.un);
        if (g.tiles == 0) {
            ++item;
            continue;
        }
        g.b = g.u / a.Hkv;
        g.kvh = g.u - g.b * a.Hkv;
        g.item = item;
        g.row0 = (item - g.u * a.row_groups) * a.item_rows;
        g.start = start;
        g.t0 = int(lo - start);
        g.t1 = int(min((long long)g.tiles, part.hi - start));
        lo = start + g.t1;
        if (g.t1 == g.tiles) {
            start += g.tiles;
            ++item;
        }
        return true;
    }
    return false;
}

template <int D, int RT>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_tc_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using SH = TcShape<D, RT>;
    constexpr uint32_t TMEM_COLS = 512, S_COL = 0, O_COL = 256;    // slot s at + 128 s
    constexpr uint32_t IDESC_S = idesc_bf16_f32(128, kTcTile, false);
    constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, true);
    constexpr int SLOT_STEP = RT == 1 ? 2 : 1;                     // tiles between a slot's tiles

    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ __align__(8) TcShared sh;
    __shared__ long long s_scan[kTcThreads / 32 + 2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;                  // swizzle atoms: 1024-byte aligned
    unsigned char* smem = smem_raw + (base - raw);

    allow_dependents_early();
    if (warp == 0) {
        tmem_alloc(&sh.tmem, TMEM_COLS);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 8; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], RT);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.o_full[s], 1);
            mbar_init(&sh.p_ready[s], 128);
        }
        sh.dead = 0;
        fence_mbar_init();
    }
    grid_dependency_wait();   // queries, pages and lengths may come from the previous kernel
    tc_fence_before_sync();
    const TreePart part = tree_part<kTcThreads>(a, s_scan);        // synchronises the CTA
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const bool dense = a.sel_ids == nullptr;
    long long lo = part.lo, start = part.start;
    int item = part.item;
    TcSegment g;

    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return;
        if (*reinterpret_cast<volatile int*>(&sh.dead) != 0) return;
        if (!mbar_wait_bounded(bar, parity, kWaitCycles)) {
            *reinterpret_cast<volatile int*>(&sh.dead) = 1;
            raise_error(a.err, SPARSE_ATTN_ERR_TIMEOUT);
        }
    };

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcRegsFew));
        uint32_t unit0 = 0;                                        // ring units used by earlier segments
        uint32_t tile0 = 0;                                        // tiles of earlier segments
        uint32_t mine0 = 0;                                        // tiles of this issuer's slot, likewise
        while (tc_next(a, part, lo, start, item, g)) {
            const int ntl = g.t1 - g.t0;
            bar_sync(1, kTcThreads);                               // queries staged, the ring is free
            if (warp == 8) {
                // ---- producer ---------------------------------------------------------
                const int n_e = a.bs >= kTcTile ? 1 : kTcTile >> a.bs_shift;   // entries of a tile
                const int per_batch = 32 / n_e;                    // tiles whose entries one batch holds
                const int e_base = (g.t0 * kTcTile) >> a.bs_shift;
                auto resolve = [&](int batch) -> int2 {
                    const int e = e_base + batch * 32 + lane;
                    return e < g.un.n_entries && batch * 32 + lane < ntl * n_e ? tree_entry(a, g.u, g.un, e)
                                                                              : make_int2(-1, 0);
                };
                int2 cur = resolve(0), nxt = resolve(1);
                for (int i = 0; i < ntl; ++i) {
                    const int at = i % per_batch;
                    if (i > 0 && at == 0) {
                        cur = nxt;
                        nxt = resolve(i / per_batch + 1);
                    }
                    int2 en;
                    en.x = __shfl_sync(kFullMask, cur.x, (at * n_e + lane) & 31);
                    en.y = __shfl_sync(kFullMask, cur.y, (at * n_e + lane) & 31);
                    const bool mine = lane < n_e, ok = mine && en.x >= 0;
                    const int e = e_base + i * n_e + lane;
                    const bool partly = mine && (!ok || en.y + a.bs > g.un.len || !(dense || e < g.un.n_ctx));
                    const uint32_t n_ok = __popc(__ballot_sync(kFullMask, ok));
                    const bool any_partly = __any_sync(kFullMask, partly);
                    const uint32_t info = (tile0 + i) % kTcInfo;
                    if (mine) sh.entry[info][lane] = make_int2(en.x, ok ? en.y : kNoToken);
                    if (lane == 0) sh.masked[info] = any_partly;
                    __syncwarp();
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const uint32_t n = unit0 + 2 * i + kv, st = n % SH::UNITS;
                        if (n >= SH::UNITS) wait(&sh.empty[st], (n / SH::UNITS - 1) & 1u);
                        if (*reinterpret_cast<volatile int*>(&sh.dead) != 0) break;   // start no more copies
                        if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], n_ok * uint32_t(a.bs * 128 * SH::HALVES));
                        __syncwarp();
                        if (ok) {
                            const uint32_t dst = base + SH::OFF_RING + st * SH::UNIT + lane * a.bs * 128;
#pragma unroll
                            for (int h = 0; h < SH::HALVES; ++h)
                                tma_load_3d(dst + h * SH::HALF, kv == 0 ? &kmap : &vmap, h * 64, 0, en.x, &sh.full[st]);
                        }
                    }
                }
            } else if (warp <= 10) {
                // ---- issuer of slot s ----------------------------------------------------
                const int s = warp - 9;
                uint32_t done = mine0;
                if (lane == 0) {
                    const uint64_t q_desc = smem_desc_sw128(base + (RT == 2 ? s * SH::Q_TILE : 0), 16, 1024);
                    const uint64_t p_desc = smem_desc_sw128(base + SH::OFF_P + s * SH::P_TILE, 16, 1024);
                    const uint64_t k_desc0 = smem_desc_sw128(base + SH::OFF_RING, 16, 1024);
                    const uint64_t v_desc0 = smem_desc_sw128(base + SH::OFF_RING, SH::HALF, 1024);
                    const uint32_t s_tm = tmem + S_COL + s * 128, o_tm = tmem + O_COL + s * 128;
                    for (int i = RT == 1 ? s : 0; i < ntl; i += SLOT_STEP, ++done) {
                        const uint32_t kn = unit0 + 2 * i, ks = kn % SH::UNITS;
                        const uint32_t vn = kn + 1, vs = vn % SH::UNITS;
                        wait(&sh.full[ks], (kn / SH::UNITS) & 1u);
                        if (done > 0) wait(&sh.o_full[s], (done - 1) & 1u);      // P of the last tile is read
                        tc_fence_after_sync();
                        const uint64_t kd = k_desc0 + uint64_t((ks * SH::UNIT) >> 4);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = uint32_t(((k >> 2) * SH::HALF + (k & 3) * 32) >> 4);
                            umma_bf16(s_tm, q_desc + off, kd + off, IDESC_S, k > 0 ? 1u : 0u);
                        }
                        umma_commit(&sh.s_full[s]);
                        umma_commit(&sh.empty[ks]);
                        wait(&sh.full[vs], (vn / SH::UNITS) & 1u);
                        wait(&sh.p_ready[s], done & 1u);
                        tc_fence_after_sync();
                        const uint64_t vd = v_desc0 + uint64_t((vs * SH::UNIT) >> 4);
                        // the small parts first
#pragma unroll
                        for (int k = 0; k < kTcTile / 16; ++k)
                            umma_bf16(o_tm, p_desc + uint32_t(((k >> 2) * SH::HALF + (k & 3) * 32) >> 4),
                                      vd + uint32_t((k * 16 * 128) >> 4), IDESC_O, k > 0 ? 1u : 0u);
#pragma unroll
                        for (int pp = 1; pp >= 0; --pp)
#pragma unroll
                            for (int k = 0; k < kTcTile / 16; ++k)
                                umma_bf16_ta(o_tm, s_tm + (k >> 1) * 32 + pp * 16 + (k & 1) * 8,
                                             vd + uint32_t((k * 16 * 128) >> 4), IDESC_O, 1u);
                        umma_commit(&sh.empty[vs]);
                        umma_commit(&sh.o_full[s]);
                    }
                }
                __syncwarp();
                mine0 += uint32_t(RT == 1 ? (ntl + 1 - s) / 2 : ntl);
            }
            unit0 += 2 * ntl;
            tile0 += ntl;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcRegsMany));
        const int s = warp >> 2;                                   // slot
        const int row = tid & 127;                                 // row of the slot's tile
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        const uint32_t s_tm = tmem + S_COL + s * 128 + lanes, o_tm = tmem + O_COL + s * 128 + lanes;
        const float scale = a.scale_log2;
        uint32_t tile0 = 0, done = 0, unit0 = 0;
        while (tc_next(a, part, lo, start, item, g)) {
            const int ntl = g.t1 - g.t0;
            const uint32_t* mask_b = a.mask != nullptr ? a.mask + (long long)g.b * a.Q * a.mask_words : nullptr;
            // ---- the item's queries, and the drafts that some query sees ----------------
            {
                constexpr int CPR = D / 8;                         // 16-byte chunks of a row
                for (int i = tid; i < RT * 128 * CPR; i += 256) {
                    const int r = i / CPR, c = i - r * CPR;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (g.row0 + r < a.R)
                        v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                 tree_out_row(a, g.b, g.kvh, g.row0 + r) * D) + c);
                    *reinterpret_cast<uint4*>(smem + (r >> 7) * SH::Q_TILE + (c >> 3) * SH::HALF + (r & 127) * 128 +
                                              (((c & 7) ^ (r & 7)) << 4)) = v;
                }
                fence_proxy_async_smem();
                const long long list = dense ? g.un.len : (long long)g.un.n_ctx << a.bs_shift;
                if ((long long)g.t1 * kTcTile > list) {            // this part meets drafts
                    for (int w = tid; w < a.mask_words; w += 256) {
                        uint32_t m = 0u;
                        if (mask_b == nullptr) m = ~0u;
                        else
                            for (int i = 0; i < a.Q; ++i) m |= mask_b[(long long)i * a.mask_words + w];
                        sh.any[w] = m;
                    }
                }
            }
            bar_sync(1, kTcThreads);

            const int r_unit = g.row0 + (RT == 2 ? s * 128 : 0) + row;
            const bool live = g.row0 + (RT == 2 ? s * 128 : 0) + 32 * (warp & 3) < a.R;    // of this warp's rows, any
            const int q_row = r_unit < a.R ? r_unit / a.G : 0;
            float acc[D];
#pragma unroll
            for (int d = 0; d < D; ++d) acc[d] = 0.f;
            float m_run = -INFINITY, l_run = 0.f;

            for (int i = RT == 1 ? s : 0; i < ntl; i += SLOT_STEP, ++done) {
                wait(&sh.s_full[s], done & 1u);
                __syncwarp();
                tc_fence_after_sync();
                const uint32_t info = (tile0 + i) % kTcInfo;
                const bool masked = sh.masked[info] != 0;
                uint32_t mk[4] = {~0u, ~0u, ~0u, ~0u};             // tokens that this row sees
                uint32_t bad[4] = {0u, 0u, 0u, 0u};
                if (masked) {
                    // which tokens the row sees; V rows of tokens that nobody sees are zeroed (their
                    // memory may hold anything), and so are drafts with infinities or NaN, which
                    // are added below where they are seen
                    const int e0 = ((g.t0 + i) * kTcTile) >> a.bs_shift;
                    auto tokens8 = [&](int g8, const uint32_t* words, int limit) -> uint32_t {
                        const int le = (g8 * 8) >> a.bs_shift;
                        const int first = sh.entry[info][le].y;
                        if (first == kNoToken) return 0u;
                        const int tok = first + ((g8 * 8) & (a.bs - 1));
                        const bool ctx = dense || e0 + le < g.un.n_ctx;
                        uint32_t bits = 0u;
                        if (ctx) {
                            const int n = min(8, max(0, g.un.len - tok));
                            bits = (1u << n) - 1u;
                        }
                        if (dense || !ctx) bits |= mask_bits8(words, tok - g.un.len, limit);
                        return bits;
                    };
                    const uint32_t* words = mask_b != nullptr ? mask_b + (long long)q_row * a.mask_words : nullptr;
                    const int limit = r_unit < a.R ? (mask_b != nullptr ? a.Q : q_row + 1) : 0;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        mk[w] = 0u;
#pragma unroll
                        for (int x = 0; x < 4; ++x) mk[w] |= tokens8(4 * w + x, words, limit) << (8 * x);
                    }
                    const uint32_t vn = unit0 + 2 * i + 1, vs = vn % SH::UNITS;
                    wait(&sh.full[vs], (vn / SH::UNITS) & 1u);
                    const int tok_row = row;                       // this thread looks after token `row`
                    uint32_t* s_bad = sh.bad[RT == 1 ? s : 0];
                    const int bar_id = RT == 1 ? 3 + s : 2, bar_n = RT == 1 ? 128 : 256;
                    constexpr int CH0 = SH::HALVES * 8 / RT;       // 16-byte chunks of the row, shared by the warpgroups
                    const int c0 = RT == 1 ? 0 : s * CH0;
                    unsigned char* vrow = smem + SH::OFF_RING + vs * SH::UNIT + tok_row * 128;
                    if (tid < 4 || (RT == 1 && s == 1 && row < 4)) s_bad[row] = 0u;
                    const bool seen = (tokens8(tok_row >> 3, sh.any, a.Q) >> (tok_row & 7)) & 1u;
                    const int first = sh.entry[info][tok_row >> a.bs_shift].y;
                    const bool draft = first != kNoToken && first + (tok_row & (a.bs - 1)) >= g.un.len;
                    bar_sync(bar_id, bar_n);
                    if (seen && draft) {
                        bool odd = false;
                        for (int c = c0; c < c0 + CH0; ++c) {
                            const uint4 v = *reinterpret_cast<const uint4*>(vrow + (c >> 3) * SH::HALF + (c & 7) * 16);
                            const uint32_t w4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                odd |= (w4[x] & 0x7f800000u) == 0x7f800000u || (w4[x] & 0x7f80u) == 0x7f80u;
                        }
                        if (odd) atomicOr(&s_bad[tok_row >> 5], 1u << (tok_row & 31));
                    }
                    bar_sync(bar_id, bar_n);
#pragma unroll
                    for (int w = 0; w < 4; ++w) bad[w] = s_bad[w];
                    if (!seen || ((bad[tok_row >> 5] >> (tok_row & 31)) & 1u)) {
                        for (int c = c0; c < c0 + CH0; ++c)
                            *reinterpret_cast<uint4*>(vrow + (c >> 3) * SH::HALF + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                        fence_proxy_async_smem();
                    }
                    if (RT == 2) bar_sync(bar_id, bar_n);
                }
                float alpha = 1.f, psum = 0.f;
                __syncwarp();
                if (live) {
                    // ---- the maximum ---------------------------------------------------------
                    float mx = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld32(s_tm + 32 * c, v);
                        tmem_wait_ld();
                        if (masked) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!((mk[c] >> j) & 1u)) v[j] = 0xff800000u;
                        }
                        float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                        for (int j = 0; j < 32; j += 2) {
                            x0 = fmaxf(x0, __uint_as_float(v[j]));
                            x1 = fmaxf(x1, __uint_as_float(v[j + 1]));
                        }
                        mx = fmaxf(mx, fmaxf(x0, x1));
                    }
                    const float m_new = fmaxf(m_run, mx * scale);
                    alpha = m_run == -INFINITY ? 0.f : fast_exp2(m_run - m_new);
                    m_run = m_new;
                    const float m_sub = m_new == -INFINITY ? 0.f : m_new;      // nothing seen yet: every weight is 0
                    if (masked && (bad[0] | bad[1] | bad[2] | bad[3])) {
#pragma unroll
                        for (int d = 0; d < D; ++d) acc[d] *= alpha;
                        l_run *= alpha;
                        alpha = 1.f;
#pragma unroll 1
                        for (int j = 0; j < kTcTile; ++j) {
                            if (!((bad[j >> 5] >> (j & 31)) & 1u)) continue;
                            const float sj = __uint_as_float(tmem_ld1(s_tm + j));
                            tmem_wait_ld();
                            const float p = (mk[j >> 5] >> (j & 31)) & 1u ? fast_exp2(fmaf(sj, scale, -m_sub)) : 0.f;
                            const int2 en = sh.entry[info][j >> a.bs_shift];
                            const uint4* vg = reinterpret_cast<const uint4*>(
                                static_cast<const uint16_t*>(a.v_pages) + (size_t(en.x) * a.bs + (j & (a.bs - 1))) * D);
                            if (p != 0.f) {
#pragma unroll
                                for (int c = 0; c < D / 8; ++c) {
                                    float f[8];
                                    unpack16<true>(__ldg(vg + c), f);
#pragma unroll
                                    for (int x = 0; x < 8; ++x) acc[8 * c + x] = fmaf(p, f[x], acc[8 * c + x]);
                                }
                            }
                            __syncwarp();
                        }
                    }
                    // ---- the weights, in three bf16 parts ----------------------------------------
                    unsigned char* p_row = smem + SH::OFF_P + s * SH::P_TILE + row * 128;
                    float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_ld32(s_tm + 32 * c, v);
                        tmem_wait_ld();
                        uint32_t hi[16], mid[16], small[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float p0 = fast_exp2(fmaf(__uint_as_float(v[2 * j]), scale, -m_sub));
                            float p1 = fast_exp2(fmaf(__uint_as_float(v[2 * j + 1]), scale, -m_sub));
                            if (masked) {
                                if (!((mk[c] >> (2 * j)) & 1u)) p0 = 0.f;
                                if (!((mk[c] >> (2 * j + 1)) & 1u)) p1 = 0.f;
                            }
                            sums[j & 1] += p0;
                            sums[2 + (j & 1)] += p1;
                            hi[j] = cut_bf16x2(p0, p1);
                            mid[j] = cut_bf16x2(p0, p1);
                            small[j] = cut_bf16x2(p0, p1);
                        }
                        tmem_st16(s_tm + 32 * c, hi);
                        tmem_st16(s_tm + 32 * c + 16, mid);
#pragma unroll
                        for (int x = 0; x < 4; ++x)
                            *reinterpret_cast<uint4*>(p_row + (c >> 1) * SH::HALF + (((((c & 1) << 2) + x) ^ (row & 7)) << 4)) =
                                make_uint4(small[4 * x], small[4 * x + 1], small[4 * x + 2], small[4 * x + 3]);
                    }
                    psum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
                    tmem_wait_st();
                    fence_proxy_async_smem();
                }
                tc_fence_before_sync();
                mbar_arrive(&sh.p_ready[s]);
                l_run = fmaf(l_run, alpha, psum);
                wait(&sh.o_full[s], done & 1u);
                __syncwarp();
                tc_fence_after_sync();
                if (live) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tmem_ld32(o_tm + 32 * c, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) acc[32 * c + j] = fmaf(acc[32 * c + j], alpha, __uint_as_float(v[j]));
                    }
                    tc_fence_before_sync();
                }
            }

            // ---- the part's (m, l, o): the output itself, or a partial -------------------------
            const bool complete = g.t0 == 0 && g.t1 == g.tiles;
            if (RT == 1) {
                // the odd tiles' rows join the even tiles' through the ring, which is idle now
                float4* x = reinterpret_cast<float4*>(smem + SH::OFF_RING) + row * (D / 4);
                float2* x_ml = reinterpret_cast<float2*>(smem + SH::OFF_P);
                bar_sync(2, 256);
                if (s == 1 && live) {
#pragma unroll
                    for (int c = 0; c < D / 4; ++c)
                        x[(c + lane) & (D / 4 - 1)] = make_float4(acc[4 * c], acc[4 * c + 1], acc[4 * c + 2], acc[4 * c + 3]);
                    x_ml[row] = make_float2(m_run, l_run);
                }
                bar_sync(2, 256);
                if (s == 0 && live) {
                    const float m1 = x_ml[row].x, m_new = fmaxf(m_run, m1);
                    const float w0 = m_run == -INFINITY ? 0.f : fast_exp2(m_run - m_new);
                    const float w1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - m_new);
                    l_run = l_run * w0 + x_ml[row].y * w1;
                    m_run = m_new;
#pragma unroll
                    for (int c = 0; c < D / 4; ++c) {
                        const float4 o = x[(c + lane) & (D / 4 - 1)];
                        acc[4 * c] = fmaf(acc[4 * c], w0, o.x * w1);
                        acc[4 * c + 1] = fmaf(acc[4 * c + 1], w0, o.y * w1);
                        acc[4 * c + 2] = fmaf(acc[4 * c + 2], w0, o.z * w1);
                        acc[4 * c + 3] = fmaf(acc[4 * c + 3], w0, o.w * w1);
                    }
                }
            }
            if ((RT == 2 || s == 0) && r_unit < a.R) {
                const int rr = r_unit - g.row0;
                const long long slot = (long long)tree_slot(blockIdx.x, part.per, g.start) * a.item_rows + rr;
                const float inv = complete ? (l_run == 0.f ? 0.f : 1.f / l_run) : 1.f;
                float* dst = complete ? a.out + tree_out_row(a, g.b, g.kvh, r_unit) * D : a.part_o + slot * D;
#pragma unroll
                for (int d = 0; d < D; d += 4)
                    *reinterpret_cast<float4*>(dst + d) =
                        make_float4(acc[d] * inv, acc[d + 1] * inv, acc[d + 2] * inv, acc[d + 3] * inv);
                if (!complete) {
                    a.part_m[slot] = m_run;
                    a.part_l[slot] = l_run;
                }
            }
            if (!complete) tree_arrive_and_merge<256>(a, g.item, g.start, g.tiles, part.per, &sh.last);
            else bar_sync(2, 256);                                 // queries and ring are free for the next item
            unit0 += 2 * ntl;
            tile0 += ntl;
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
    if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

// A tensor map over a page pool [num_pages * Hkv][bs][D] bf16: boxes of 64 channels x one
// block's tokens, written with the 128-byte swizzle that the products read.
inline cudaError_t encode_tree_map(CUtensorMap* map, const void* pool, int D, int bs, long long tiles)
{
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> cached{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 encode = cached.load(std::memory_order_acquire);
    if (encode == nullptr) {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess || fn == nullptr)
            return cudaErrorNotSupported;
        encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        cached.store(encode, std::memory_order_release);
    }
    const cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(bs), cuuint64_t(tiles)};
    const cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(D) * 2 * bs};
    const cuuint32_t box[3] = {64u, cuuint32_t(bs), 1u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(pool), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int RT>
cudaError_t launch_tc_t(const TreeArgs& a, cudaStream_t s)
{
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(tree_tc_kernel<D, RT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(TcShape<D, RT>::SMEM));
    });
    if (cfg != cudaSuccess) return cfg;
    CUtensorMap kmap, vmap;
    const long long tiles = (long long)a.num_pages * a.Hkv;
    cudaError_t e = encode_tree_map(&kmap, a.k_pages, D, a.bs, tiles);
    if (e != cudaSuccess) return e;
    e = encode_tree_map(&vmap, a.v_pages, D, a.bs, tiles);
    if (e != cudaSuccess) return e;
    const int ctas = num_sms() < kTreeMaxCtas ? num_sms() : kTreeMaxCtas;
    return launch_after_previous(tree_tc_kernel<D, RT>, dim3(unsigned(ctas)), dim3(kTcThreads), TcShape<D, RT>::SMEM, s, a,
                                 kmap, vmap);
}

}  // namespace

cudaError_t launch_tree_tc(TreeArgs a, cudaStream_t s)
{
    a.tile = kTcTile;
    a.item_rows = a.R <= 16 ? 16 : (a.R <= 64 ? 64 : (a.R <= 128 ? 128 : 256));
    a.row_groups = (a.R + a.item_rows - 1) / a.item_rows;
    a.min_per = 2;
    if (a.R <= 128) return a.D == 128 ? launch_tc_t<128, 1>(a, s) : launch_tc_t<64, 1>(a, s);
    return a.D == 128 ? launch_tc_t<128, 2>(a, s) : launch_tc_t<64, 2>(a, s);
}

}  // namespace sa
