// Draft-tree attention on the fifth-generation tensor cores (bf16 queries and K/V).
//
// A CTA holds up to 128 query rows of a (sequence, KV head) unit and walks the unit's list
// (sa_tree.cuh) in tiles of 128 tokens; more rows are further items over the same keys, which
// the L2 then holds.  Two slots take the even and the odd tiles, each with a score tile and an
// output tile in tensor memory (all 512 columns) and a softmax warpgroup pair of its own, so
// that one slot's products run while the other's softmax does.
//
// Few rows: with at most 64 (32) query rows the 128 rows of the tiles hold each of them 2 (4)
// times.  A copy takes its share of the tile's tokens, 16-token steps of P are zero in the
// others, and the copies are joined at the item's end like parts.  The products cost the same,
// the softmax, which they wait for, half (a quarter).
//
// Roles (20 warps):
//   warps 0-7, 8-15  the slots' softmax: two threads of a slot own a query row, each half of the
//               tile's tokens.  They read S, take the maximum, write P.  All four threads of a
//               row then add every finished O tile, a quarter of the channels each, to the
//               row's running O in registers (half as many registers as an O per slot).
//   warp 16     resolves the list's entries 32 at a time and brings K and V by TMA, one box
//               of 64 channels x one block per entry and channel half, into a ring of K and
//               V units that it refills as the products release them, into the next item;
//   warps 17, 18  one thread each: S = Q K^T, then O = P V for one slot (tcgen05.mma).
//
// Precision.  The output is fp32, so P goes into the product as three bf16 parts that hold
// its 24 bits exactly: two of them overwrite S in tensor memory (A operands there), the third
// goes through shared memory.  The tensor core rounds its running sum toward zero at every
// step (measured: the drift of a sum kept over 8K tokens is 1e-5), so O starts from zero in
// every tile and the rows add it up in registers by one FMA, which carries the softmax's
// rescaling as well.
//
// Per 128 tokens the tensor core does 4 x 128 x 128 x D multiply-adds (one part for S, three
// for P V), about 2050 cycles at D = 128; the 64 KB of K and V arrive in about 2800 cycles
// at the SM's share of the HBM bandwidth.
#include "sa_tcgen05.cuh"
#include "sa_tree.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

namespace sa {
namespace {

constexpr int kTcSoft = 512;           // softmax threads, 256 a slot
constexpr int kTcThreads = kTcSoft + 128;
constexpr int kTcTile = 128;

template <int D>
struct TcShape {
    static constexpr int HALVES = D / 64;
    static constexpr int HALF = kTcTile * 128;              // 128 rows x 64 bf16
    static constexpr int UNIT = HALVES * HALF;              // K or V of a tile
    static constexpr int Q_TILE = HALVES * HALF;
    static constexpr int P_TILE = 2 * HALF;                 // 128 rows x 128 tokens
    static constexpr int UNITS = D == 128 ? 4 : 7;
    // Tiles whose entries are remembered: while a tile's O is not yet added up, the V two tiles on
    // is still in the ring, and the producer is at most (UNITS + 1) / 2 tiles past that one.
    static constexpr int INFO = (UNITS + 1) / 2 + 4;
    static constexpr int OFF_P = Q_TILE;
    static constexpr int OFF_RING = OFF_P + 2 * P_TILE;
    static constexpr int OFF_SHARED = OFF_RING + UNITS * UNIT;
    static_assert(2 * P_TILE >= 128 * D * 4, "the rows leave through the P tiles");
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

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
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

// Waits for the loads in flight; the registers are named so that nothing uses them earlier.
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// Two fp32 operations in one instruction (each rounded as usual).
union F2 {
    unsigned long long u;
    float2 f;
};
__device__ __forceinline__ F2 make_f2(float x, float y)
{
    F2 r;
    r.f = make_float2(x, y);
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.u) : "l"(a.u), "l"(b.u), "l"(c.u));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}
__device__ __forceinline__ F2 sub2(F2 a, F2 b)
{
    F2 r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.u) : "l"(a.u), "l"(b.u));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A pair of fp32 cut to bf16 (the upper halves of the words; the first in the low half), the
// remainders left behind.
__device__ __forceinline__ uint32_t cut_bf16x2(F2& p)
{
    const uint32_t ux = __float_as_uint(p.f.x), uy = __float_as_uint(p.f.y);
    p = sub2(p, make_f2(__uint_as_float(ux & 0xffff0000u), __uint_as_float(uy & 0xffff0000u)));
    return __byte_perm(ux, uy, 0x7632);
}

// The smallest bf16 not below x, as an fp32's bits (NaN may become anything).
__device__ __forceinline__ uint32_t round_up_bf16(float x)
{
    const uint32_t u = __float_as_uint(x);
    // toward zero is up for negative values; positive ones go up unless they are exact
    return (u & 0x80000000u) ? u & 0xffff0000u : (u + (x < INFINITY ? 0xffffu : 0u)) & 0xffff0000u;
}

// Register shares: the CTA starts with 20 warps x 96; the softmax threads hold a quarter of an
// output row and half of a tile's scores.
constexpr int kTcRegsFew = 64, kTcRegsMany = 104;
static_assert(kTcRegsFew * 128 + kTcRegsMany * kTcSoft <= 96 * kTcThreads, "no more registers than the launch got");

template <int D>
struct TcShared {
    using SH = TcShape<D>;
    uint64_t full[SH::UNITS], empty[SH::UNITS], s_full[2], o_full[2], p_ready[2], o_read[2];
    union {
        int scan[kTreeScan<kTcThreads>];
        uint16_t top[2][2][2][128];             // half rows' maxima (slot, tile parity, half, row), bf16 rounded up
    };
    int token[SH::INFO][16];                    // first token of each entry of a tile
    int masked[SH::INFO];
    uint32_t odd[SH::INFO][4];                  // drafts of a tile whose V holds infinities or NaN
    uint32_t any[kTreeMaxDrafts / 32];
    uint32_t tmem;
    int dead;                                   // a bounded wait ran out: no more waiting
    int last;
};
template <int D>
constexpr size_t tc_smem()
{
    static_assert(TcShape<D>::OFF_SHARED + sizeof(TcShared<D>) <= 227 * 1024, "shared memory of a CTA");
    return TcShape<D>::OFF_SHARED + sizeof(TcShared<D>);
}

// One item's share of this CTA's part: tiles [t0, t1) of the item's list.
struct TcSegment {
    int u, b, kvh, item, row0, t0, t1, tiles, start;
    TreeUnit un;
};

__device__ __forceinline__ bool tc_next(const TreeArgs& a, const TreePart& part, int& lo, int& start, int& item,
                                        TcSegment& g)
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
        g.t0 = lo - start;
        g.t1 = min(g.tiles, part.hi - start);
        lo = start + g.t1;
        if (g.t1 == g.tiles) {
            start += g.tiles;
            ++item;
        }
        return true;
    }
    return false;
}

template <int D, int REP>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_tc_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using SH = TcShape<D>;
    constexpr uint32_t TMEM_COLS = 512, S_COL = 0, O_COL = 256;    // slot s at + 128 s
    constexpr uint32_t IDESC_S = idesc_bf16_f32(128, kTcTile, false);
    constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, true);

    extern __shared__ __align__(1024) unsigned char smem[];        // swizzle atoms: 1024-byte aligned
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_u32(smem);
    TcShared<D>& sh = *reinterpret_cast<TcShared<D>*>(smem + SH::OFF_SHARED);
    if ((base & 1023u) != 0u) {                                    // the alignment above is not kept: no result
        if (tid == 0) raise_error(a.err, SPARSE_ATTN_ERR_CAPACITY);
        return;
    }

    allow_dependents_early();
    if (warp == 0) {
        tmem_alloc(&sh.tmem, TMEM_COLS);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < SH::UNITS; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&sh.s_full[s], 1);
            mbar_init(&sh.o_full[s], 1);
            mbar_init(&sh.p_ready[s], kTcSoft / 2);
            mbar_init(&sh.o_read[s], kTcSoft / 2);
        }
        sh.dead = 0;
        fence_mbar_init();
    }
    grid_dependency_wait();   // queries, pages and lengths may come from the previous kernel
    tc_fence_before_sync();
    const TreePart part = tree_part<kTcThreads>(a, sh.scan);       // synchronises the CTA
    tc_fence_after_sync();
    const uint32_t tmem = sh.tmem;
    const bool dense = a.sel_ids == nullptr;
    int lo = part.lo, start = part.start, item = part.item;
    TcSegment g;

    auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (mbar_try_wait(bar, parity)) return;
        if (*reinterpret_cast<volatile int*>(&sh.dead) != 0) return;
        if (!mbar_wait_bounded(bar, parity, kWaitCycles)) {
            *reinterpret_cast<volatile int*>(&sh.dead) = 1;
            raise_error(a.err, SPARSE_ATTN_ERR_TIMEOUT);
        }
    };

    if (warp >= 16) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcRegsFew));
        uint32_t unit0 = 0;                                        // ring units used by earlier segments
        uint32_t tile0 = 0;                                        // tiles of earlier segments
        uint32_t done = 0;                                         // tiles of this issuer's slot so far
        while (tc_next(a, part, lo, start, item, g)) {
            const int ntl = g.t1 - g.t0;
            if (warp == 16) {
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
                    const uint32_t info = (tile0 + i) % SH::INFO;
                    if (mine) sh.token[info][lane] = ok ? en.y : kNoToken;
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
            } else if (warp <= 18) {
                // ---- issuer of slot s ----------------------------------------------------
                const int s = warp - 17;
                bar_sync(1, kTcSoft + 64);                         // queries staged
                if (lane == 0) {
                    const uint64_t q_desc = smem_desc_sw128(base, 16, 1024);
                    const uint64_t p_desc = smem_desc_sw128(base + SH::OFF_P + s * SH::P_TILE, 16, 1024);
                    const uint64_t k_desc0 = smem_desc_sw128(base + SH::OFF_RING, 16, 1024);
                    const uint64_t v_desc0 = smem_desc_sw128(base + SH::OFF_RING, SH::HALF, 1024);
                    const uint32_t s_tm = tmem + S_COL + s * 128, o_tm = tmem + O_COL + s * 128;
                    for (int i = s; i < ntl; i += 2, ++done) {
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
                        if (done > 0) wait(&sh.o_read[s], (done - 1) & 1u);      // the other slot's threads read O
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
                                umma_bf16_ta(o_tm, s_tm + k * 16 + pp * 8, vd + uint32_t((k * 16 * 128) >> 4), IDESC_O, 1u);
                        umma_commit(&sh.empty[vs]);
                        umma_commit(&sh.o_full[s]);
                    }
                }
                __syncwarp();
            }
            unit0 += 2 * ntl;
            tile0 += ntl;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcRegsMany));
        constexpr int CW = D / 4;                                  // channels of a thread
        constexpr int COPY = 128 / REP;                            // rows of a copy
        constexpr int OWN = 4 / REP;                               // 16-token steps a thread has of its half
        const int s = warp >> 3;                                   // slot
        const int h = (warp >> 2) & 1;                             // which half of a tile's tokens
        const int row = 32 * (warp & 3) + lane;                    // query row of the item
        const int ch0 = (2 * s + h) * CW;                          // first channel
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        const uint32_t s_tm = tmem + S_COL + s * 128 + 64 * h + lanes, o_tm = tmem + O_COL + ch0 + lanes;
        const int pair_bar = 5 + 4 * s + (warp & 3);               // the two warps that share rows of a slot
        const int own0 = row / COPY * OWN;                         // the first of them
        unsigned char* p_row = smem + SH::OFF_P + s * SH::P_TILE + h * SH::HALF + row * 128;
        const float scale = a.scale_log2;
        uint32_t tile0 = 0, unit0 = 0, soft_n = 0, acc_n[2] = {0, 0};
        while (tc_next(a, part, lo, start, item, g)) {
            const int ntl = g.t1 - g.t0;
            const uint32_t* mask_b = a.mask != nullptr ? a.mask + (long long)g.b * a.Q * a.mask_words : nullptr;
            // ---- the item's queries, and the drafts that some query sees ----------------
            {
                constexpr int CPR = D / 8;                         // 16-byte chunks of a row
                for (int i = tid; i < 128 * CPR; i += kTcSoft) {
                    const int r = i / CPR, c = i - r * CPR;
                    const int ru = g.row0 + r % COPY;
                    uint4 v = make_uint4(0u, 0u, 0u, 0u);
                    if (ru < a.R)
                        v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                 tree_out_row(a, g.b, g.kvh, ru) * D) + c);
                    *reinterpret_cast<uint4*>(smem + (c >> 3) * SH::HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
                }
                if (REP > 1) {                                     // the third part's tokens of other copies
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        *reinterpret_cast<uint4*>(p_row + 16 * x) = make_uint4(0u, 0u, 0u, 0u);
                }
                const long long list = dense ? g.un.len : (long long)g.un.n_ctx << a.bs_shift;
                if ((long long)g.t1 * kTcTile > list) {            // this part meets drafts
                    if (tid < a.mask_words) sh.any[tid] = mask_b == nullptr ? ~0u : 0u;
                    if (mask_b != nullptr) {
                        tree_sync<kTcSoft>();
                        for (int i = tid; i < a.Q * a.mask_words; i += kTcSoft) atomicOr(&sh.any[i % a.mask_words], mask_b[i]);
                    }
                }
                fence_proxy_async_smem();                          // before the tensor core uses this memory
            }
            bar_sync(1, kTcSoft + 64);

            const int r_unit = g.row0 + row % COPY;
            const bool live = g.row0 + 32 * (warp & 3) % COPY < a.R;           // any of this warp's rows
            const int q_row = r_unit < a.R ? r_unit / a.G : 0;
            // what the row sees of the drafts, and what any query sees
            const uint32_t* words = mask_b != nullptr ? mask_b + (long long)q_row * a.mask_words : nullptr;
            const DraftView view = draft_view(words, a.mask_words, r_unit < a.R ? (mask_b != nullptr ? a.Q : q_row + 1) : 0);
            F2 acc[CW / 2];
#pragma unroll
            for (int d = 0; d < CW / 2; ++d) acc[d] = make_f2(0.f, 0.f);
            float m_soft = -INFINITY, l_run = 0.f;                 // this slot's reference and half-row sum
            float m_other = -INFINITY;                             // the other slot's reference
            float m_acc = -INFINITY;                               // what acc is relative to

            // Tokens 8 g8 .. + 7 of local tile i that a query with this view sees.
            auto tokens8 = [&](int i, int g8, const DraftView& v) -> uint32_t {
                const int le = (g8 * 8) >> a.bs_shift;
                return tree_tokens8(a, g.un, g8 * 8, (((g.t0 + i) * kTcTile) >> a.bs_shift) + le,
                                    sh.token[(tile0 + i) % SH::INFO][le], v);
            };
            // Adds O of local tile i to this thread's channels.
            auto add_up = [&](int i) {
                const int sl = i & 1;
                wait(&sh.o_full[sl], acc_n[sl] & 1u);
                __syncwarp();
                tc_fence_after_sync();
                if (live) {
                    uint32_t v[CW / 16][16];
#pragma unroll
                    for (int c = 0; c < CW / 16; ++c) tmem_ld16(o_tm + sl * 128 + 16 * c, v[c]);
                    float m = m_soft;
                    if (sl != s) {
                        const uint32_t pr = acc_n[sl] & 1u;
                        m_other = fmaxf(m_other, fmaxf(__uint_as_float(uint32_t(sh.top[sl][pr][0][row]) << 16),
                                                       __uint_as_float(uint32_t(sh.top[sl][pr][1][row]) << 16)));
                        m = m_other;
                    }
                    const float m_new = fmaxf(m_acc, m);
                    const float w0 = m_acc == -INFINITY ? 0.f : fast_exp2(m_acc - m_new);
                    const float w1 = m == -INFINITY ? 0.f : fast_exp2(m - m_new);
                    m_acc = m_new;
                    const F2 w02 = make_f2(w0, w0), w12 = make_f2(w1, w1);
                    const bool move = __any_sync(kFullMask, w0 != 1.f);          // rarely after the first tiles
#pragma unroll
                    for (int c = 0; c < CW / 16; ++c) {
                        tmem_wait_ld16(v[c]);
                        if (move) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) acc[8 * c + j] = mul2(acc[8 * c + j], w02);
                        }
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            acc[8 * c + j] = fma2(make_f2(__uint_as_float(v[c][2 * j]), __uint_as_float(v[c][2 * j + 1])), w12,
                                                  acc[8 * c + j]);
                    }
                    const uint32_t info = (tile0 + i) % SH::INFO;
                    if (sh.masked[info] != 0 && (sh.odd[info][0] | sh.odd[info][1] | sh.odd[info][2] | sh.odd[info][3])) {
                        // infinities and NaN were taken out of V: they come back where they are seen
#pragma unroll 1
                        for (int j = 0; j < kTcTile; ++j) {
                            if (!((sh.odd[info][j >> 5] >> (j & 31)) & 1u)) continue;
                            if (unsigned(((j >> 4) & 3) - own0) >= unsigned(OWN) || !((tokens8(i, j >> 3, view) >> (j & 7)) & 1u)) continue;
                            const int2 en = tree_entry(a, g.u, g.un, (((g.t0 + i) * kTcTile) + j) >> a.bs_shift);
                            const uint16_t* vg = static_cast<const uint16_t*>(a.v_pages) +
                                                 (size_t(en.x) * a.bs + (j & (a.bs - 1))) * D + ch0;
#pragma unroll
                            for (int x = 0; x < CW / 2; ++x) {
                                const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(vg) + x);
                                if ((w & 0x7f80u) == 0x7f80u) acc[x].f.x += bf16_lo(w);
                                if ((w & 0x7f800000u) == 0x7f800000u) acc[x].f.y += bf16_hi(w);
                            }
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before_sync();
                if (sl != s) mbar_arrive(&sh.o_read[sl]);
                ++acc_n[sl];
            };

            int added = 0;                                         // tiles whose O is added up
            for (int i = s; i < ntl; i += 2, ++soft_n) {
                wait(&sh.s_full[s], soft_n & 1u);
                __syncwarp();
                tc_fence_after_sync();
                const uint32_t info = (tile0 + i) % SH::INFO;
                if (sh.masked[info] != 0) {
                    // Scores of tokens that the row does not see become -infinity.  V rows of tokens
                    // that nobody sees are zeroed (their memory may hold anything), and so are
                    // infinities and NaN of drafts, which are added back where they are seen.
                    if (live) {
#pragma unroll 1
                        for (int c = own0; c < own0 + OWN; ++c) {
                            const uint32_t mk = tokens8(i, 8 * h + 2 * c, view) |
                                                tokens8(i, 8 * h + 2 * c + 1, view) << 8;
                            uint32_t v[16];
                            __syncwarp();
                            tmem_ld16(s_tm + 16 * c, v);
                            tmem_wait_ld16(v);
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if (!((mk >> j) & 1u)) v[j] = 0xff800000u;
                            tmem_st16(s_tm + 16 * c, v);
                        }
                        tmem_wait_st();
                    }
                    const uint32_t vn = unit0 + 2 * i + 1, vs = vn % SH::UNITS;
                    wait(&sh.full[vs], (vn / SH::UNITS) & 1u);
                    // the slot's two threads of number `row` look after token `row`, half its channels each
                    constexpr int CHUNKS = SH::HALVES * 4;
                    unsigned char* vrow = smem + SH::OFF_RING + vs * SH::UNIT + row * 128;
                    const bool seen = (tokens8(i, row >> 3, draft_view(sh.any, a.mask_words, a.Q)) >> (row & 7)) & 1u;
                    const int first = sh.token[info][row >> a.bs_shift];
                    const bool draft = first != kNoToken && first + (row & (a.bs - 1)) >= g.un.len;
                    if (h == 0 && row < 4) sh.odd[info][row] = 0u;
                    bar_sync(3 + s, kTcSoft / 2);
                    bool changed = false;
                    for (int c = h * CHUNKS; c < (h + 1) * CHUNKS; ++c) {
                        uint4* at = reinterpret_cast<uint4*>(vrow + (c >> 3) * SH::HALF + (c & 7) * 16);
                        if (!seen) {
                            *at = make_uint4(0u, 0u, 0u, 0u);
                            changed = true;
                        } else if (draft) {
                            const uint4 v = *at;
                            uint32_t w4[4] = {v.x, v.y, v.z, v.w};
                            bool odd = false;
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                if ((w4[x] & 0x7f800000u) == 0x7f800000u) {
                                    w4[x] &= 0xffffu;
                                    odd = true;
                                }
                                if ((w4[x] & 0x7f80u) == 0x7f80u) {
                                    w4[x] &= 0xffff0000u;
                                    odd = true;
                                }
                            }
                            if (odd) {
                                *at = make_uint4(w4[0], w4[1], w4[2], w4[3]);
                                atomicOr(&sh.odd[info][row >> 5], 1u << (row & 31));
                                changed = true;
                            }
                        }
                    }
                    if (changed) fence_proxy_async_smem();
                }
                __syncwarp();
                if (live) {
                    // ---- the maximum: of half a row, then of both halves ----------------------
                    // The first steps stay in registers; with four, two are read again below.
                    constexpr int KEEP = OWN == 1 ? 1 : 2;
                    uint32_t va[2][16], vb[KEEP][16];
                    float x0 = -INFINITY, x1 = -INFINITY;
                    auto top_of = [&](const uint32_t (&v)[16]) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            x0 = max3(x0, __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
                            x1 = max3(x1, __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]));
                        }
                    };
                    const uint32_t own_tm = s_tm + 16 * own0;
                    if (OWN == 4) {
                        tmem_ld16(own_tm + 32, va[0]);
                        tmem_ld16(own_tm + 48, va[1]);
                        tmem_wait_ld16(va[0]);
                        tmem_wait_ld16(va[1]);
                    }
#pragma unroll
                    for (int c = 0; c < KEEP; ++c) tmem_ld16(own_tm + 16 * c, vb[c]);
                    if (OWN == 4) {
                        top_of(va[0]);
                        top_of(va[1]);
                    }
#pragma unroll
                    for (int c = 0; c < KEEP; ++c) {
                        tmem_wait_ld16(vb[c]);
                        top_of(vb[c]);
                    }
                    // Any reference near the maximum will do, as long as the row's threads use the
                    // same one: they exchange it as bf16, rounded up.
                    const uint32_t top = round_up_bf16(fmaxf(x0, x1) * scale), pr = soft_n & 1u;
                    sh.top[s][pr][h][row] = uint16_t(top >> 16);
                    bar_sync(pair_bar, 64);
                    const float other = __uint_as_float(uint32_t(sh.top[s][pr][1 - h][row]) << 16);
                    const float m_new = fmaxf(m_soft, fmaxf(__uint_as_float(top), other));
                    l_run *= m_soft == -INFINITY ? 0.f : fast_exp2(m_soft - m_new);
                    m_soft = m_new;
                    const float m_sub = m_new == -INFINITY ? 0.f : m_new;      // nothing seen yet: every weight is 0
                    // ---- the weights, in three bf16 parts, over the scores' own columns -----------
                    const F2 scale2 = make_f2(scale, scale), m2 = make_f2(-m_sub, -m_sub);
                    F2 sum_a = make_f2(0.f, 0.f), sum_b = make_f2(0.f, 0.f);
                    auto weights = [&](int c, const uint32_t (&v)[16]) {
                        uint32_t hm[16], small[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            F2 p = fma2(make_f2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), scale2, m2);
                            p = make_f2(fast_exp2(p.f.x), fast_exp2(p.f.y));
                            if (j & 1) sum_b = add2(sum_b, p);
                            else sum_a = add2(sum_a, p);
                            hm[j] = cut_bf16x2(p);
                            hm[8 + j] = cut_bf16x2(p);
                            small[j] = __byte_perm(__float_as_uint(p.f.x), __float_as_uint(p.f.y), 0x7632);
                        }
                        tmem_st16(own_tm + 16 * c, hm);
#pragma unroll
                        for (int x = 0; x < 2; ++x)
                            *reinterpret_cast<uint4*>(p_row + (((2 * (own0 + c) + x) ^ (row & 7)) << 4)) =
                                make_uint4(small[4 * x], small[4 * x + 1], small[4 * x + 2], small[4 * x + 3]);
                    };
                    if (REP > 1) {
                        uint32_t none[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) none[j] = 0u;
#pragma unroll
                        for (int c = OWN; c < 4; ++c) tmem_st16(s_tm + 16 * ((own0 + c) & 3), none);
                    }
                    weights(0, vb[0]);
                    if (OWN == 4) tmem_ld16(own_tm + 32, va[0]);
                    if (OWN > 1) weights(1, vb[KEEP - 1]);
                    if (OWN == 4) {
                        tmem_wait_ld16(va[0]);
                        tmem_ld16(own_tm + 48, va[1]);
                        weights(2, va[0]);
                        tmem_wait_ld16(va[1]);
                        weights(3, va[1]);
                    }
                    const F2 sum = add2(sum_a, sum_b);
                    l_run += sum.f.x + sum.f.y;
                    tmem_wait_st();
                    fence_proxy_async_smem();
                }
                tc_fence_before_sync();
                mbar_arrive(&sh.p_ready[s]);
                for (; added <= i; ++added) add_up(added);         // the other slot's last tile, then this one
            }
            for (; added < ntl; ++added) add_up(added);

            // ---- the part's (m, l, o): the output itself, or a partial -------------------------
            // The four threads' sums (and the copies') meet through the query tile, the rows leave through
            // the P tiles (both idle now), a warp 512 bytes at a time.
            const bool complete = g.t0 == 0 && g.t1 == g.tiles;
            constexpr int V4 = D / 4;
            float* x_l = reinterpret_cast<float*>(smem);                       // [slot][half][row]
            float* x_m = x_l + 512;                                            // [row]
            float4* x_rows = reinterpret_cast<float4*>(smem + SH::OFF_P);
            auto cell = [&](int r, int c) -> float4& { return x_rows[r * V4 + ((c + r) & (V4 - 1))]; };
            if (live) l_run = m_soft == -INFINITY ? 0.f : l_run * fast_exp2(m_soft - m_acc);
            tree_sync<kTcSoft>();
            x_l[(2 * s + h) * 128 + row] = l_run;
            if (s == 0 && h == 0) x_m[row] = m_acc;
            tree_sync<kTcSoft>();
            if (live) {
                float M = m_acc;
#pragma unroll
                for (int y = 1; y < REP; ++y) M = fmaxf(M, x_m[(row + y * COPY) & 127]);
                float w = 1.f;
                l_run = 0.f;
#pragma unroll
                for (int y = 0; y < REP; ++y) {                                // in the copies' order
                    const int r = row % COPY + y * COPY;
                    const float my = x_m[r], wy = REP == 1 ? 1.f : (my == -INFINITY ? 0.f : fast_exp2(my - M));
                    l_run = fmaf(wy, (x_l[r] + x_l[128 + r]) + (x_l[256 + r] + x_l[384 + r]), l_run);
                    if (REP > 1 && r == row) w = wy;
                }
                if (complete) {
                    w = l_run == 0.f ? 0.f : w / l_run;
                } else if (s == 0 && h == 0 && row < COPY && r_unit < a.R) {
                    const long long slot = (long long)tree_slot(blockIdx.x, part.per, g.start) * a.item_rows + row;
                    a.part_m[slot] = M;
                    a.part_l[slot] = l_run;
                }
#pragma unroll
                for (int c = 0; c < CW / 4; ++c)
                    cell(row, ch0 / 4 + c) = make_float4(acc[2 * c].f.x * w, acc[2 * c].f.y * w, acc[2 * c + 1].f.x * w,
                                                         acc[2 * c + 1].f.y * w);
            }
            tree_sync<kTcSoft>();
            {
                const int rows = min(a.item_rows, a.R - g.row0);
                float4* part_rows = reinterpret_cast<float4*>(a.part_o) +
                                    (long long)tree_slot(blockIdx.x, part.per, g.start) * a.item_rows * V4;
                for (int i = tid; i < rows * V4; i += kTcSoft) {
                    const int r = i / V4, c = i % V4;
                    float4* dst = complete ? reinterpret_cast<float4*>(a.out) + tree_out_row(a, g.b, g.kvh, g.row0 + r) * V4
                                           : part_rows + (long long)r * V4;
                    float4 o = cell(r, c);
#pragma unroll
                    for (int y = 1; y < REP; ++y) {
                        const float4 z = cell(r + y * COPY, c);
                        o = make_float4(o.x + z.x, o.y + z.y, o.z + z.z, o.w + z.w);
                    }
                    dst[c] = o;
                }
            }
            if (a.combine) {
                if (tid == 0 && g.t0 == 0) tree_note_parts(a, g.item, g.start, g.tiles, part.per);
            } else if (!complete) {
                tree_arrive_and_merge<kTcSoft>(a, g.item, g.start, g.tiles, part.per, &sh.last,
                                               reinterpret_cast<float*>(smem + SH::OFF_P), 2 * SH::P_TILE / 4);
            }
            tree_sync<kTcSoft>();                                  // this memory is free for the next item
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

template <int D, int REP>
cudaError_t launch_tc_t(TreeArgs a, cudaStream_t s)
{
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(tree_tc_kernel<D, REP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(tc_smem<D>()));
    });
    if (cfg != cudaSuccess) return cfg;
    CUtensorMap kmap, vmap;
    const long long tiles = (long long)a.num_pages * a.Hkv;
    cudaError_t e = encode_tree_map(&kmap, a.k_pages, D, a.bs, tiles);
    if (e != cudaSuccess) return e;
    e = encode_tree_map(&vmap, a.v_pages, D, a.bs, tiles);
    if (e != cudaSuccess) return e;
    const int ctas = num_sms() < kTreeMaxCtas ? num_sms() : kTreeMaxCtas;
    tree_choose_combine(a, ctas);
    e = launch_after_previous(tree_tc_kernel<D, REP>, dim3(unsigned(ctas)), dim3(kTcThreads), tc_smem<D>(), s, a, kmap, vmap);
    return e == cudaSuccess && a.combine ? launch_tree_combine(a, s) : e;
}

}  // namespace

cudaError_t launch_tree_tc(TreeArgs a, cudaStream_t s)
{
    a.tile = kTcTile;
    a.item_rows = tree_item_rows(a.R);
    a.row_groups = (a.R + a.item_rows - 1) / a.item_rows;
    a.min_per = 2;
    a.half_slack = 3;
    if (a.R <= 32) return a.D == 128 ? launch_tc_t<128, 4>(a, s) : launch_tc_t<64, 4>(a, s);
    if (a.R <= 64) return a.D == 128 ? launch_tc_t<128, 2>(a, s) : launch_tc_t<64, 2>(a, s);
    return a.D == 128 ? launch_tc_t<128, 1>(a, s) : launch_tc_t<64, 1>(a, s);
}

}  // namespace sa
