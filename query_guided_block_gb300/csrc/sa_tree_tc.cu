// Draft-tree attention on the fifth-generation tensor cores (bf16 queries and K/V).
//
// A CTA holds up to 128 query rows of a (sequence, KV head) unit and walks the unit's list
// (sa_tree.cuh) in tiles of 128 tokens; more rows are further items over the same keys, which
// the L2 then holds.  Two slots take the tiles in turn, each with a score tile and an
// output tile in tensor memory (all 512 columns), so that one tile's products run while the
// next one's softmax does.  (Three score tiles and one output tile: 96 rows over 128K tokens 131 us
// for 117, since adding up the output, 1000 cycles, then lies between two tiles' products.)
//
// Few rows: with at most 64 (32) query rows the 128 rows of the tiles hold each of them 2 (4)
// times, and the copies' rows of P are different parts of the weights: one pass over V multiplies
// the first two (all three) parts at once, and the copies of O are added up at the item's end.  V
// is read from shared memory twice (once) instead of three times, and all parts fit into tensor
// memory, which leaves room for two more ring units.  Against copies that share the tokens out
// (three passes over V, the third part through shared memory): 32 rows over 16 x 32K tokens 328 us
// for 402, 64 rows over 16 ragged contexts of up to 32K 277 for 320, 80 selected blocks 48 for 53.
//
// Roles (16 warps):
//   warps 0-7   the softmax: two threads own a query row, each half of the tile's tokens.  They
//               read S, join their maxima in a word of shared memory, write P.
//   warps 8-11  add every finished O tile to the running O: a thread per row, the whole row in
//               registers.
//   warp 12     resolves the list's entries 32 at a time and brings K and V by TMA, one box
//               of 64 channels x one block per entry and channel half, into a ring of K and
//               V units that it refills as the products release them, into the next item;
//   warps 13, 14  one thread each: S = Q K^T and O = P V (tcgen05.mma).
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
// at the SM's share of the HBM bandwidth.  Up to 64 rows memory bounds it (32 rows: 95% of the
// measured copy bandwidth); at 96 rows over 128K tokens (114 us, 79 us of memory) and 256 rows
// over 8 x 16K (233 us, 81 us of memory, 162 us of the four products) it is the chain S, softmax, P V
// of a tile and the passes over V, whose shared-memory reads (3 x 32 KB, with Q, K and the third
// part 190 KB a tile) take about as long as the products.
#include "sa_tcgen05.cuh"
#include "sa_tree.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

namespace sa {
namespace {

constexpr int kTcSoft = 256;           // softmax threads
constexpr int kTcWork = kTcSoft + 128; // and those that hold the running O
constexpr int kTcThreads = kTcWork + 128;
constexpr int kTcTile = 128;

template <int D, int REP>
struct TcShape {
    static constexpr int HALVES = D / 64;
    static constexpr int HALF = kTcTile * 128;              // 128 rows x 64 bf16
    static constexpr int UNIT = HALVES * HALF;              // K or V of a tile
    static constexpr int Q_TILE = HALVES * HALF;
    static constexpr int P_TILE = 2 * HALF;                 // 128 rows x 128 tokens
    static constexpr int P_TILES = REP == 1 ? 2 : 0;        // of P's third part in shared memory
    // The ring.  A parity tells a load into a stage from the next one but not from the one before,
    // so a thread may wait for a load once the one before it in that stage is known to have landed.
    // That holds for K of tile i once tile i - 2's output is done, and for V of tile i once its
    // weights are there (they follow those of the tile before, and its scores).
    static constexpr int UNITS = (D == 128 ? 4 : 8) + (2 - P_TILES) * P_TILE / UNIT;
    // Tiles whose entries are remembered: while a tile's O is not yet added up, the V two tiles on
    // is still in the ring, and the producer is at most (UNITS + 1) / 2 + 1 tiles past that one.
    static constexpr int INFO = (UNITS + 1) / 2 + 4;
    static constexpr int OFF_P = Q_TILE;
    static constexpr int OFF_RING = OFF_P + P_TILES * P_TILE;
    static constexpr int OFF_SHARED = OFF_RING + UNITS * UNIT;
    // Memory that is idle at an item's end, where its rows leave through: the P tiles, or the query
    // tile, where the copies are added up in turn.
    static constexpr int OFF_ROWS = P_TILES ? OFF_P : 0;
    static constexpr int ROWS_BYTES = P_TILES ? P_TILES * P_TILE : Q_TILE;
    static_assert(ROWS_BYTES >= (REP == 4 ? 2 : 1) * (128 / REP) * D * 4, "an item's rows, of two copies with four");
};

// Where the weights of tokens 16 k .. + 15 lie in the 64 columns of their half tile's scores: two
// parts in turn, or first one and then the other.
template <int REP>
__device__ __forceinline__ constexpr uint32_t tc_part_col(int k, int part)
{
    return (k >> 2) * 64 + (REP == 1 ? (k & 3) * 16 + part * 8 : part * 32 + (k & 3) * 8);
}

// Position in a segment's sequence of loads of local tile i's K and V: a tile's K comes before the
// V of the tile before it, which is needed later.
__device__ __forceinline__ uint32_t k_unit(int i) { return i == 0 ? 0u : uint32_t(2 * i - 1); }
__device__ __forceinline__ uint32_t v_unit(int i, int n) { return uint32_t(min(2 * i + 2, 2 * n - 1)); }

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

// The upper halves of a pair; the pair without what a mask keeps of it.
__device__ __forceinline__ uint32_t top_bf16x2(F2 p) { return __byte_perm(__float_as_uint(p.f.x), __float_as_uint(p.f.y), 0x7632); }
__device__ __forceinline__ F2 less(F2 p, uint32_t mask)
{
    return sub2(p, make_f2(__uint_as_float(__float_as_uint(p.f.x) & mask), __uint_as_float(__float_as_uint(p.f.y) & mask)));
}

// fp32 values as whole numbers of the same order (its own inverse), so that an integer maximum finds
// the largest.
__device__ __forceinline__ int ordered_bits(int x) { return x ^ ((x >> 31) & 0x7fffffff); }
constexpr int kOrderedLeast = int(0x807fffffu);                     // -infinity

// A row's reference for a tile: the largest score so far, unscaled and whatever its size, or an earlier
// one at most 6 below it in base-2 logits, so that it changes rarely (a weight is 2^6 at most then).  Its
// product with the scale is rounded by itself wherever it is used (__fmul_rn): what the weights are
// relative to is the rounded one.
__device__ __forceinline__ float tc_reference(float m, int top, float scale)
{
    const float t = __int_as_float(ordered_bits(top));
    return __fmul_rn(t, scale) > __fmul_rn(m, scale) + 6.f ? t : m;   // beyond 2^28 any larger one
}

// A weight is exp2(score * scale - m) by one fused multiply-add, m = reference * scale rounded: all weights
// are off by the same factor, which the total takes out again.  From |m| = 2^29 on (2^16 in that
// factor) two scores are equal or at least 2^5 apart, so that only equal ones of the largest count:
// there the scale gives way to a power of two that takes the reference to 2^30 .. 2^31, exactly.
__device__ __forceinline__ bool tc_large(float m) { return fabsf(m) >= 536870912.f; }
__device__ __forceinline__ float tc_power(float reference)
{
    const int e = 284 - ((__float_as_int(reference) >> 23) & 255);  // 127 + 30 - (its exponent)
    return __int_as_float(min(e, 254) << 23);
}

// Register shares: the CTA starts with 16 warps x 128.  With 152 for both the output threads have two
// loads fewer in flight: 96 rows over 128K tokens 123 us instead of 119.
constexpr int kTcRegsSoft = 136;       // half of a tile's scores of a row
constexpr int kTcRegsSum = 184;        // an output row
constexpr int kTcRegsFew = 56;
static_assert(kTcRegsSoft * kTcSoft + kTcRegsSum * 128 + kTcRegsFew * 128 <= 128 * kTcThreads,
              "no more registers than the launch got");

template <int D, int REP>
struct TcShared {
    using SH = TcShape<D, REP>;
    uint64_t full[SH::UNITS], empty[SH::UNITS], s_full[2], o_full[2], p_ready[2], o_read[2];
    union {
        int scan[kTreeScan<kTcThreads>];
        int top[4][128];                        // a row's maximum (tile mod 4, row) as ordered_bits
    };
    int token[SH::INFO][16];                    // first token of each entry of a tile
    int masked[SH::INFO];
    uint32_t odd[SH::INFO][4];                  // drafts of a tile whose V holds infinities or NaN
    uint32_t any[kTreeMaxDrafts / 32];
    uint32_t tmem;
    int dead;                                   // a bounded wait ran out: no more waiting
    int last;
};
template <int D, int REP>
constexpr size_t tc_smem()
{
    static_assert(TcShape<D, REP>::OFF_SHARED + sizeof(TcShared<D, REP>) <= 227 * 1024, "shared memory of a CTA");
    return TcShape<D, REP>::OFF_SHARED + sizeof(TcShared<D, REP>);
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
        g.t1 = part.whole ? g.tiles : min(g.tiles, part.hi - start);
        lo = start + g.t1;
        if (g.t1 == g.tiles) {
            start += g.tiles;
            ++item;
        }
        return true;
    }
    return false;
}

// The item's rows from the P tiles to the output or the partials, a warp 512 bytes at a time, by
// the softmax and the O threads together (the query and P tiles are free afterwards).
template <int D, int REP>
__device__ __forceinline__ void tc_store_rows(const TreeArgs& a, const TreePart& part, const TcSegment& g,
                                              unsigned char* smem, int* s_last, int tid)
{
    using SH = TcShape<D, REP>;
    constexpr int V4 = D / 4;
    const bool complete = g.t0 == 0 && g.t1 == g.tiles;
    const float4* x_rows = reinterpret_cast<const float4*>(smem + SH::OFF_ROWS);
    tree_sync<kTcWork>();
    const int rows = min(a.item_rows, a.R - g.row0);
    float4* part_rows = reinterpret_cast<float4*>(a.part_o) +
                        (long long)tree_slot(blockIdx.x, part.per, g.start) * a.item_rows * V4;
    for (int i = tid; i < rows * V4; i += kTcWork) {
        const int r = i / V4, c = i % V4;
        float4* dst = complete ? reinterpret_cast<float4*>(a.out) + tree_out_row(a, g.b, g.kvh, g.row0 + r) * V4
                               : part_rows + (long long)r * V4;
        dst[c] = x_rows[r * V4 + ((c + r) & (V4 - 1))];
    }
    if (a.combine) {
        if (tid == 0 && g.t0 == 0) tree_note_parts(a, g.item, g.start, g.tiles, part.per);
    } else if (!complete) {
        tree_arrive_and_merge<kTcWork>(a, g.item, g.start, g.tiles, part.per, s_last,
                                       reinterpret_cast<float*>(smem + SH::OFF_ROWS), SH::ROWS_BYTES / 4);
    }
    tree_sync<kTcWork>();
}

template <int D, int REP>
__global__ void __launch_bounds__(kTcThreads, 1)
    tree_tc_kernel(const TreeArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap)
{
    using SH = TcShape<D, REP>;
    constexpr uint32_t TMEM_COLS = 512, S_COL = 0, O_COL = 256;    // slot s at + 128 s
    constexpr uint32_t IDESC_S = idesc_bf16_f32(128, kTcTile, false);
    constexpr uint32_t IDESC_O = idesc_bf16_f32(128, D, true);

    extern __shared__ __align__(1024) unsigned char smem[];        // swizzle atoms: 1024-byte aligned
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base = smem_u32(smem);
    TcShared<D, REP>& sh = *reinterpret_cast<TcShared<D, REP>*>(smem + SH::OFF_SHARED);
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
            mbar_init(&sh.p_ready[s], kTcSoft);
            mbar_init(&sh.o_read[s], kTcWork - kTcSoft);
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

    if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcRegsFew));
        uint32_t unit0 = 0;                                        // ring units used by earlier segments
        uint32_t tile0 = 0;                                        // tiles of earlier segments
        while (tc_next(a, part, lo, start, item, g)) {
            const int ntl = g.t1 - g.t0;
            if (warp == 12) {
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
                int2 en = make_int2(-1, 0), en_v;
                uint32_t n_ok = 0, n_ok_v;
                auto load = [&](uint32_t n, const void* map, int tile_index, uint32_t entries) {
                    const uint32_t st = n % SH::UNITS;
                    if (n >= SH::UNITS) wait(&sh.empty[st], (n / SH::UNITS - 1) & 1u);
                    if (*reinterpret_cast<volatile int*>(&sh.dead) != 0) return;      // start no more copies
                    if (lane == 0) mbar_arrive_expect_tx(&sh.full[st], entries * uint32_t(a.bs * 128 * SH::HALVES));
                    __syncwarp();
                    if (lane < n_e && tile_index >= 0) {
                        const uint32_t dst = base + SH::OFF_RING + st * SH::UNIT + lane * a.bs * 128;
#pragma unroll
                        for (int h = 0; h < SH::HALVES; ++h)
                            tma_load_3d(dst + h * SH::HALF, map, h * 64, 0, tile_index, &sh.full[st]);
                    }
                };
                for (int i = 0; i <= ntl; ++i) {                   // K of tile i, then V of the one before
                    en_v = en;
                    n_ok_v = n_ok;
                    if (i < ntl) {
                        const int at = i % per_batch;
                        if (i > 0 && at == 0) {
                            cur = nxt;
                            nxt = resolve(i / per_batch + 1);
                        }
                        en.x = __shfl_sync(kFullMask, cur.x, (at * n_e + lane) & 31);
                        en.y = __shfl_sync(kFullMask, cur.y, (at * n_e + lane) & 31);
                        const bool mine = lane < n_e, ok = mine && en.x >= 0;
                        const int e = e_base + i * n_e + lane;
                        const bool partly = mine && (!ok || en.y + a.bs > g.un.len || !(dense || e < g.un.n_ctx));
                        n_ok = __popc(__ballot_sync(kFullMask, ok));
                        const bool any_partly = __any_sync(kFullMask, partly);
                        const uint32_t info = (tile0 + i) % SH::INFO;
                        if (mine) sh.token[info][lane] = ok ? en.y : kNoToken;
                        if (lane == 0) sh.masked[info] = any_partly;
                        if (lane < 4) sh.odd[info][lane] = 0u;
                        __syncwarp();
                        load(unit0 + k_unit(i), &kmap, en.x, n_ok);
                    }
                    if (i > 0) load(unit0 + v_unit(i - 1, ntl), &vmap, en_v.x, n_ok_v);
                }
            } else if (warp == 13) {
                // ---- scores -------------------------------------------------------------------
                bar_sync(1, kTcSoft + 32);                         // queries staged
                if (lane == 0) {
                    const uint64_t q_desc = smem_desc_sw128(base, 16, 1024);
                    const uint64_t k_desc0 = smem_desc_sw128(base + SH::OFF_RING, 16, 1024);
                    for (int i = 0; i < ntl; ++i) {
                        const uint32_t gt = tile0 + i, s = gt & 1u, s_tm = tmem + S_COL + s * 128;
                        const uint32_t kn = unit0 + k_unit(i), ks = kn % SH::UNITS;
                        if (gt >= 2) wait(&sh.o_full[s], ((gt - 2) >> 1) & 1u);  // P in these columns is read
                        wait(&sh.full[ks], (kn / SH::UNITS) & 1u);
                        tc_fence_after_sync();
                        const uint64_t kd = k_desc0 + uint64_t((ks * SH::UNIT) >> 4);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = uint32_t(((k >> 2) * SH::HALF + (k & 3) * 32) >> 4);
                            umma_bf16(s_tm, q_desc + off, kd + off, IDESC_S, k > 0 ? 1u : 0u);
                        }
                        umma_commit(&sh.s_full[s]);
                        umma_commit(&sh.empty[ks]);
                    }
                }
                __syncwarp();
            } else if (warp == 14) {
                // ---- output -------------------------------------------------------------------
                if (lane == 0) {
                    const uint64_t p_desc0 = smem_desc_sw128(base + SH::OFF_P, 16, 1024);
                    const uint64_t v_desc0 = smem_desc_sw128(base + SH::OFF_RING, SH::HALF, 1024);
                    for (int i = 0; i < ntl; ++i) {
                        const uint32_t gt = tile0 + i, s = gt & 1u;
                        const uint32_t s_tm = tmem + S_COL + s * 128, o_tm = tmem + O_COL + s * 128;
                        const uint32_t vn = unit0 + v_unit(i, ntl), vs = vn % SH::UNITS;
                        if (gt >= 2) wait(&sh.o_read[s], ((gt - 2) >> 1) & 1u);  // the last O here is added up
                        wait(&sh.p_ready[s], (gt >> 1) & 1u);
                        wait(&sh.full[vs], (vn / SH::UNITS) & 1u);
                        tc_fence_after_sync();
                        const uint64_t vd = v_desc0 + uint64_t((vs * SH::UNIT) >> 4);
                        const uint64_t pd = p_desc0 + uint64_t((s * SH::P_TILE) >> 4);
                        if (REP == 1) {                            // the small parts first
#pragma unroll
                            for (int k = 0; k < kTcTile / 16; ++k)
                                umma_bf16(o_tm, pd + uint32_t(((k >> 2) * SH::HALF + (k & 3) * 32) >> 4),
                                          vd + uint32_t((k * 16 * 128) >> 4), IDESC_O, k > 0 ? 1u : 0u);
                        }
#pragma unroll
                        for (int pp = REP < 4 ? 1 : 0; pp >= 0; --pp)
#pragma unroll
                            for (int k = 0; k < kTcTile / 16; ++k)
                                umma_bf16_ta(o_tm, s_tm + tc_part_col<REP>(k, pp), vd + uint32_t((k * 16 * 128) >> 4), IDESC_O,
                                             REP == 1 || pp < (REP < 4 ? 1 : 0) || k > 0 ? 1u : 0u);
                        umma_commit(&sh.empty[vs]);
                        umma_commit(&sh.o_full[s]);
                    }
                }
                __syncwarp();
            }
            unit0 += 2 * ntl;
            tile0 += ntl;
        }
    } else if (warp >= 8) {
        // ---- the running O: thread = row ----------------------------------------------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcRegsSum));
        constexpr int COPY = 128 / REP;
        const int row = 32 * (warp & 3) + lane;
        const uint32_t o_tm = tmem + O_COL + (uint32_t(32 * (warp & 3)) << 16);
        float* x_l = reinterpret_cast<float*>(smem);               // [half][row], by the softmax threads
        uint32_t tile0 = 0;
        while (tc_next(a, part, lo, start, item, g)) {
            const int ntl = g.t1 - g.t0;
            const int r_unit = g.row0 + row % COPY;
            const bool live = g.row0 + 32 * (warp & 3) % COPY < a.R && row / COPY < 3;   // any of this warp's rows
            F2 acc[D / 2];
#pragma unroll
            for (int d = 0; d < D / 2; ++d) acc[d] = make_f2(0.f, 0.f);
            float m_acc = -INFINITY;                               // what acc is relative to
            for (int i = 0; i < ntl; ++i) {
                const uint32_t gt = tile0 + i, sl = gt & 1u;
                wait(&sh.o_full[sl], (gt >> 1) & 1u);
                __syncwarp();
                tc_fence_after_sync();
                if (live) {
                    // the softmax's reference of this tile
                    const float m_old = __fmul_rn(m_acc, a.scale_log2);
                    m_acc = tc_reference(m_acc, sh.top[gt & 3u][row], a.scale_log2);
                    sh.top[gt & 3u][row] = kOrderedLeast;          // for the tile four on (its scores wait for o_read of this one)
                    const float w0 = m_old == -INFINITY ? 0.f : fast_exp2(m_old - __fmul_rn(m_acc, a.scale_log2));
                    if (__any_sync(kFullMask, w0 != 1.f)) {                    // rarely after the first tiles
                        const F2 w02 = make_f2(w0, w0);
#pragma unroll
                        for (int d = 0; d < D / 2; ++d) acc[d] = mul2(acc[d], w02);
                    }
#pragma unroll
                    for (int c = 0; c < D / 16; c += 2) {
                        uint32_t v[2][16];
                        tmem_ld16(o_tm + sl * 128 + 16 * c, v[0]);
                        tmem_ld16(o_tm + sl * 128 + 16 * c + 16, v[1]);
                        tmem_wait_ld16(v[0]);
                        tmem_wait_ld16(v[1]);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            acc[8 * c + j] = add2(acc[8 * c + j],
                                                  make_f2(__uint_as_float(v[j >> 3][2 * (j & 7)]), __uint_as_float(v[j >> 3][2 * (j & 7) + 1])));
                    }
                    const uint32_t info = (tile0 + i) % SH::INFO;
                    if (sh.masked[info] != 0 && (sh.odd[info][0] | sh.odd[info][1] | sh.odd[info][2] | sh.odd[info][3])) {
                        // infinities and NaN were taken out of V: the first copy adds them where they are seen
                        const int q_row = r_unit < a.R ? r_unit / a.G : 0;
                        const DraftView view = draft_view(
                            a.mask != nullptr ? a.mask + ((long long)g.b * a.Q + q_row) * a.mask_words : nullptr, a.mask_words,
                            r_unit < a.R ? (a.mask != nullptr ? a.Q : q_row + 1) : 0);
#pragma unroll 1
                        for (int j = 0; j < kTcTile; ++j) {
                            if (!((sh.odd[info][j >> 5] >> (j & 31)) & 1u)) continue;
                            if (row >= COPY) break;
                            const int p = (g.t0 + i) * kTcTile + j, e = p >> a.bs_shift;
                            if (!((tree_tokens8(a, g.un, p & ~7, e, sh.token[info][j >> a.bs_shift], view) >> (j & 7)) & 1u)) continue;
                            const uint32_t* vg = reinterpret_cast<const uint32_t*>(
                                static_cast<const uint16_t*>(a.v_pages) +
                                (size_t(tree_entry(a, g.u, g.un, e).x) * a.bs + (j & (a.bs - 1))) * D);
#pragma unroll
                            for (int x = 0; x < D / 2; ++x) {
                                const uint32_t w = vg[x];
                                if ((w & 0x7f80u) == 0x7f80u) acc[x].f.x += bf16_lo(w);
                                if ((w & 0x7f800000u) == 0x7f800000u) acc[x].f.y += bf16_hi(w);
                            }
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before_sync();
                mbar_arrive(&sh.o_read[sl]);
            }
            // ---- the part's (m, l, o) --------------------------------------------------------------
            const bool complete = g.t0 == 0 && g.t1 == g.tiles;
            tree_sync<kTcWork>();                                  // the softmax threads' sums are there
            const float l = x_l[row % COPY] + x_l[128 + row % COPY];
            const float w = !complete ? 1.f : (l == 0.f ? 0.f : 1.f / l);
            if (!complete && row < COPY && r_unit < a.R) {
                const long long slot = (long long)tree_slot(blockIdx.x, part.per, g.start) * a.item_rows + row;
                a.part_m[slot] = m_acc * a.scale_log2;
                a.part_l[slot] = l;
            }
            constexpr int V4 = D / 4;
            float4* x_row = reinterpret_cast<float4*>(smem + SH::OFF_ROWS) + row % COPY * V4;
            auto scaled = [&](int c) {
                return make_float4(acc[2 * c].f.x * w, acc[2 * c].f.y * w, acc[2 * c + 1].f.x * w, acc[2 * c + 1].f.y * w);
            };
            if (REP > 1) {                                         // the first copy adds up the others
                bar_sync(14, kTcWork - kTcSoft);                   // the sums there have been read
                if (live && row >= COPY) {
#pragma unroll
                    for (int c = 0; c < V4; ++c) x_row[(row / COPY - 1) * COPY * V4 + ((c + row) & (V4 - 1))] = scaled(c);
                }
                bar_sync(14, kTcWork - kTcSoft);
            }
            if (live && row < COPY) {
#pragma unroll
                for (int c0 = 0; c0 < V4; c0 += 4) {
                    float4 x[REP == 4 ? 2 : 1][4];
#pragma unroll
                    for (int y = 0; y < (REP == 4 ? 2 : REP - 1); ++y)
#pragma unroll
                        for (int c = 0; c < 4; ++c) x[y][c] = x_row[y * COPY * V4 + ((c0 + c + row) & (V4 - 1))];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float4 o = scaled(c0 + c);
#pragma unroll
                        for (int y = 0; y < (REP == 4 ? 2 : REP - 1); ++y)
                            o = make_float4(o.x + x[y][c].x, o.y + x[y][c].y, o.z + x[y][c].z, o.w + x[y][c].w);
                        x_row[(c0 + c + row) & (V4 - 1)] = o;
                    }
                }
            }
            tc_store_rows<D, REP>(a, part, g, smem, &sh.last, tid);
            tile0 += ntl;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcRegsSoft));
        constexpr int COPY = 128 / REP;                            // rows of a copy
        const int h = warp >> 2;                                   // which half of a tile's tokens
        const int row = 32 * (warp & 3) + lane;                    // query row of the item
        const uint32_t lanes = uint32_t(32 * (warp & 3)) << 16;
        const int pair_bar = 4 + (warp & 3);                       // the two warps that share rows
        const int copy = 32 * (warp & 3) / COPY;                   // which copy of the row: one for a whole warp
        const float scale = a.scale_log2;
        uint32_t tile0 = 0, unit0 = 0;
        sh.top[2 * h][row] = sh.top[2 * h + 1][row] = kOrderedLeast;           // before the first item's barriers
        while (tc_next(a, part, lo, start, item, g)) {
            const int ntl = g.t1 - g.t0;
            const uint32_t* mask_b = a.mask != nullptr ? a.mask + (long long)g.b * a.Q * a.mask_words : nullptr;
            // ---- the item's queries, and the drafts that some query sees ----------------
            {
                constexpr int CPR = D / 8;                         // 16-byte chunks of a row
                constexpr int N = COPY * CPR / kTcSoft;            // chunks of this thread
                const long long list = dense ? g.un.len : (long long)g.un.n_ctx << a.bs_shift;
                const bool drafts = (long long)g.t1 * kTcTile > list;               // this part meets drafts
                const int bits = mask_b != nullptr && drafts ? a.Q * a.mask_words : 0;
                const uint32_t first_bits = tid < bits ? mask_b[tid] : 0u;  // on its way with the queries
                uint4 v[N];
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    const int r = (tid + x * kTcSoft) / CPR, c = (tid + x * kTcSoft) % CPR;
                    v[x] = make_uint4(0u, 0u, 0u, 0u);
                    if (g.row0 + r < a.R)
                        v[x] = *(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                    tree_out_row(a, g.b, g.kvh, g.row0 + r) * D) + c);
                }
#pragma unroll
                for (int x = 0; x < N; ++x) {
                    const int r = (tid + x * kTcSoft) / CPR, c = (tid + x * kTcSoft) % CPR;
#pragma unroll
                    for (int y = 0; y < REP; ++y)
                        *reinterpret_cast<uint4*>(smem + (c >> 3) * SH::HALF + (r + y * COPY) * 128 +
                                                  (((c & 7) ^ (r & 7)) << 4)) = v[x];
                }
                if (drafts) {
                    if (tid < a.mask_words) sh.any[tid] = mask_b == nullptr ? ~0u : 0u;
                    if (mask_b != nullptr) {
                        bar_sync(15, kTcSoft);
                        if (tid < bits) atomicOr(&sh.any[tid % a.mask_words], first_bits);
                        for (int i = tid + kTcSoft; i < bits; i += kTcSoft) atomicOr(&sh.any[i % a.mask_words], mask_b[i]);
                    }
                }
                fence_proxy_async_smem();                          // before the tensor core uses this memory
            }
            bar_sync(1, kTcSoft + 32);

            const int r_unit = g.row0 + row % COPY;
            const bool live = g.row0 + 32 * (warp & 3) % COPY < a.R && row / COPY < 3;   // any of this warp's rows
            const int q_row = r_unit < a.R ? r_unit / a.G : 0;
            // what the row sees of the drafts, and what any query sees
            const uint32_t* words = mask_b != nullptr ? mask_b + (long long)q_row * a.mask_words : nullptr;
            const DraftView view = draft_view(words, a.mask_words, r_unit < a.R ? (mask_b != nullptr ? a.Q : q_row + 1) : 0);
            float reference = -INFINITY, l_run = 0.f;              // the row's, the half-row's sum

            // Tokens 8 g8 .. + 7 of local tile i that a query with this view sees.
            auto tokens8 = [&](int i, int g8, const DraftView& v) -> uint32_t {
                const int le = (g8 * 8) >> a.bs_shift;
                return tree_tokens8(a, g.un, g8 * 8, (((g.t0 + i) * kTcTile) >> a.bs_shift) + le,
                                    sh.token[(tile0 + i) % SH::INFO][le], v);
            };
            for (int i = 0; i < ntl; ++i) {
                const uint32_t gt = tile0 + i, s = gt & 1u;
                const uint32_t s_tm = tmem + S_COL + s * 128 + 64 * h + lanes;
                unsigned char* p_row = smem + SH::OFF_P + s * SH::P_TILE + h * SH::HALF + row * 128;
                wait(&sh.s_full[s], (gt >> 1) & 1u);
                __syncwarp();
                tc_fence_after_sync();
                const uint32_t info = (tile0 + i) % SH::INFO;
                if (sh.masked[info] != 0) {
                    // Scores of tokens that the row does not see become -infinity.  V rows of tokens
                    // that nobody sees are zeroed (their memory may hold anything), and so are
                    // infinities and NaN of drafts, which are added back where they are seen.
                    if (live) {
#pragma unroll 1
                        for (int c = 0; c < 4; ++c) {
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
                    const uint32_t vn = unit0 + v_unit(i, ntl), vs = vn % SH::UNITS;
                    wait(&sh.full[vs], (vn / SH::UNITS) & 1u);
                    // the two threads of number `row` look after token `row`, half its channels each
                    constexpr int CHUNKS = SH::HALVES * 4;
                    unsigned char* vrow = smem + SH::OFF_RING + vs * SH::UNIT + row * 128;
                    const bool seen = (tokens8(i, row >> 3, draft_view(sh.any, a.mask_words, a.Q)) >> (row & 7)) & 1u;
                    const int first = sh.token[info][row >> a.bs_shift];
                    const bool draft = first != kNoToken && first + (row & (a.bs - 1)) >= g.un.len;
                    bool changed = false;
                    for (int c = h * CHUNKS; c < (h + 1) * CHUNKS && (!seen || draft); ++c) {
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
                    uint32_t v[4][16];
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld16(s_tm + 16 * c, v[c]);
                    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        tmem_wait_ld16(v[c]);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            x0 = max3(x0, __uint_as_float(v[c][j]), __uint_as_float(v[c][j + 1]));
                            x1 = max3(x1, __uint_as_float(v[c][j + 2]), __uint_as_float(v[c][j + 3]));
                        }
                    }
                    int* top = &sh.top[gt & 3u][row];
                    atomicMax(top, ordered_bits(__float_as_int(fmaxf(x0, x1))));
                    bar_sync(pair_bar, 64);
                    const float m_old = __fmul_rn(reference, scale);
                    reference = tc_reference(reference, *reinterpret_cast<volatile int*>(top), scale);
                    const float m_new = __fmul_rn(reference, scale);
                    l_run *= m_old == -INFINITY ? 0.f : fast_exp2(m_old - m_new);
                    // ---- the weights, in three bf16 parts, over the scores' own columns -----------
                    const float factor = tc_large(m_new) ? tc_power(reference) : scale;
                    const float m_sub = m_new == -INFINITY ? 0.f : __fmul_rn(reference, factor);   // -infinity: every weight is 0
                    const F2 scale2 = make_f2(factor, factor), m2 = make_f2(-m_sub, -m_sub);
                    F2 sum_a = make_f2(0.f, 0.f), sum_b = make_f2(0.f, 0.f);
                    auto weight = [&](uint32_t (&x)[16], int j) {
                        const F2 p = fma2(make_f2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), scale2, m2);
                        return make_f2(fast_exp2(p.f.x), fast_exp2(p.f.y));
                    };
                    auto add = [&](F2 p, int j) {
                        if (j & 1) sum_b = add2(sum_b, p);
                        else sum_a = add2(sum_a, p);
                    };
                    uint32_t u[16];
                    if (REP == 1) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t small[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                F2 p = weight(v[c], j);
                                add(p, j);
                                u[j] = cut_bf16x2(p);
                                u[8 + j] = cut_bf16x2(p);
                                small[j] = top_bf16x2(p);
                            }
                            tmem_st16(s_tm + 16 * c, u);
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                *reinterpret_cast<uint4*>(p_row + (((2 * c + x) ^ (row & 7)) << 4)) =
                                    make_uint4(small[4 * x], small[4 * x + 1], small[4 * x + 2], small[4 * x + 3]);
                        }
                    } else if (copy == 0) {                        // the first part, and the row's sum
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const F2 p = weight(v[c], j);
                                add(p, j);
                                u[(c & 1) * 8 + j] = top_bf16x2(p);
                            }
                            if (c & 1) tmem_st16(s_tm + 8 * (c - 1), u);
                        }
                        if (REP == 2) {                            // none of the third
#pragma unroll
                            for (int j = 0; j < 16; ++j) u[j] = 0u;
                            tmem_st16(s_tm + 32, u);
                            tmem_st16(s_tm + 48, u);
                        }
                    } else {                                       // the second, the third
                        const uint32_t mid = REP == 4 && copy == 2 ? 0xffff0000u : 0u;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            uint32_t small[16];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                F2 p = weight(v[c], j);
                                cut_bf16x2(p);
                                if (REP == 2) {
                                    u[(c & 1) * 8 + j] = cut_bf16x2(p);
                                    v[c][j] = top_bf16x2(p);       // (its scores are done with)
                                } else {
                                    u[(c & 1) * 8 + j] = top_bf16x2(less(p, mid));
                                }
                            }
                            if (c & 1) tmem_st16(s_tm + 8 * (c - 1), u);
                            if (REP == 2 && (c & 1)) {
#pragma unroll
                                for (int j = 0; j < 16; ++j) small[j] = v[c - 1 + (j >> 3)][j & 7];
                                tmem_st16(s_tm + 32 + 8 * (c - 1), small);
                            }
                        }
                    }
                    const F2 sum = add2(sum_a, sum_b);
                    l_run += sum.f.x + sum.f.y;
                    tmem_wait_st();
                    fence_proxy_async_smem();
                }
                tc_fence_before_sync();
                mbar_arrive(&sh.p_ready[s]);
            }
            // the row's sums, through the query tile, which nothing reads after the last scores
            reinterpret_cast<float*>(smem)[h * 128 + row] = l_run;
            tree_sync<kTcWork>();
            tc_store_rows<D, REP>(a, part, g, smem, &sh.last, tid);
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
                                    int(tc_smem<D, REP>()));
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
    e = launch_after_previous(tree_tc_kernel<D, REP>, dim3(unsigned(ctas)), dim3(kTcThreads), tc_smem<D, REP>(), s, a, kmap, vmap);
    return e == cudaSuccess && a.combine ? launch_tree_combine(a, s) : e;
}

}  // namespace

cudaError_t launch_tree_tc(TreeArgs a, cudaStream_t s)
{
    a.tile = kTcTile;
    a.merge_scale = 1.f;           // maxima are scaled
    a.item_rows = tree_item_rows(a.R);
    a.row_groups = (a.R + a.item_rows - 1) / a.item_rows;
    // 128 rows over 777 tokens 19.6 us, with parts of at least 1 tile 20.4, of 4 35.4; an item's start and
    // end take about as long as six tiles.
    a.min_per = 2;
    a.half_slack = 3;
    if (a.R <= 32) return a.D == 128 ? launch_tc_t<128, 4>(a, s) : launch_tc_t<64, 4>(a, s);
    if (a.R <= 64) return a.D == 128 ? launch_tc_t<128, 2>(a, s) : launch_tc_t<64, 2>(a, s);
    return a.D == 128 ? launch_tc_t<128, 1>(a, s) : launch_tc_t<64, 1>(a, s);
}

}  // namespace sa
