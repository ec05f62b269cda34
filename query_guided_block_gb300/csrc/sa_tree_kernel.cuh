// The draft-tree attention kernel on warp-level matrix instructions (described in sa_tree.cu), and its
// EXT form for the units of shared prefixes and for weighed attention (sa_shared.cu, sa_weigh.cu).
#pragma once

#include "sa_tree.cuh"

namespace sa {

constexpr int kTrThreads = 128;
constexpr int kTrTile = 64;
constexpr uint32_t kNotSeen = 0xffffffffu;   // score of a token that the row does not see: a NaN that no product gives
constexpr int kTrEntries = 512;      // list entries resolved at a time
constexpr int kTrInfo = 4;           // tiles looked up ahead of their copies, at least the stages + 1

__device__ __forceinline__ void mma_tf32_1688(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t to_tf32(float x)
{
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo)
{
    hi = to_tf32(x);
    lo = to_tf32(x - __uint_as_float(hi));
}

// A pair of fp32 cut to bf16 (the upper halves of the words; the first in the low half), the
// remainders left behind: three cuts hold the 24 bits of an fp32 exactly.
__device__ __forceinline__ uint32_t cut_bf16x2(float& x, float& y)
{
    const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
    x -= __uint_as_float(ux & 0xffff0000u);
    y -= __uint_as_float(uy & 0xffff0000u);
    return __byte_perm(ux, uy, 0x7632);
}

template <int D, bool KB>
struct TrShape {
    static constexpr int ROW = D * (KB ? 2 : 4);            // bytes of a token row
    static constexpr int CPR = ROW / 16;                    // 16-byte chunks
    static constexpr int TENSOR = kTrTile * ROW;
    static constexpr int STAGE = 2 * TENSOR;
    static constexpr int STAGES = STAGE > 32768 ? 2 : 3;    // 64 to 96 KB of tiles (fp32, D = 128: 128 KB)
    static constexpr int Q_ROW = D + 8;                     // floats of a query row (fp32 K/V)
    // Chunk c of token row r.  bf16: 128-byte groups, c ^ (r mod 8) (ldmatrix reads 8 rows).
    // fp32: a fragment load touches 4 rows x 2 chunks; f takes 4 values over rows 0-3 and
    // 4-7 (keys) and over the even and the odd rows (values).
    static __device__ __forceinline__ uint32_t at(int r, int c)
    {
        if constexpr (KB) {
            return uint32_t((c >> 3) * (kTrTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
        } else {
            const int f = (r ^ (r >> 2)) & 3;
            return uint32_t(r * ROW + ((c ^ (f << 1)) << 4));
        }
    }
};

template <int D, bool KB, int NQ, int RW, bool EXT>
__global__ void __launch_bounds__(kTrThreads, 2) tree_kernel(TreeArgs a)
{
    using SH = TrShape<D, KB>;
    constexpr int TW = 4 / RW;                // warps that split a tile's tokens
    constexpr int NT = 8 / TW;                // 8-token groups per warp
    constexpr int DT = D / 8;
    constexpr int ROWS = 16 * RW;
    constexpr int CPT = kTrTile * SH::CPR / kTrThreads;     // chunks a thread copies per tensor

    extern __shared__ __align__(128) unsigned char smem_raw[];
    __shared__ int2 s_ent[kTrEntries];
    __shared__ long long s_src[kTrInfo][kTrTile];           // a tile's token rows in the pools, -1: none
    __shared__ uint32_t s_part[kTrInfo][2];                 // a tile's halves: 1 not only context tokens, 2 drafts
    __shared__ uint32_t s_see[ROWS][2];                     // tokens of the tile that a row sees
    __shared__ uint32_t s_any[kTreeMaxDrafts / 32];         // drafts that some query sees
    __shared__ int s_scan[kTreeScan<kTrThreads>];
    __shared__ int s_last;
    __shared__ uint32_t s_bad[2];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g4 = lane >> 2, t4 = lane & 3;
    const int wr = warp % RW, wt = warp / RW;                      // the warp's rows / tokens
    unsigned char* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
    const uint32_t base = smem_u32(smem);
    float* s_q = reinterpret_cast<float*>(smem + SH::STAGES * SH::STAGE);   // fp32 K/V: [ROWS][Q_ROW]

    allow_dependents_early();
    grid_dependency_wait();   // queries, pages and lengths may come from the previous kernel,
                              // so nothing of them is read through the read-only cache

    const TreePart part = tree_part<kTrThreads, EXT>(a, s_scan);
    if constexpr (EXT) tree_note_sequences(a, kTrThreads);
    const bool dense = EXT || a.sel_ids == nullptr;
    int lo = part.lo, start = part.start, item = part.item;

    while (lo < part.hi) {
        const int u = item / a.row_groups, rg = item - u * a.row_groups;
        const int kvh = u % a.Hkv;
        const TreeUnit un = tree_unit<EXT>(a, u);
        const int b = EXT ? un.b0 : u / a.Hkv;
        const int R = EXT ? un.rows : a.R;                   // query rows of the unit
        const int tiles = tree_tiles<EXT>(a, un);
        if (tiles == 0) {
            item = tree_next_item<EXT>(a, un, item);
            continue;
        }
        const int t0 = lo - start, t1 = part.whole ? tiles : min(tiles, part.hi - start);
        const int row0 = rg * ROWS;                          // first unit row of the item
        const uint32_t* mask_b = a.mask != nullptr ? a.mask + (long long)b * a.Q * a.mask_words : nullptr;

        __syncthreads();                                     // the previous item is done with shared memory
        const long long list = EXT ? un.len - (un.first_blk << a.bs_shift)
                                   : (dense ? un.len : (long long)un.n_ctx << a.bs_shift);
        if ((long long)t1 * kTrTile > list && (!EXT || un.drafts > 0)) {     // this part meets drafts
            if (tid < a.mask_words) s_any[tid] = mask_b == nullptr ? ~0u : 0u;
            __syncthreads();
            if (mask_b != nullptr)
                for (int i = tid; i < a.Q * a.mask_words; i += kTrThreads) atomicOr(&s_any[i % a.mask_words], mask_b[i]);
        }

        // ---- the queries: A fragments in registers, or fp32 rows in shared memory -------
        const int r_lo = row0 + wr * 16 + g4, r_hi = r_lo + 8;
        uint32_t qa[KB ? NQ : 1][KB ? D / 16 : 1][4];
        if constexpr (KB) {
            const size_t at_lo = r_lo < R ? size_t(tree_out_row(a, b, kvh, r_lo)) * D + 2 * t4 : 0;
            const size_t at_hi = r_hi < R ? size_t(tree_out_row(a, b, kvh, r_hi)) * D + 2 * t4 : 0;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
                for (int hc = 0; hc < 4; ++hc) {             // a0, a1: k 0-7 of rows lo, hi; a2, a3: k 8-15
                    const bool have = ((hc & 1) ? r_hi : r_lo) < R;
                    const size_t at = ((hc & 1) ? at_hi : at_lo) + ks * 16 + (hc >> 1) * 8;
                    if constexpr (NQ == 1) {
                        qa[0][ks][hc] = have ? *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + at) : 0u;
                    } else {
                        float2 f = have ? *reinterpret_cast<const float2*>(static_cast<const float*>(a.q) + at)
                                        : make_float2(0.f, 0.f);
#pragma unroll
                        for (int part_q = 0; part_q < NQ; ++part_q) qa[part_q][ks][hc] = cut_bf16x2(f.x, f.y);
                    }
                }
        } else {
#pragma unroll
            for (int i = tid; i < ROWS * (D / 4); i += kTrThreads) {
                const int rr = i / (D / 4), d = (i - rr * (D / 4)) * 4;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row0 + rr < R) {
                    const size_t at = size_t(tree_out_row(a, b, kvh, row0 + rr)) * D + d;
                    if (a.q_bf16) {
                        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at);
                        x = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
                    } else {
                        x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + at);
                    }
                }
                float* dst = s_q + rr * SH::Q_ROW + d;
                dst[0] = x.x;
                dst[1] = x.y;
                dst[2] = x.z;
                dst[3] = x.w;
            }
        }

        float acc[DT][4];
#pragma unroll
        for (int j = 0; j < DT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};

        const int step = ((kTrEntries - 1) << a.bs_shift) / kTrTile;      // tiles whose entries fit s_ent
        for (int ca = t0; ca < t1; ca += step) {
            const int cb = min(t1, ca + step);
            const int e0 = (ca * kTrTile) >> a.bs_shift;
            const int e1 = min(un.n_entries, ((cb * kTrTile - 1) >> a.bs_shift) + 1);
            __syncthreads();
            for (int e = e0 + tid; e < e1; e += kTrThreads) s_ent[e - e0] = tree_entry<EXT>(a, u, un, e);
            __syncthreads();

            // Where the rows of a tile's tokens are, by two warps a tile: tokens that nobody sees get
            // no row (their memory may hold anything).
            auto look_up = [&](int tile, int tr) {
                const int p = tile * kTrTile + tr, e = p >> a.bs_shift;
                const int2 en = e < e1 ? s_ent[e - e0] : make_int2(-1, 0);
                const int tok = en.y + (p & (a.bs - 1)), draft = tok - un.len;
                const bool in_ctx = en.x >= 0 && draft < 0 && (dense || e < un.n_ctx) && (!EXT || tok >= un.from);
                const bool is_draft = en.x >= 0 && draft >= 0 && draft < (EXT ? un.drafts : a.Q) && (dense || e >= un.n_ctx);
                const bool row = in_ctx || (is_draft && ((s_any[draft >> 5] >> (draft & 31)) & 1u));
                s_src[tile % kTrInfo][tr] = row ? (long long)en.x * a.bs + (p & (a.bs - 1)) : -1;
                const uint32_t part_of = __any_sync(kFullMask, !in_ctx) | (__any_sync(kFullMask, is_draft) << 1);
                if ((tr & 31) == 0) s_part[tile % kTrInfo][tr >> 5] = part_of;
            };
            const int cp_c = tid % SH::CPR, cp_r = tid / SH::CPR;
            const char* kp = static_cast<const char*>(a.k_pages) + cp_c * 16;
            const char* vp = static_cast<const char*>(a.v_pages) + cp_c * 16;
            auto issue_tile = [&](int tile, int st) {
                const uint32_t kd = base + uint32_t(st) * SH::STAGE, vd = kd + SH::TENSOR;
#pragma unroll
                for (int i = 0; i < CPT; ++i) {
                    const int tr = cp_r + i * (kTrThreads / SH::CPR);
                    const long long src = s_src[tile % kTrInfo][tr];
                    const size_t off = src < 0 ? 0 : size_t(src) * SH::ROW;
                    cp_async_16_zfill(kd + SH::at(tr, cp_c), kp + off, src < 0 ? 0u : 16u);
                    cp_async_16_zfill(vd + SH::at(tr, cp_c), vp + off, src < 0 ? 0u : 16u);
                }
            };
            for (int kk = tid >> 6; kk < SH::STAGES; kk += 2) look_up(ca + kk, tid & 63);
            __syncthreads();
#pragma unroll 1
            for (int kk = 0; kk < SH::STAGES - 1; ++kk) {
                if (ca + kk < cb) issue_tile(ca + kk, kk);
                cp_async_commit();
            }

            for (int tile = ca; tile < cb; ++tile) {
                const int k = tile - ca;
                cp_async_wait_group<SH::STAGES - 2>();
                __syncthreads();          // tile k is staged; stage k - 1 is free
                if (tile + SH::STAGES - 1 < cb) issue_tile(tile + SH::STAGES - 1, (k + SH::STAGES - 1) % SH::STAGES);
                cp_async_commit();
                if (tid < kTrTile) look_up(tile + SH::STAGES, tid);
                unsigned char* stage = smem + (k % SH::STAGES) * SH::STAGE;
                const uint32_t kst = base + uint32_t(k % SH::STAGES) * SH::STAGE, vst = kst + SH::TENSOR;
                const uint32_t parts = s_part[tile % kTrInfo][0] | s_part[tile % kTrInfo][1];
                const bool whole = (parts & 1u) == 0u, drafts = (parts & 2u) != 0u;
                if (!whole) {
                    for (int i = tid; i < ROWS * 2; i += kTrThreads) {
                        const int r = row0 + (i >> 1), t = r / a.G;
                        const DraftView view = draft_view(
                            mask_b != nullptr && r < R && (!EXT || un.drafts > 0) ? mask_b + (long long)t * a.mask_words : nullptr,
                            a.mask_words, r >= R || (EXT && un.drafts == 0) ? 0 : (mask_b != nullptr ? a.Q : t + 1));
                        uint32_t bits = 0u;
#pragma unroll 1
                        for (int x = 0; x < 4; ++x) {
                            const int p = tile * kTrTile + 32 * (i & 1) + 8 * x, e = p >> a.bs_shift;
                            const int2 en = e < e1 ? s_ent[e - e0] : make_int2(-1, 0);
                            bits |= tree_tokens8<EXT>(a, un, p, e, en.x < 0 ? kNoToken : en.y, view) << (8 * x);
                        }
                        s_see[i >> 1][i & 1] = bits;
                    }
                    __syncthreads();
                }

                // A draft's V may hold infinities or NaN that other queries must not meet as
                // 0 * inf: such rows are taken out of the product and added where they are seen.
                uint32_t bad0 = 0u, bad1 = 0u;
                if (drafts) {
                    if (tid < 2) s_bad[tid] = 0u;
                    __syncthreads();
                    for (int i = tid; i < kTrTile * SH::CPR; i += kTrThreads) {
                        const int tr = i / SH::CPR;
                        const uint4 v = *reinterpret_cast<const uint4*>(stage + SH::TENSOR + SH::at(tr, i - tr * SH::CPR));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        bool odd = false;
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            odd |= (w[x] & 0x7f800000u) == 0x7f800000u;
                            if constexpr (KB) odd |= (w[x] & 0x7f80u) == 0x7f80u;
                        }
                        if (odd) atomicOr(&s_bad[tr >> 5], 1u << (tr & 31));
                    }
                    __syncthreads();
                    bad0 = s_bad[0];
                    bad1 = s_bad[1];
                    if (bad0 | bad1) {
                        for (int i = tid; i < kTrTile * SH::CPR; i += kTrThreads) {
                            const int tr = i / SH::CPR;
                            if (((tr < 32 ? bad0 : bad1) >> (tr & 31)) & 1u)
                                *reinterpret_cast<uint4*>(stage + SH::TENSOR + SH::at(tr, i - tr * SH::CPR)) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                        __syncthreads();
                    }
                }

                // ---- S = Q K^T ------------------------------------------------------
                float c[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
                const int tok0 = wt * NT * 8;                // the warp's first token of the tile
                if constexpr (KB) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int kp2 = 0; kp2 < D / 32; ++kp2) {
                            uint32_t b0, b1, b2, b3;
                            ldsm_x4(kst + SH::at(tok0 + nt * 8 + (lane & 7), kp2 * 4 + (lane >> 3)), b0, b1, b2, b3);
#pragma unroll
                            for (int pq = NQ - 1; pq >= 0; --pq) {
                                mma_bf16_16816(c[nt], qa[pq][2 * kp2][0], qa[pq][2 * kp2][1], qa[pq][2 * kp2][2],
                                               qa[pq][2 * kp2][3], b0, b1);
                                mma_bf16_16816(c[nt], qa[pq][2 * kp2 + 1][0], qa[pq][2 * kp2 + 1][1],
                                               qa[pq][2 * kp2 + 1][2], qa[pq][2 * kp2 + 1][3], b2, b3);
                            }
                        }
                } else {
                    float cs[NT][4];                         // the small products, apart
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) cs[nt][0] = cs[nt][1] = cs[nt][2] = cs[nt][3] = 0.f;
#pragma unroll 2
                    for (int ks = 0; ks < D / 8; ++ks) {
                        const float* q0 = s_q + (wr * 16 + g4) * SH::Q_ROW + ks * 8 + 2 * t4;
                        const float2 x = *reinterpret_cast<const float2*>(q0);
                        const float2 y = *reinterpret_cast<const float2*>(q0 + 8 * SH::Q_ROW);
                        uint32_t ah[4], al[4];
                        split_tf32(x.x, ah[0], al[0]);
                        split_tf32(y.x, ah[1], al[1]);
                        split_tf32(x.y, ah[2], al[2]);
                        split_tf32(y.y, ah[3], al[3]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int tr = tok0 + nt * 8 + g4;
                            const float2 kf = *reinterpret_cast<const float2*>(stage + SH::at(tr, ks * 2 + (t4 >> 1)) + (t4 & 1) * 8);
                            uint32_t bh0, bl0, bh1, bl1;
                            split_tf32(kf.x, bh0, bl0);
                            split_tf32(kf.y, bh1, bl1);
                            mma_tf32_1688(cs[nt], al, bh0, bh1);
                            mma_tf32_1688(cs[nt], ah, bl0, bl1);
                            mma_tf32_1688(c[nt], ah, bh0, bh1);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) c[nt][e] += cs[nt][e];
                }
                // ---- scale, mask, running maximum and sum ---------------------------------
                float mx[2] = {-INFINITY, -INFINITY};
                uint32_t see[2][(NT + 3) / 4];               // this warp's tokens, rows lo and hi
#pragma unroll
                for (int w = 0; w < (NT + 3) / 4; ++w) see[0][w] = see[1][w] = ~0u;
                if (!whole) {
#pragma unroll
                    for (int w = 0; w < (NT + 3) / 4; ++w) {
                        see[0][w] = s_see[wr * 16 + g4][(tok0 >> 5) + w] >> (tok0 & 31);
                        see[1][w] = s_see[wr * 16 + g4 + 8][(tok0 >> 5) + w] >> (tok0 & 31);
                    }
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const bool ok0 = (see[0][nt / 4] >> ((nt & 3) * 8 + 2 * t4 + e)) & 1u;
                        const bool ok1 = (see[1][nt / 4] >> ((nt & 3) * 8 + 2 * t4 + e)) & 1u;
                        c[nt][e] = ok0 ? c[nt][e] : __uint_as_float(kNotSeen);
                        c[nt][e + 2] = ok1 ? c[nt][e + 2] : __uint_as_float(kNotSeen);
                        mx[0] = fmaxf(mx[0], c[nt][e]);
                        mx[1] = fmaxf(mx[1], c[nt][e + 2]);
                    }
                if constexpr (EXT) {
                    if (a.scores != nullptr) {               // for the sums of weights, once every row's total is known
                        float* at = a.scores + ((long long)u * a.R + r_lo) * a.score_stride + tile * kTrTile + tok0 + 2 * t4;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (r_lo < R) *reinterpret_cast<float2*>(at + nt * 8) = make_float2(c[nt][0], c[nt][1]);
                            if (r_hi < R)
                                *reinterpret_cast<float2*>(at + 8 * a.score_stride + nt * 8) = make_float2(c[nt][2], c[nt][3]);
                        }
                    }
                }
                float alpha[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFullMask, mx[h], 1));
                    mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFullMask, mx[h], 2));
                    const float m_new = fmaxf(m_run[h], mx[h]);
                    alpha[h] = (m_run[h] == -INFINITY) ? 0.f : fast_exp2((m_run[h] - m_new) * a.scale_log2);
                    m_run[h] = m_new;
                }
                // (score - maximum) * scale, in that order: a rounded product would be off by its own size.
                float psum[2] = {0.f, 0.f};
                const F2 scale2 = make_f2(a.scale_log2, a.scale_log2);
                const float sub[2] = {m_run[0] == -INFINITY ? 0.f : -m_run[0], m_run[1] == -INFINITY ? 0.f : -m_run[1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float &x = c[nt][2 * h], &y = c[nt][2 * h + 1];
                        const F2 d = mul2(add2(make_f2(x, y), make_f2(sub[h], sub[h])), scale2);
                        x = __float_as_uint(x) == kNotSeen ? -0.f : fast_exp2(d.f.x);
                        y = __float_as_uint(y) == kNotSeen ? -0.f : fast_exp2(d.f.y);
                        psum[h] += x;
                        psum[h] += y;
                    }
                l_run[0] = fmaf(l_run[0], alpha[0], psum[0]);
                l_run[1] = fmaf(l_run[1], alpha[1], psum[1]);
                // ---- O = alpha O + P V ---------------------------------------------------
                auto join = [&](float (&o)[4], const float (&x)[4]) {
                    o[0] = fmaf(o[0], alpha[0], x[0]);
                    o[1] = fmaf(o[1], alpha[0], x[1]);
                    o[2] = fmaf(o[2], alpha[1], x[2]);
                    o[3] = fmaf(o[3], alpha[1], x[3]);
                };
                if constexpr (KB) {
                    uint32_t pa[3][NT / 2][4];               // parts of P as A fragments, 16 tokens each
#pragma unroll
                    for (int kk = 0; kk < NT / 2; ++kk)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            float p0 = c[2 * kk + (x >> 1)][2 * (x & 1)], p1 = c[2 * kk + (x >> 1)][2 * (x & 1) + 1];
#pragma unroll
                            for (int pp = 0; pp < 3; ++pp) pa[pp][kk][x] = cut_bf16x2(p0, p1);
                        }
#pragma unroll
                    for (int jp = 0; jp < DT; jp += 2) {
                        const int mtx = lane >> 3;
                        float x0[4] = {0.f, 0.f, 0.f, 0.f}, x1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int kk = 0; kk < NT / 2; ++kk) {
                            uint32_t v0, v1, v2, v3;
                            ldsm_x4_trans(vst + SH::at(tok0 + kk * 16 + (mtx & 1) * 8 + (lane & 7), jp + (mtx >> 1)), v0, v1,
                                          v2, v3);
#pragma unroll
                            for (int pp = 2; pp >= 0; --pp) {
                                mma_bf16_16816(x0, pa[pp][kk][0], pa[pp][kk][1], pa[pp][kk][2], pa[pp][kk][3], v0, v1);
                                mma_bf16_16816(x1, pa[pp][kk][0], pa[pp][kk][1], pa[pp][kk][2], pa[pp][kk][3], v2, v3);
                            }
                        }
                        join(acc[jp], x0);
                        join(acc[jp + 1], x1);
                    }
                } else {
                    uint32_t ah[NT][4], al[NT][4];           // k index t4 <-> token 2 t4, t4 + 4 <-> 2 t4 + 1
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        split_tf32(c[nt][0], ah[nt][0], al[nt][0]);
                        split_tf32(c[nt][2], ah[nt][1], al[nt][1]);
                        split_tf32(c[nt][1], ah[nt][2], al[nt][2]);
                        split_tf32(c[nt][3], ah[nt][3], al[nt][3]);
                    }
                    const unsigned char* vs = stage + SH::TENSOR;
#pragma unroll
                    for (int j = 0; j < DT; ++j) {
                        const int ch = j * 2 + (g4 >> 2), by = (g4 & 3) * 4;
                        float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const int tr = tok0 + nt * 8 + 2 * t4;
                            const float v0 = *reinterpret_cast<const float*>(vs + SH::at(tr, ch) + by);
                            const float v1 = *reinterpret_cast<const float*>(vs + SH::at(tr + 1, ch) + by);
                            uint32_t bh0, bl0, bh1, bl1;
                            split_tf32(v0, bh0, bl0);
                            split_tf32(v1, bh1, bl1);
                            mma_tf32_1688(x, al[nt], bh0, bh1);
                            mma_tf32_1688(x, ah[nt], bl0, bl1);
                            mma_tf32_1688(x, ah[nt], bh0, bh1);
                        }
                        join(acc[j], x);
                    }
                }
                if (bad0 | bad1) {                           // rows taken out above, where they are seen (their
                                                             // weight may be 0; those not seen have -0)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll 1
                        for (int x = 0; x < 8; ++x) {
                            const int tr = tok0 + nt * 8 + x;
                            if (!(((tr < 32 ? bad0 : bad1) >> (tr & 31)) & 1u)) continue;
                            const float p0 = __shfl_sync(kFullMask, (x & 1) ? c[nt][1] : c[nt][0], (lane & ~3) | (x >> 1));
                            const float p1 = __shfl_sync(kFullMask, (x & 1) ? c[nt][3] : c[nt][2], (lane & ~3) | (x >> 1));
                            const size_t at = size_t(s_src[tile % kTrInfo][tr]) * D;
#pragma unroll
                            for (int j = 0; j < DT; ++j)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float v = load_q(a.v_pages, at + j * 8 + 2 * t4 + e, KB);
                                    if (!signbit(p0)) acc[j][e] = fmaf(p0, v, acc[j][e]);
                                    if (!signbit(p1)) acc[j][2 + e] = fmaf(p1, v, acc[j][2 + e]);
                                }
                        }
                }
            }
            cp_async_wait_group<0>();
        }

        // ---- the part's (m, l, o): the output itself, or a partial ---------------------
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l_run[h] += __shfl_xor_sync(kFullMask, l_run[h], 1);
            l_run[h] += __shfl_xor_sync(kFullMask, l_run[h], 2);
        }
        float* out = EXT && a.pass == kTreeBoth && !un.prefix ? a.own_out : a.out;
        const bool complete = t0 == 0 && t1 == tiles, done = complete && (!EXT || a.pass == kTreeAll);
        const long long slot = (long long)tree_slot(blockIdx.x, part.per, start) * a.item_rows;
        if constexpr (TW == 1) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = h ? r_hi : r_lo, rr = r - row0;
                if (r >= R) continue;
                const float inv = done ? (l_run[h] == 0.f ? 0.f : 1.f / l_run[h]) : 1.f;
                float* dst = (complete ? out + tree_out_row(a, b, kvh, r) * D : a.part_o + (slot + rr) * D) + 2 * t4;
#pragma unroll
                for (int j = 0; j < DT; ++j)
                    *reinterpret_cast<float2*>(dst + j * 8) = make_float2(acc[j][2 * h] * inv, acc[j][2 * h + 1] * inv);
                if (!complete && t4 == 0) {
                    a.part_m[slot + rr] = m_run[h];
                    a.part_l[slot + rr] = l_run[h];
                }
                if (EXT && complete && t4 == 0) tree_note_row(a, un, tree_out_row(a, b, kvh, r), done, m_run[h], l_run[h], inv);
            }
        } else {
            // the warps' token shares of the same rows, through the freed stages
            float* x_o = reinterpret_cast<float*>(smem);                 // [TW][ROWS][D + 4]
            float* x_m = x_o + TW * ROWS * (D + 4);                      // [TW][ROWS]
            float* x_l = x_m + TW * ROWS;
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int rr = wt * ROWS + wr * 16 + g4 + 8 * h;
                float* dst = x_o + rr * (D + 4) + 2 * t4;
#pragma unroll
                for (int j = 0; j < DT; ++j) *reinterpret_cast<float2*>(dst + j * 8) = make_float2(acc[j][2 * h], acc[j][2 * h + 1]);
                if (t4 == 0) {
                    x_m[rr] = m_run[h];
                    x_l[rr] = l_run[h];
                }
            }
            __syncthreads();
            for (int i = tid; i < ROWS * (D / 4); i += kTrThreads) {
                const int rr = i / (D / 4), d = (i - rr * (D / 4)) * 4;
                if (row0 + rr >= R) continue;
                float M = -INFINITY;
#pragma unroll
                for (int w = 0; w < TW; ++w) M = fmaxf(M, x_m[w * ROWS + rr]);
                float den = 0.f;
                float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < TW; ++w) {
                    const float mw = x_m[w * ROWS + rr];
                    const float wgt = tree_share(mw, M, x_l[w * ROWS + rr], a.scale_log2);
                    den = fmaf(x_l[w * ROWS + rr], wgt, den);
                    const float4 o = *reinterpret_cast<const float4*>(x_o + (w * ROWS + rr) * (D + 4) + d);
                    num.x = fmaf(o.x, wgt, num.x);
                    num.y = fmaf(o.y, wgt, num.y);
                    num.z = fmaf(o.z, wgt, num.z);
                    num.w = fmaf(o.w, wgt, num.w);
                }
                const float inv = done ? (den == 0.f ? 0.f : 1.f / den) : 1.f;
                float* dst = complete ? out + tree_out_row(a, b, kvh, row0 + rr) * D : a.part_o + (slot + rr) * D;
                *reinterpret_cast<float4*>(dst + d) = make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
                if (!complete && d == 0) {
                    a.part_m[slot + rr] = M;
                    a.part_l[slot + rr] = den;
                }
                if (EXT && complete && d == 0) tree_note_row(a, un, tree_out_row(a, b, kvh, row0 + rr), done, M, den, inv);
            }
        }
        if constexpr (EXT) {
            if (tid == 0 && t0 == 0) tree_note(a, u, un, rg) = tree_parts(start, tiles, part.per);
        } else if (a.combine) {
            if (tid == 0 && t0 == 0) tree_note_parts(a, item, start, tiles, part.per);
        } else if (!complete) {
            tree_arrive_and_merge<kTrThreads>(a, item, start, tiles, part.per, &s_last, reinterpret_cast<float*>(smem),
                                              SH::STAGES * SH::STAGE / 4);
        }
        lo = start + t1;
        if (t1 == tiles) {
            start += tiles;
            item = tree_next_item<EXT>(a, un, item);
        }
    }
}

// Launches the EXT form: a.pass, a.R and what belongs to them are set; item_rows and row_groups are set
// for the joining launch, to which all shares are left.
template <int D, bool KB, int NQ, int RW>
cudaError_t launch_tree_ext_t(TreeArgs& a, cudaStream_t s)
{
    using SH = TrShape<D, KB>;
    const size_t smem = 128 + size_t(SH::STAGES) * SH::STAGE + (KB ? 0 : size_t(16 * RW) * SH::Q_ROW * 4);
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(tree_kernel<D, KB, NQ, RW, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    });
    if (cfg != cudaSuccess) return cfg;
    a.tile = kTrTile;
    a.item_rows = 16 * RW;
    a.min_per = 2;
    a.half_slack = 4;
    const bool prefixes = a.pass == kTreePrefix || a.pass == kTreeBoth;
    a.row_groups = int(((prefixes ? a.seqs : 1LL) * a.R + a.item_rows - 1) / a.item_rows);
    int ctas = num_sms() * (2 * (smem + 10 * 1024) <= size_t(kSmemPerSm) ? 2 : 1);
    if (ctas > kTreeMaxCtas) ctas = kTreeMaxCtas;
    return launch_after_previous(tree_kernel<D, KB, NQ, RW, true>, dim3(unsigned(ctas)), dim3(kTrThreads), smem, s, a);
}

// `rows`: query rows that a unit has, about.  bf16 has an item of 32 rows too, two warps to each half of a
// tile's tokens: 20 rows of 48 sequences with about 1500 tokens each 92 us, with 16-row items, which read
// everything twice, 132, with 64-row items, half of them empty, 133 (the tensor-core kernel 126).
template <int D>
cudaError_t launch_tree_ext_d(TreeArgs& a, bool kv_bf16, int rows, cudaStream_t s)
{
    const bool few = rows <= 16;
    if (!kv_bf16) return few ? launch_tree_ext_t<D, false, 1, 1>(a, s) : launch_tree_ext_t<D, false, 1, 4>(a, s);
    if (!a.q_bf16) return few ? launch_tree_ext_t<D, true, 3, 1>(a, s) : launch_tree_ext_t<D, true, 3, 4>(a, s);
    if (!few && rows <= 32) return launch_tree_ext_t<D, true, 1, 2>(a, s);
    return few ? launch_tree_ext_t<D, true, 1, 1>(a, s) : launch_tree_ext_t<D, true, 1, 4>(a, s);
}

}  // namespace sa
