// New tokens into the paged cache: rotation of queries and keys to their positions, K/V
// stored in the pages, the key box of the touched blocks; and the move of accepted drafts.
//
// Append.  With position p and frequency w_i the pair (x_a, x_b) becomes
// (x_a cos(p w_i) - x_b sin(p w_i), x_b cos(p w_i) + x_a sin(p w_i)).  p w_i is needed to
// far below a turn although p may be in the millions: the frequency is held in turns per
// position as a 64-bit fraction f = frac(w_i / 2 pi) 2^64, so p f mod 2^64 is the exact
// fraction of a turn of the rounded frequency (the integer product wraps at a turn).  What the
// nearest quarter turn leaves of it, at most an eighth, goes to sincospi in fp32: off by 2.4e-8
// at most, where the whole fraction in fp32 would be off by 9.4e-8, more than a step of a sine.
//
// Mapping: CTA = a run of tokens of one sequence (a block, or as many blocks as make 64
// tokens) and a share of the heads.  The run's cosines and sines are computed once into
// shared memory for all heads.  A thread's item is 16 channels of one head row: the 8 pairs
// that one 16-byte load of each half brings (bf16).  Key items of one head sit in one warp,
// rows over its lane groups, so a block's minimum and maximum need shuffles only; the block
// belongs to one CTA, so the box is updated without atomics.  HBM traffic: every new row
// once in and once out, the box rows of the touched blocks.
//
// Bound by memory on long inputs, by latency on short ones.  What bounds the long ones is the bytes
// in flight: each thread copies its next three items ahead into shared memory.  48K rows of 32
// query and 8 KV heads of 128 channels (1.2 GB moved): 198 us, 6.0 TB/s; with two plain loads in
// flight a thread 248 us, with five items ahead 198 us, with 256 threads and 3 CTAs an SM 216 us.
// One token: 4.5 us, the chain of lengths, pages, rows and box.
#include "sa_common.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kAppThreads = 384;
constexpr int kAppWarps = kAppThreads / 32;
constexpr int kAppRun = 64;          // tokens of a run when blocks are smaller
constexpr int kAppSlots = 4;         // items of a thread on their way from memory
constexpr int kAppMaxBlocks = 8;     // blocks of a run

struct AppendArgs {
    const int32_t *cu_rows, *seq_lens, *positions, *block_table;
    const double* inv_freq;
    const void *q_new, *k_new, *v_new;
    void *q_out, *k_pages, *v_pages, *kmin, *kmax;
    uint32_t* err;
    long long q_stride, k_stride, v_stride;
    int B, Hq, Hkv, D, bs, nb_cap, num_pages, capacity;
    int num_rows, uniform_rows, uniform_len;
    int run;                 // tokens per run, a multiple of bs
    int runs_uniform;        // cu_rows null: runs a sequence may touch
    int cs_words;            // 16-byte words of the cosines and sines
    int rotary, pairs;       // pairs: neighbouring channels turn together
};

// 16 channels of a row as fp32: 8 at `a`, 8 at `b` (16-byte aligned both).
template <bool BF16>
struct Raw16 {
    uint4 v[BF16 ? 2 : 4];
};

template <bool BF16>
__device__ __forceinline__ const char* at_elem(const void* p, long long elem)
{
    return reinterpret_cast<const char*>(p) + elem * (BF16 ? 2 : 4);
}

template <bool BF16>
__device__ __forceinline__ Raw16<BF16> load16(const void* row, int a, int b)
{
    // plain loads: q_out may be the memory that q_new is read from
    Raw16<BF16> r;
    const uint4* pa = reinterpret_cast<const uint4*>(at_elem<BF16>(row, a));
    const uint4* pb = reinterpret_cast<const uint4*>(at_elem<BF16>(row, b));
    if constexpr (BF16) {
        r.v[0] = __ldcs(pa);
        r.v[1] = __ldcs(pb);
    } else {
        r.v[0] = __ldcs(pa);
        r.v[1] = __ldcs(pa + 1);
        r.v[2] = __ldcs(pb);
        r.v[3] = __ldcs(pb + 1);
    }
    return r;
}

// A thread's own ring of kAppSlots items in shared memory, filled by asynchronous copies: nobody
// else reads it, so waiting for the thread's own copies is all the order it needs.
template <bool BF16>
struct Ring16 {
    static constexpr int WORDS = BF16 ? 2 : 4;
    uint4* at;                                                // this thread's first word

    __device__ __forceinline__ void fetch(int slot, const void* row, int a, int b) const
    {
        const uint4* pa = reinterpret_cast<const uint4*>(at_elem<BF16>(row, a));
        const uint4* pb = reinterpret_cast<const uint4*>(at_elem<BF16>(row, b));
#pragma unroll
        for (int i = 0; i < WORDS; ++i)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                             smem_u32(at + (slot * WORDS + i) * kAppThreads)),
                         "l"(i < WORDS / 2 ? pa + i : pb + (i - WORDS / 2))
                         : "memory");
    }
    // Every step ends a group of copies, an empty one too, so that "all but the newest
    // kAppSlots - 1" always means the item of this step.
    __device__ __forceinline__ static void close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    __device__ __forceinline__ static void wait()
    {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAppSlots - 1) : "memory");
    }
    __device__ __forceinline__ Raw16<BF16> item(int slot) const
    {
        Raw16<BF16> r;
#pragma unroll
        for (int i = 0; i < WORDS; ++i) r.v[i] = at[(slot * WORDS + i) * kAppThreads];
        return r;
    }
};

template <bool BF16>
__device__ __forceinline__ void widen16(const Raw16<BF16>& r, float (&f)[16])
{
    if constexpr (BF16) {
        unpack16<true>(r.v[0], f);
        unpack16<true>(r.v[1], f + 8);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) unpack16<false>(r.v[i], f + 4 * i);
    }
}

// fp32 -> stored type (round to nearest even): 8 words of bf16 pairs, or 16 floats.
template <bool BF16>
__device__ __forceinline__ void narrow16(const float (&f)[16], uint32_t (&w)[BF16 ? 8 : 16])
{
#pragma unroll
    for (int i = 0; i < (BF16 ? 8 : 16); ++i) {
        if constexpr (BF16) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
        else w[i] = __float_as_uint(f[i]);
    }
}

template <bool BF16, int N>
__device__ __forceinline__ void store16(void* row, int a, int b, const uint32_t (&w)[N])
{
    static_assert(N == (BF16 ? 8 : 16), "16 channels");
    uint4* pa = reinterpret_cast<uint4*>(const_cast<char*>(at_elem<BF16>(row, a)));
    uint4* pb = reinterpret_cast<uint4*>(const_cast<char*>(at_elem<BF16>(row, b)));
#pragma unroll
    for (int i = 0; i < N / 8; ++i) {
        pa[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        pb[i] = make_uint4(w[N / 2 + 4 * i], w[N / 2 + 4 * i + 1], w[N / 2 + 4 * i + 2], w[N / 2 + 4 * i + 3]);
    }
}

template <bool BF16>
__device__ __forceinline__ void store16(void* row, int a, int b, const float (&f)[16])
{
    uint32_t w[BF16 ? 8 : 16];
    narrow16<BF16>(f, w);
    store16<BF16>(row, a, b, w);
}

// The minimum and maximum of 16 channels over rows, in the stored type: its values are what a later
// reader of the pages sees, and pairs of bf16 take half the registers.  A NaN counts as no value.
template <bool BF16>
struct Box16 {
    uint32_t lo[BF16 ? 8 : 16], hi[BF16 ? 8 : 16];
};

template <bool BF16>
__device__ __forceinline__ void box_join(uint32_t& lo, uint32_t& hi, uint32_t x, uint32_t y)
{
    if constexpr (BF16) {
        asm("min.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(x));
        asm("max.bf16x2 %0, %0, %1;" : "+r"(hi) : "r"(y));
    } else {
        lo = __float_as_uint(fminf(__uint_as_float(lo), __uint_as_float(x)));
        hi = __float_as_uint(fmaxf(__uint_as_float(hi), __uint_as_float(y)));
    }
}

// Turns the 8 pairs of a rotary chunk.  Cosines and sines of a row: chunk c's pairs 2p and
// 2p + 1 at 16-byte word p * chunks + c, so that a row's chunks are read without bank
// conflicts.
__device__ __forceinline__ void rotate16(float (&f)[16], const float4* cs_row, int c, int chunks, bool pairs)
{
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const float4 w = cs_row[p * chunks + c];
        if (pairs) {
            const float a0 = f[4 * p], b0 = f[4 * p + 1], a1 = f[4 * p + 2], b1 = f[4 * p + 3];
            f[4 * p] = fmaf(a0, w.x, -(b0 * w.y));
            f[4 * p + 1] = fmaf(b0, w.x, a0 * w.y);
            f[4 * p + 2] = fmaf(a1, w.z, -(b1 * w.w));
            f[4 * p + 3] = fmaf(b1, w.z, a1 * w.w);
        } else {
            const float a0 = f[2 * p], b0 = f[8 + 2 * p], a1 = f[2 * p + 1], b1 = f[9 + 2 * p];
            f[2 * p] = fmaf(a0, w.x, -(b0 * w.y));
            f[8 + 2 * p] = fmaf(b0, w.x, a0 * w.y);
            f[2 * p + 1] = fmaf(a1, w.z, -(b1 * w.w));
            f[9 + 2 * p] = fmaf(b1, w.z, a1 * w.w);
        }
    }
}

// The rows and the context length of sequence b; 0 rows when it is inactive or its numbers
// are out of range.
__device__ __forceinline__ int sequence_rows(const AppendArgs& a, int b, int& row0, int& len)
{
    int n;
    if (a.cu_rows != nullptr) {
        row0 = a.cu_rows[b];
        n = a.cu_rows[b + 1] - row0;
    } else {
        row0 = b * a.uniform_rows;
        n = a.uniform_rows;
    }
    len = a.seq_lens != nullptr ? a.seq_lens[b] : a.uniform_len;
    if (len == -1) return 0;
    if (row0 < 0 || n < 0 || row0 > a.num_rows - n || len < 0 || len > a.capacity - n) {
        raise_error(a.err, SPARSE_ATTN_ERR_LENGTH);
        return 0;
    }
    return n;
}

__device__ __forceinline__ int runs_of(int n, int len, int run) { return n > 0 ? (len + n - 1) / run - len / run + 1 : 0; }

template <bool QB, bool KB>
__global__ void __launch_bounds__(kAppThreads, 2) append_kernel(AppendArgs a)
{
    extern __shared__ __align__(16) float4 s_cs[];            // [rows of the run][rotary / 4]
    __shared__ unsigned long long s_freq[64];
    __shared__ int s_warp[kAppWarps], s_find[2], s_page[kAppMaxBlocks];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    allow_dependents_early();
    grid_dependency_wait();   // rows, lengths and pages may come from the previous kernel

    if (tid < a.rotary / 2) {
        double f = a.inv_freq[tid] * 0.15915494309189533577;   // turns per position
        f -= floor(f);
        s_freq[tid] = __double2ull_rn(f * 18446744073709551616.0);
    }
    // ---- which run of which sequence ------------------------------------------
    int b, k;                                                 // run k of sequence b
    if (a.cu_rows == nullptr) {
        b = int(blockIdx.x) / a.runs_uniform;
        k = int(blockIdx.x) - b * a.runs_uniform;
    } else {
        // runs of the sequences are numbered in order: a scan over the run counts finds the
        // sequence that holds number blockIdx.x
        int before = 0;
        b = -1;
        k = 0;
        for (int base = 0; base < a.B && b < 0; base += kAppThreads) {
            int row0, len, mine = 0;
            if (base + tid < a.B) {
                const int n = sequence_rows(a, base + tid, row0, len);
                mine = runs_of(n, len, a.run);
            }
            const int incl = warp_inclusive_scan(mine, lane);
            if (tid == 0) s_find[0] = -1;
            if (lane == 31) s_warp[warp] = incl;
            __syncthreads();
            int off = before, all = before;
            for (int w = 0; w < kAppWarps; ++w) {
                if (w < warp) off += s_warp[w];
                all += s_warp[w];
            }
            const int x = int(blockIdx.x);
            if (mine > 0 && x >= off + incl - mine && x < off + incl) {
                s_find[0] = base + tid;
                s_find[1] = x - (off + incl - mine);
            }
            __syncthreads();
            b = s_find[0];
            k = s_find[1];
            before = all;
            __syncthreads();
        }
        if (b < 0) return;
    }
    int row0, len;
    const int n_seq = sequence_rows(a, b, row0, len);
    if (k >= runs_of(n_seq, len, a.run)) return;
    const int run_first = (len / a.run + k) * a.run;          // the run's first token slot
    const int t0 = max(len, run_first), t1 = min(len + n_seq, run_first + a.run);
    const int n = t1 - t0;                                    // tokens [t0, t1)
    const int r0 = row0 + (t0 - len);                         // their first row
    const int blk0 = t0 / a.bs, blks = (t1 - 1) / a.bs - blk0 + 1;
    if (tid < blks) {
        const int page = a.block_table[(long long)b * a.nb_cap + blk0 + tid];
        const bool ok = page >= 0 && page < a.num_pages;
        if (!ok) raise_error(a.err, SPARSE_ATTN_ERR_PAGE);
        s_page[tid] = ok ? page : -1;
    }
    __syncthreads();          // s_freq, s_page

    // ---- cosines and sines of the run's rows --------------------------------------
    const int half = a.rotary / 2, rchunks = a.rotary / 16;
    for (int e = tid; e < n * half; e += kAppThreads) {
        const int r = e / half, i = e - r * half;
        const long long pos = a.positions != nullptr ? a.positions[r0 + r] : t0 + r;
        const unsigned long long phase = (unsigned long long)pos * s_freq[i];
        const unsigned quarter = (unsigned(phase >> 32) + 0x20000000u) >> 30;           // the nearest one
        const long long rest = (long long)(phase - ((unsigned long long)quarter << 62));
        float sn, cn;
        sincospif(float(int(rest >> 30)) * 1.16415321826934814453125e-10f, &sn, &cn);  // 2^-33: in half turns
        if (quarter & 1u) {
            const float c = cn;
            cn = -sn;
            sn = c;
        }
        if (quarter & 2u) {
            cn = -cn;
            sn = -sn;
        }
        float2* dst = reinterpret_cast<float2*>(s_cs + size_t(r) * (a.rotary / 4));
        dst[(((i & 7) >> 1) * rchunks + (i >> 3)) * 2 + (i & 1)] = make_float2(cn, sn);
    }
    const Ring16<QB> ring{reinterpret_cast<uint4*>(s_cs) + a.cs_words + tid};
    __syncthreads();

    const int CH = a.D / 16, ch_shift = __ffs(CH) - 1;        // 16-channel items of a row
    auto elem_a = [&](int c) { return c < rchunks && !a.pairs ? 8 * c : 16 * c; };
    auto elem_b = [&](int c) { return c < rchunks && !a.pairs ? half + 8 * c : 16 * c + 8; };
    const int Y = gridDim.y, y = blockIdx.y;
    const int kv0 = a.Hkv * y / Y, kvn = a.Hkv * (y + 1) / Y - kv0;
    const int q0 = a.Hq * y / Y, qn = a.q_new != nullptr ? a.Hq * (y + 1) / Y - q0 : 0;

    // ---- keys: lane groups of a warp take a head's rows; the last warps start ------
    {
        int rl = 1;                                           // rows of one head side by side
        while (rl < n && rl * CH < 32) rl *= 2;
        const int items = kvn * rl * CH;                      // (head, row lane, chunk)
        const int first = (kAppWarps - 1 - warp) * 32 + lane;
        for (int i0 = first - lane; i0 < items; i0 += kAppThreads) {
            const int it = i0 + lane;
            const bool live = it < items;
            const int c = it & (CH - 1), rlane = (it >> ch_shift) & (rl - 1);
            const int kvh = kv0 + (live ? (it >> ch_shift) / rl : 0);
            const int ea = elem_a(c), eb = elem_b(c);
            for (int j = 0; j < blks; ++j) {
                const int page = s_page[j];
                if (page < 0) continue;
                const int tb = (blk0 + j) * a.bs;
                const int ra = max(t0, tb) - t0, rb = min(t1, tb + a.bs) - t0;
                char* tile = const_cast<char*>(
                    at_elem<KB>(a.k_pages, ((long long)page * a.Hkv + kvh) * a.bs * a.D));
                constexpr int W = KB ? 8 : 16;
                Box16<KB> box;
#pragma unroll
                for (int e = 0; e < W; ++e) {
                    box.lo[e] = KB ? 0x7f807f80u : 0x7f800000u;
                    box.hi[e] = KB ? 0xff80ff80u : 0xff800000u;
                }
                const int first_row = live ? ra + rlane : rb;
                auto fetch = [&](int r, int slot) {
                    if (r < rb) ring.fetch(slot, at_elem<QB>(a.k_new, (r0 + r) * a.k_stride + kvh * a.D), ea, eb);
                    ring.close();
                };
#pragma unroll
                for (int s = 0; s < kAppSlots - 1; ++s) fetch(first_row + s * rl, s);
                int slot = 0;
                for (int r = first_row; r < rb; r += rl) {
                    fetch(r + (kAppSlots - 1) * rl, (slot + kAppSlots - 1) % kAppSlots);
                    ring.wait();
                    float f[16];
                    widen16<QB>(ring.item(slot), f);
                    if (c < rchunks) rotate16(f, s_cs + size_t(r) * (a.rotary / 4), c, rchunks, a.pairs);
                    uint32_t w[W];
                    narrow16<KB>(f, w);
                    store16<KB>(const_cast<char*>(at_elem<KB>(tile, (long long)(t0 + r - tb) * a.D)), ea, eb, w);
#pragma unroll
                    for (int e = 0; e < W; ++e) box_join<KB>(box.lo[e], box.hi[e], w[e], w[e]);
                    slot = (slot + 1) % kAppSlots;
                }
                if (a.kmin == nullptr) continue;
                for (int m = CH; m < CH * rl; m <<= 1) {
#pragma unroll
                    for (int e = 0; e < W; ++e)
                        box_join<KB>(box.lo[e], box.hi[e], __shfl_xor_sync(kFullMask, box.lo[e], m),
                                     __shfl_xor_sync(kFullMask, box.hi[e], m));
                }
                if (live && rlane == 0) {
                    const long long row = (((long long)b * a.Hkv + kvh) * a.nb_cap + blk0 + j) * a.D;
                    char* pmin = const_cast<char*>(at_elem<KB>(a.kmin, row));
                    char* pmax = const_cast<char*>(at_elem<KB>(a.kmax, row));
                    if (tb < t0) {                            // the block held tokens before
                        const Raw16<KB> lo = load16<KB>(pmin, ea, eb), hi = load16<KB>(pmax, ea, eb);
#pragma unroll
                        for (int x = 0; x < W / 4; ++x) {
                            box_join<KB>(box.lo[4 * x], box.hi[4 * x], lo.v[x].x, hi.v[x].x);
                            box_join<KB>(box.lo[4 * x + 1], box.hi[4 * x + 1], lo.v[x].y, hi.v[x].y);
                            box_join<KB>(box.lo[4 * x + 2], box.hi[4 * x + 2], lo.v[x].z, hi.v[x].z);
                            box_join<KB>(box.lo[4 * x + 3], box.hi[4 * x + 3], lo.v[x].w, hi.v[x].w);
                        }
                    }
                    store16<KB>(pmin, ea, eb, box.lo);
                    store16<KB>(pmax, ea, eb, box.hi);
                }
            }
        }
    }
    // ---- queries and values: chunk fastest, then head, then row ----------------------
    {
        const int per_row = (qn + kvn) * CH;
        if (per_row == 0) return;                             // without queries, more shares than heads
        struct Cursor {
            int row, rest;                                    // rest: channel chunk fastest, then head
        };
        const int rows_step = kAppThreads / per_row, rest_step = kAppThreads - rows_step * per_row;
        auto step = [&](Cursor& x) {
            x.row += rows_step;
            x.rest += rest_step;
            if (x.rest >= per_row) {
                x.rest -= per_row;
                ++x.row;
            }
        };
        auto fetch = [&](const Cursor& x, int slot) {
            const int c = x.rest & (CH - 1), head = x.rest >> ch_shift;
            if (x.row < n) {
                if (head < qn)
                    ring.fetch(slot, at_elem<QB>(a.q_new, (r0 + x.row) * a.q_stride + (q0 + head) * a.D), elem_a(c), elem_b(c));
                else
                    ring.fetch(slot, at_elem<QB>(a.v_new, (r0 + x.row) * a.v_stride + (kv0 + head - qn) * a.D), 16 * c,
                               16 * c + 8);
            }
            ring.close();
        };
        Cursor at{tid / per_row, tid % per_row}, ahead = at;
#pragma unroll
        for (int s = 0; s < kAppSlots - 1; ++s) {
            fetch(ahead, s);
            step(ahead);
        }
        for (int slot = 0; at.row < n; step(at), slot = (slot + 1) % kAppSlots) {
            fetch(ahead, (slot + kAppSlots - 1) % kAppSlots);
            step(ahead);
            ring.wait();
            const Raw16<QB> raw = ring.item(slot);
            const int c = at.rest & (CH - 1), head = at.rest >> ch_shift;
            if (head < qn) {
                float f[16];
                widen16<QB>(raw, f);
                if (c < rchunks) rotate16(f, s_cs + size_t(at.row) * (a.rotary / 4), c, rchunks, a.pairs);
                store16<QB>(const_cast<char*>(at_elem<QB>(a.q_out, ((long long)(r0 + at.row) * a.Hq + q0 + head) * a.D)),
                            elem_a(c), elem_b(c), f);
                continue;
            }
            const int t = t0 + at.row, page = s_page[t / a.bs - blk0];
            if (page < 0) continue;
            void* dst = const_cast<char*>(at_elem<KB>(
                a.v_pages, (((long long)page * a.Hkv + kv0 + head - qn) * a.bs + t % a.bs) * a.D));
            if constexpr (QB == KB) {                         // same type: the bits as they are
                uint4* p = reinterpret_cast<uint4*>(const_cast<char*>(at_elem<KB>(dst, 16 * c)));
#pragma unroll
                for (int i = 0; i < (KB ? 2 : 4); ++i) p[i] = raw.v[i];
            } else {
                float f[16];
                widen16<QB>(raw, f);
                store16<KB>(dst, 16 * c, 16 * c + 8, f);
            }
        }
    }
}

template <bool QB, bool KB>
cudaError_t launch_append_t(const AppendArgs& a, dim3 grid, cudaStream_t s)
{
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(append_kernel<QB, KB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    128 * 64 * 8 + kAppThreads * kAppSlots * (QB ? 32 : 64));
    });
    if (cfg != cudaSuccess) return cfg;
    return launch_after_previous(append_kernel<QB, KB>, grid, dim3(kAppThreads),
                                 16 * size_t(a.cs_words) + kAppThreads * kAppSlots * (QB ? 32 : 64), s, a);
}

// ------------------------------------------------------------------ commit ---
// CTA = (sequence, KV head).  Accepted rows move in ascending order, a batch at a time: all
// of a batch's rows are loaded before any is stored, and since the path is strictly
// ascending (path[i] >= i) a later batch never reads what an earlier one wrote.  The box of
// the touched blocks follows from the moved keys.  A few kilobytes per CTA: bound by the
// chain of dependent loads (lengths, path, pages, rows).
constexpr int kComThreads = 128;
constexpr int kComBatch = 4;         // 16-byte elements of K and of V a thread holds

struct CommitArgs {
    const int32_t *seq_lens, *path, *path_len, *block_table;
    int path_stride;
    char *k_pages, *v_pages, *kmin, *kmax;
    int32_t* new_lens;
    uint32_t* err;
    int Hkv, D, bs, N, Q, nb_cap, num_pages, row_bytes;
};

template <bool KB>
__global__ void __launch_bounds__(kComThreads) commit_kernel(CommitArgs a)
{
    __shared__ long long s_src[kTreeMaxDrafts], s_dst[kTreeMaxDrafts];   // byte offsets of the rows
    const int tid = threadIdx.x;
    const int b = blockIdx.x / a.Hkv, kvh = blockIdx.x - b * a.Hkv;
    allow_dependents_early();
    grid_dependency_wait();   // the path and the pages may come from the previous kernel

    const int len = a.seq_lens != nullptr ? a.seq_lens[b] : a.N;
    const int n = a.path_len[b];
    const bool active = len >= 0 && len <= a.N;
    bool bad_len = (!active && len != -1) || (active && (n < 0 || n > a.path_stride || n > a.Q)), bad_page = false;
    if (active && !bad_len) {
        for (int i = tid; i < n; i += kComThreads) {
            const int j = a.path[(long long)b * a.path_stride + i];
            const int prev = i > 0 ? a.path[(long long)b * a.path_stride + i - 1] : -1;
            if (j <= prev || j >= a.Q) {                      // prev >= -1 is checked by its own entry
                bad_len = true;
                continue;
            }
            if (j < 0) {
                bad_len = true;
                continue;
            }
            const int src = len + j, dst = len + i;           // below the capacity: len <= N, j, i < Q
            const int sp = a.block_table[(long long)b * a.nb_cap + src / a.bs];
            const int dp = a.block_table[(long long)b * a.nb_cap + dst / a.bs];
            if (sp < 0 || sp >= a.num_pages || dp < 0 || dp >= a.num_pages) {
                bad_page = true;
                continue;
            }
            s_src[i] = (((long long)sp * a.Hkv + kvh) * a.bs + src % a.bs) * a.row_bytes;
            s_dst[i] = (((long long)dp * a.Hkv + kvh) * a.bs + dst % a.bs) * a.row_bytes;
        }
    }
    const bool any_len = __syncthreads_or(bad_len) != 0, any_page = __syncthreads_or(bad_page) != 0;
    if (tid == 0 && kvh == 0) {
        if (any_len) raise_error(a.err, SPARSE_ATTN_ERR_LENGTH);
        if (any_page) raise_error(a.err, SPARSE_ATTN_ERR_PAGE);
        a.new_lens[b] = active && !any_len && !any_page ? len + n : len;
    }
    if (!active || any_len || any_page || n == 0) return;

    const int C16 = a.row_bytes / 16, c_shift = __ffs(C16) - 1;   // 8, 16 or 32
    const int rows = kComBatch * kComThreads / C16;               // rows of a batch
    for (int i0 = 0; i0 < n; i0 += rows) {
        const int items = min(rows, n - i0) * C16;
        uint4 kv[kComBatch], vv[kComBatch];
#pragma unroll
        for (int u = 0; u < kComBatch; ++u) {
            const int it = tid + u * kComThreads;
            if (it >= items) break;
            const long long off = s_src[i0 + (it >> c_shift)] + (it & (C16 - 1)) * 16;
            kv[u] = *reinterpret_cast<const uint4*>(a.k_pages + off);
            vv[u] = *reinterpret_cast<const uint4*>(a.v_pages + off);
        }
        __syncthreads();      // every row of the batch is read before one is written
#pragma unroll
        for (int u = 0; u < kComBatch; ++u) {
            const int it = tid + u * kComThreads;
            if (it >= items) break;
            const long long off = s_dst[i0 + (it >> c_shift)] + (it & (C16 - 1)) * 16;
            *reinterpret_cast<uint4*>(a.k_pages + off) = kv[u];
            *reinterpret_cast<uint4*>(a.v_pages + off) = vv[u];
        }
    }
    if (a.kmin == nullptr) return;
    __syncthreads();          // the moved keys, read back below
    constexpr int EPL = KB ? 8 : 4;
    const int blk0 = len / a.bs, blks = (len + n - 1) / a.bs - blk0 + 1;
    for (int it = tid; it < blks * C16; it += kComThreads) {
        const int j = it >> c_shift, c = it & (C16 - 1);
        const int tb = (blk0 + j) * a.bs;
        const int ia = max(len, tb) - len, ib = min(len + n, tb + a.bs) - len;
        const long long box = (((long long)b * a.Hkv + kvh) * a.nb_cap + blk0 + j) * a.row_bytes + c * 16;
        uint4* pmin = reinterpret_cast<uint4*>(a.kmin + box);
        uint4* pmax = reinterpret_cast<uint4*>(a.kmax + box);
        float lo[EPL], hi[EPL];
        if (tb < len) {
            unpack16<KB>(*pmin, lo);
            unpack16<KB>(*pmax, hi);
        } else {
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                lo[e] = INFINITY;
                hi[e] = -INFINITY;
            }
        }
#pragma unroll 4
        for (int i = ia; i < ib; ++i) {
            float f[EPL];
            unpack16<KB>(__ldcg(reinterpret_cast<const uint4*>(a.k_pages + s_dst[i] + c * 16)), f);
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                lo[e] = fminf(lo[e], f[e]);
                hi[e] = fmaxf(hi[e], f[e]);
            }
        }
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

}  // namespace

cudaError_t launch_append(const Geometry& g, const AppendCall& c, uint32_t* err, cudaStream_t s)
{
    AppendArgs a{};
    a.cu_rows = c.cu_rows;
    a.seq_lens = c.seq_lens;
    a.positions = c.positions;
    a.block_table = c.block_table;
    a.inv_freq = c.inv_freq;
    a.q_new = c.q_new;
    a.k_new = c.k_new;
    a.v_new = c.v_new;
    a.q_out = c.q_out;
    a.k_pages = c.k_pages;
    a.v_pages = c.v_pages;
    a.kmin = c.kmin;
    a.kmax = c.kmax;
    a.err = err;
    a.q_stride = c.q_stride;
    a.k_stride = c.k_stride;
    a.v_stride = c.v_stride;
    a.B = g.B;
    a.Hq = g.Hq;
    a.Hkv = g.Hkv;
    a.D = g.D;
    a.bs = g.bs;
    a.nb_cap = g.nb_cap;
    a.num_pages = g.num_pages;
    a.capacity = c.capacity;
    a.num_rows = c.num_rows;
    a.uniform_rows = c.num_rows / g.B;
    a.uniform_len = c.uniform_len;
    a.run = g.bs > kAppRun ? g.bs : kAppRun;
    a.rotary = c.rotary_dim;
    a.pairs = c.pairing == SPARSE_ATTN_ROTATE_PAIRS;
    // n > 0 tokens touch at most (n - 2 + run) / run + 1 aligned runs
    a.runs_uniform = (a.uniform_rows - 2 + a.run) / a.run + 1;
    const long long runs = c.cu_rows ? (long long)c.num_rows / a.run + 2LL * g.B : (long long)g.B * a.runs_uniform;
    // rows of a run that the head split's rule goes by
    const int rows = a.uniform_rows < 1 ? 1 : (a.uniform_rows < a.run ? a.uniform_rows : a.run);
    const long long items = (long long)rows * (g.Hq + 2 * g.Hkv) * (g.D / 16);
    unsigned Y = 1;
    while (Y < 8 && runs * Y < num_sms() && items / Y > 2 * kAppThreads) Y *= 2;
    a.cs_words = (rows < a.run && !c.cu_rows ? rows : a.run) * (c.rotary_dim / 4);
    const dim3 grid{unsigned(runs), Y, 1};
    if (g.q_bf16) return g.kv_bf16 ? launch_append_t<true, true>(a, grid, s) : launch_append_t<true, false>(a, grid, s);
    return g.kv_bf16 ? launch_append_t<false, true>(a, grid, s) : launch_append_t<false, false>(a, grid, s);
}

cudaError_t launch_commit(const Geometry& g, const int32_t* seq_lens, const int32_t* path, int path_stride,
                          const int32_t* path_len, void* k_pages, void* v_pages, const int32_t* block_table,
                          void* kmin, void* kmax, int32_t* new_lens, uint32_t* err, cudaStream_t s)
{
    CommitArgs a{};
    a.seq_lens = seq_lens;
    a.path = path;
    a.path_len = path_len;
    a.block_table = block_table;
    a.path_stride = path_stride;
    a.k_pages = static_cast<char*>(k_pages);
    a.v_pages = static_cast<char*>(v_pages);
    a.kmin = static_cast<char*>(kmin);
    a.kmax = static_cast<char*>(kmax);
    a.new_lens = new_lens;
    a.err = err;
    a.Hkv = g.Hkv;
    a.D = g.D;
    a.bs = g.bs;
    a.N = g.N;
    a.Q = g.Q;
    a.nb_cap = g.nb_cap;
    a.num_pages = g.num_pages;
    a.row_bytes = g.D * (g.kv_bf16 ? 2 : 4);
    const dim3 grid{unsigned(g.units())};
    if (g.kv_bf16) return launch_after_previous(commit_kernel<true>, grid, dim3(kComThreads), 0, s, a);
    return launch_after_previous(commit_kernel<false>, grid, dim3(kComThreads), 0, s, a);
}

}  // namespace sa
