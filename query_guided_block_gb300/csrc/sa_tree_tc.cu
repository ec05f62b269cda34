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
#include "sa_tree_tc_kernel.cuh"

namespace sa {
namespace {

template <int D, int REP>
cudaError_t launch_tc_t(TreeArgs a, cudaStream_t s)
{
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(tree_tc_kernel<D, REP, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
    e = launch_after_previous(tree_tc_kernel<D, REP, false>, dim3(unsigned(ctas)), dim3(kTcThreads), tc_smem<D, REP>(), s, a, kmap, vmap);
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
