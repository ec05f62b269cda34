// The EXT forms of the tensor-core draft-tree kernel: a translation unit of its own.
#include "sa_tree_tc_kernel.cuh"

namespace sa {
namespace {

template <int D, int REP>
cudaError_t launch_t(TreeArgs& a, cudaStream_t s)
{
    static std::atomic<unsigned long long> configured{0};   // devices set up
    const cudaError_t cfg = once_per_device(configured, [&]() -> cudaError_t {
        return cudaFuncSetAttribute(tree_tc_kernel<D, REP, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    int(tc_smem<D, REP>()));
    });
    if (cfg != cudaSuccess) return cfg;
    CUtensorMap kmap, vmap;
    const long long tiles = (long long)a.num_pages * a.Hkv;
    cudaError_t e = encode_tree_map(&kmap, a.k_pages, D, a.bs, tiles);
    if (e != cudaSuccess) return e;
    e = encode_tree_map(&vmap, a.v_pages, D, a.bs, tiles);
    if (e != cudaSuccess) return e;
    a.item_rows = 128 / REP;
    a.row_groups = int(((a.pass == kTreePrefix ? a.seqs : 1LL) * a.R + a.item_rows - 1) / a.item_rows);
    const int ctas = num_sms() < kTreeMaxCtas ? num_sms() : kTreeMaxCtas;
    return launch_after_previous(tree_tc_kernel<D, REP, true>, dim3(unsigned(ctas)), dim3(kTcThreads), tc_smem<D, REP>(), s, a,
                                 kmap, vmap);
}

}  // namespace

cudaError_t launch_tree_tc_ext(TreeArgs& a, int rows, cudaStream_t s)
{
    a.tensor = 1;
    a.tile = kTcTile;
    a.min_per = 2;                 // as in the draft-tree launch
    a.half_slack = 3;
    if (rows <= 32) return a.D == 128 ? launch_t<128, 4>(a, s) : launch_t<64, 4>(a, s);
    if (rows <= 64) return a.D == 128 ? launch_t<128, 2>(a, s) : launch_t<64, 2>(a, s);
    return a.D == 128 ? launch_t<128, 1>(a, s) : launch_t<64, 1>(a, s);
}

}  // namespace sa
