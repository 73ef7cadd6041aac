// Instances of the tensor-memory (tcgen05) kernel of attention with modified scores.
#include "kvc_mod_tc.cuh"

namespace kvc {

template <int D, bool FIXED>
static DecodeKernel instance()
{
    static DecodeKernel k = [] {
        DecodeKernel r{nullptr, 0, 0};
        const void *fn = reinterpret_cast<const void *>(&mod_tc_kernel<D, FIXED>);
        r.fn = fn;
        r.smem = ModTcCfg<D>::SMEM;
        r.threads = kMtThreads;
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, r.smem) == cudaSuccess) {
            int n = 0;
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, kMtThreads, r.smem) == cudaSuccess) r.ctas_per_sm = n;
        }
        return r;
    }();
    return k;
}

DecodeKernel select_mod_tc(int D, bool fixed)
{
    if (D == 64) return fixed ? instance<64, true>() : instance<64, false>();
    return fixed ? instance<128, true>() : instance<128, false>();
}

const void *select_mod_tc_merge(int D, bool few)
{
    if (D == 64)
        return few ? reinterpret_cast<const void *>(&mod_tc_merge_kernel<64, 8>)
                   : reinterpret_cast<const void *>(&mod_tc_merge_kernel<64, 1>);
    return few ? reinterpret_cast<const void *>(&mod_tc_merge_kernel<128, 8>)
               : reinterpret_cast<const void *>(&mod_tc_merge_kernel<128, 1>);
}

}  // namespace kvc
