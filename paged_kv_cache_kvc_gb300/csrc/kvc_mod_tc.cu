// bf16-pool instances of the tensor-memory (tcgen05) kernel of attention with modified scores, and its merge.
#include "kvc_mod_tc.cuh"

namespace kvc {

template <int D>
static DecodeKernel bf16_instance(TcMode mode)
{
    return mode == kMtPlain         ? mod_tc_instance<D, KV_BF16, kMtPlain>()
           : mode == kMtCapped      ? mod_tc_instance<D, KV_BF16, kMtCapped>()
           : mode == kMtCappedBrief ? mod_tc_instance<D, KV_BF16, kMtCappedBrief>() : mod_tc_instance<D, KV_BF16, kMtGeneral>();
}

DecodeKernel select_mod_tc_bf16(int D, TcMode mode) { return D == 64 ? bf16_instance<64>(mode) : bf16_instance<128>(mode); }

const void *select_mod_tc_merge(int D, bool few)
{
    if (D == 64)
        return few ? reinterpret_cast<const void *>(&mod_tc_merge_kernel<64, 8>)
                   : reinterpret_cast<const void *>(&mod_tc_merge_kernel<64, 1>);
    return few ? reinterpret_cast<const void *>(&mod_tc_merge_kernel<128, 8>)
               : reinterpret_cast<const void *>(&mod_tc_merge_kernel<128, 1>);
}

}  // namespace kvc
