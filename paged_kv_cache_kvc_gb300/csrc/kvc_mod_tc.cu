// bf16-pool instances of the tensor-memory (tcgen05) kernel of attention with modified scores, and its merge.
#include "kvc_mod_tc.cuh"

namespace kvc {

DecodeKernel select_mod_tc_bf16(int D, bool fixed)
{
    if (D == 64) return fixed ? mod_tc_instance<64, KV_BF16, true>() : mod_tc_instance<64, KV_BF16, false>();
    return fixed ? mod_tc_instance<128, KV_BF16, true>() : mod_tc_instance<128, KV_BF16, false>();
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
