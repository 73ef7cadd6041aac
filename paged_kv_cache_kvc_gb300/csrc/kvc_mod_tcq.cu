// e4m3- and int4-pool instances of the tensor-memory (tcgen05) kernel of attention with modified scores.
#include "kvc_mod_tc.cuh"

namespace kvc {

DecodeKernel select_mod_tc_quant(bool int4, bool fixed)
{
    if (int4) return fixed ? mod_tc_instance<128, KV_INT4, true>() : mod_tc_instance<128, KV_INT4, false>();
    return fixed ? mod_tc_instance<128, KV_E4M3, true>() : mod_tc_instance<128, KV_E4M3, false>();
}

}  // namespace kvc
