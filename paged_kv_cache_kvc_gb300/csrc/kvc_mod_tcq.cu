// e4m3- and int4-pool instances of the tensor-memory (tcgen05) kernel of attention with modified scores.
#include "kvc_mod_tc.cuh"

namespace kvc {

DecodeKernel select_mod_tc_quant(bool int4)
{
    return int4 ? mod_tc_instance<128, KV_INT4, false>() : mod_tc_instance<128, KV_E4M3, false>();
}

}  // namespace kvc
