// e4m3- and int4-pool instances of the tensor-memory (tcgen05) kernel of attention with modified scores.
#include "kvc_mod_tc.cuh"

namespace kvc {

template <int KIND>
static DecodeKernel quant_instance(TcMode mode)
{
    return mode == kMtPlain    ? mod_tc_instance<128, KIND, kMtPlain>()
           : mode == kMtCapped ? mod_tc_instance<128, KIND, kMtCapped>() : mod_tc_instance<128, KIND, kMtGeneral>();
}

DecodeKernel select_mod_tc_quant(bool int4, TcMode mode) { return int4 ? quant_instance<KV_INT4>(mode) : quant_instance<KV_E4M3>(mode); }

}  // namespace kvc
