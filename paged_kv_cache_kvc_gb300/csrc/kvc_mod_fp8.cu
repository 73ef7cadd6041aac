// e4m3-pool instances of the modified-score split kernel (f16 operands, as in the plain kernels).
#include "kvc_mod.cuh"

namespace kvc {

DecodeKernel select_mod_fp8(int cols, bool tile)
{
    if (tile) return mod_instance<128, 4, KV_E4M3, false, true>();
    switch (n_tiles(cols)) {
    case 1: return mod_instance<128, 1, KV_E4M3, false, false>();
    case 2: return mod_instance<128, 2, KV_E4M3, false, false>();
    }
    return mod_instance<128, 4, KV_E4M3, false, false>();
}

}  // namespace kvc
