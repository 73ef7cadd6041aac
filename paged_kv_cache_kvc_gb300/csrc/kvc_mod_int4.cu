// int4-pool instances of the modified-score split kernel (f16 operands, as in the plain kernels).
#include "kvc_mod.cuh"

namespace kvc {

DecodeKernel select_mod_int4(int cols, bool tile)
{
    if (tile) return mod_instance<128, 4, KV_INT4, false, true>();
    switch (n_tiles(cols)) {
    case 1: return mod_instance<128, 1, KV_INT4, false, false>();
    case 2: return mod_instance<128, 2, KV_INT4, false, false>();
    }
    return mod_instance<128, 4, KV_INT4, false, false>();
}

}  // namespace kvc
