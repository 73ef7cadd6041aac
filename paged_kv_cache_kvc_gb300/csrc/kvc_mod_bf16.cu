// bf16-pool instances of the modified-score split kernel.  Weights enter the value mixture as a
// bf16 high / low pair (about 16 bits) for up to 16 query columns; 32-column units take one bf16
// operand so that their accumulators fit in registers.
#include "kvc_mod.cuh"

namespace kvc {

template <int D>
static DecodeKernel pick(int cols, bool tile)
{
    if (tile) return mod_instance<D, 4, KV_BF16, false, true>();
    switch (n_tiles(cols)) {
    case 1: return mod_instance<D, 1, KV_BF16, true, false>();
    case 2: return mod_instance<D, 2, KV_BF16, true, false>();
    }
    return mod_instance<D, 4, KV_BF16, false, false>();
}

DecodeKernel select_mod_bf16(int D, int cols, bool tile) { return D == 64 ? pick<64>(cols, tile) : pick<128>(cols, tile); }

}  // namespace kvc
