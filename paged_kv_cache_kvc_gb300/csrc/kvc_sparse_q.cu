// Sparse attention: e4m3 and int4 instances (d_h 128).  Weights enter the value product as f16.
#include "kvc_sparse.cuh"

namespace kvc {

template <int KIND, int W>
static SparseKernel pick(int g)
{
    switch (n_tiles(g)) {
    case 1: return sparse_instance<128, 1, KIND, false, W>();
    case 2: return sparse_instance<128, 2, KIND, false, W>();
    }
    return sparse_instance<128, 4, KIND, false, W>();
}

SparseKernel select_sparse_fp8(int g, int warps) { return warps == 2 ? pick<KV_E4M3, 2>(g) : pick<KV_E4M3, 4>(g); }
SparseKernel select_sparse_int4(int g, int warps) { return warps == 2 ? pick<KV_INT4, 2>(g) : pick<KV_INT4, 4>(g); }

}  // namespace kvc
