// Sparse attention: bf16 instances and the entry point.
#include <algorithm>
#include <cstdlib>

#include "kvc_sparse.cuh"

namespace kvc {

// Weights enter the value product as a bf16 high / low pair for up to 16 query heads per KV head (1.5e-6 of the output's norm),
// as one bf16 with more (1.0e-3, below the output's own rounding: the second part would double four column tiles' products),
// as in kvc_decode_attn_mod.
template <int D, int W>
static SparseKernel pick(int g)
{
    switch (n_tiles(g)) {
    case 1: return sparse_instance<D, 1, KV_BF16, true, W>();
    case 2: return sparse_instance<D, 2, KV_BF16, true, W>();
    }
    return sparse_instance<D, 4, KV_BF16, false, W>();
}

SparseKernel select_sparse_bf16(int D, int g, int warps)
{
    if (D == 64) return warps == 2 ? pick<64, 2>(g) : pick<64, 4>(g);
    return warps == 2 ? pick<128, 2>(g) : pick<128, 4>(g);
}

static bool aligned(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_sparse_attn(kvc_pool *pool, int32_t layer, const void *q, int32_t num_q_heads,
                                      const int32_t *block_tables, int32_t max_blocks, int32_t B,
                                      const int32_t *seq_ids, const int32_t *positions, int64_t n_rows,
                                      const int32_t *selected, int32_t top_k, void *out, float *lse, float scale,
                                      kvc_stream_t stream)
{
    if (!pool || B < 0 || n_rows < 0 || n_rows > 0x0FFFFFFF || num_q_heads <= 0 || num_q_heads % pool->H_KV != 0 ||
        top_k < 1 || top_k > 65536 || !(std::isfinite(scale) && scale > 0.f))
        return KVC_ERR_ARG;
    const int D = pool->D, g = num_q_heads / pool->H_KV;
    if (g > 32 || pool->bs % kBS != 0) return KVC_ERR_UNSUPPORTED;
    if (n_rows == 0) return KVC_OK;
    if (layer < 0 || layer >= pool->L || max_blocks <= 0 || (!seq_ids && n_rows > B)) return KVC_ERR_ARG;
    if (!q || !block_tables || !positions || !selected || !out || !aligned(q, 16) || !aligned(out, 16) ||
        !aligned(block_tables, 4) || !aligned(positions, 4) || !aligned(seq_ids, 4) || !aligned(selected, 4) ||
        !aligned(lse, 4))
        return KVC_ERR_ARG;
    if (out != q) {   // a row's heads are read and written by one cluster: the same place is fine, a shifted one is not
        const uintptr_t a = reinterpret_cast<uintptr_t>(q), b = reinterpret_cast<uintptr_t>(out);
        const uintptr_t n = static_cast<uintptr_t>(n_rows) * num_q_heads * D * 2;
        if (a < b + n && b < a + n) return KVC_ERR_ARG;
    }
    const kvc_status st = check_device(pool);
    if (st != KVC_OK) return st;
    if (!pool->tmap_ok || !pool->tmap_sub_ok) return KVC_ERR_CUDA;
    const int64_t units = n_rows * pool->H_KV;
    // Warps of a CTA: four, and two where there are more CTAs than a GPU takes in several turns, as in a chunk's rows: their
    // starts and ends then overlap better and fewer warps' partials are joined.  Measured with four and with two, lists of
    // 64 blocks, 8 KV heads: 512 rows of one sequence 137 and 128 us (bf16), 110 and 105 (e4m3), 146 and 141 (int4), with 16
    // query heads per KV head 199 and 184, 182 and 169, 239 and 211; 256 rows of one sequence 75.7 and 76.5 (bf16); 64
    // sequences of different lengths 43 and 56, 256 of them 149 and 160: a long row beside short ones wants more warps.
    const int warps = units >= 16ll * pool->num_sms ? 2 : 4;
    const SparseKernel k = pool->dtype == KVC_BF16 ? select_sparse_bf16(D, g, warps)
                                                   : (pool->dtype == KVC_INT4 ? select_sparse_int4(g, warps) : select_sparse_fp8(g, warps));
    if (k.k.ctas_per_sm <= 0) return KVC_ERR_CUDA;
    SparseParams sp{};
    DecodeParams &p = sp.m.d;
    p.q = static_cast<const uint16_t *>(q);
    p.bt = block_tables;
    p.bt_stride = max_blocks;
    p.max_blocks = max_blocks;
    p.B = B;
    p.H_Q = num_q_heads;
    p.H_KV = pool->H_KV;
    p.g = g;
    p.layer = layer;
    p.N = pool->N;
    p.scale_log2 = scale * 1.4426950408889634f;
    if (pool->scales) {
        p.s_k = pool->scales + static_cast<size_t>(layer) * 2 * pool->H_KV * D;
        p.s_v = p.s_k + static_cast<size_t>(pool->H_KV) * D;
    }
    p.lse = lse;
    p.err = pool->err;
    p.stall_loads = std::getenv("KVC_TEST_STALL") ? 1 : 0;
    sp.m.out = static_cast<uint16_t *>(out);
    sp.seqs = seq_ids;
    sp.positions = positions;
    sp.lists = selected;
    sp.top_k = top_k;
    sp.sub = pool->bs / kBS;
    // CTAs per (row, KV head): as many as the grid has room for, each with a few tiles for every warp
    const int64_t tiles = static_cast<int64_t>(top_k) * sp.sub;
    int c = 1;
    while (c < kSparseMost && units * c * 2 <= static_cast<int64_t>(pool->num_sms) * k.k.ctas_per_sm && tiles >= 2 * warps * c) c *= 2;
    // Measured by number and longest first, rows of 1 to 128 blocks, 8 KV heads: 64 rows 38.2 and 35.5 us (e4m3), 45.8 and
    // 42.8 (bf16), 48.7 and 39.6 (int4), with 16 query heads per KV head 50 and 40 (e4m3); 128 rows 67 and 61 (e4m3), 70 and
    // 56 (int4), 76.8 and 77.7 (bf16); 32 rows 22.3 and 22.0.  64 rows of one length 94.1 and 95.3; finding the row costs more
    // than it gives with clusters of 4 (16 rows 19.8 and 20.1) and when CTAs come by the thousand (256 rows 106 and 112).
    sp.longest_first = c <= 2 && longest_first(n_rows, B, units, c, pool->num_sms);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n_rows * c), pool->H_KV);
    cfg.blockDim = dim3(32 * warps);
    cfg.dynamicSmemBytes = static_cast<size_t>(k.k.smem);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = c > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k.fn, sp.sub == 1 ? pool->tmap : pool->tmap_sub, sp);
    if (e != cudaSuccess) return cuda_status(e);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return KVC_OK;
}
