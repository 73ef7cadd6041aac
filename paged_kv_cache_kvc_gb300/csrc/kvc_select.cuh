// What the kernels of block selection share.
#pragma once
#include "kvc_cluster.cuh"
#include "kvc_configured.cuh"

namespace kvc {

// The smallest e in [-100, 100] with x <= 127 * 2^e (100 if none), x >= 0 as float bits.
__device__ __forceinline__ int unit_exponent(float x)
{
    const uint32_t u = __float_as_uint(x) & 0x7FFFFFFFu;
    // x = (1 + f / 2^23) 2^(E - 127); it fits into 127 * 2^e = 1.984375 * 2^(e + 6) from e = E - 133 on, or one later
    const int e = static_cast<int>(u >> 23) - 133 + ((u & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    return min(max(e, -100), 100);
}

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

struct SelectParams {
    const int8_t *codes;
    const float *units;
    const uint16_t *q;         // bf16 [rows][H_Q][D]
    int32_t H_Q, H_KV, g, bs;
    int64_t N;
    const int32_t *bt;
    int32_t max_blocks, B;
    const int32_t *seqs, *positions;
    int32_t top_k, sink, recent;
    int32_t *lists;            // [rows][H_KV][top_k]
    uint32_t *err;
};

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMostBlocks = 262144;
constexpr int kSelKeys = 32768;     // keys that a CTA holds

// Scores as unsigned numbers of the same order; 0 and ~0 are no finite score's.
__device__ __forceinline__ uint32_t score_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

// A launch that may start while the kernel before it drains, in clusters of `cluster` CTAs along x.
template <typename P>
kvc_status launch(void (*fn)(P), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream, const P &p)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, p);
    if (e != cudaSuccess) return cuda_status(e);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return KVC_OK;
}


// Scores on the tensor cores for runs of rows of one sequence (kvc_select_tc.cu); KVC_ERR_UNSUPPORTED, with nothing
// launched, for tables that it has no room for.
kvc_status select_tiles(const SelectParams &p, int D, int64_t rows, int sms, cudaStream_t stream);

}  // namespace kvc
