// Kernels configured per device, for the launchers of the rotary write and of attention with modified scores.
#pragma once
#include <mutex>

#include "kvc_decode.cuh"

namespace kvc {

// A kernel with its dynamic shared memory, configured once on every device that it runs on.  Tag: one per kernel.
// ctas_per_sm 0: the device refused the configuration or the query.
template <typename Tag>
DecodeKernel configured(const void *fn, int smem, int threads, bool tmap16)
{
    constexpr int kDevices = 64;
    static std::once_flag once[kDevices];
    static DecodeKernel kernels[kDevices];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return DecodeKernel{nullptr, 0, 0};
    std::call_once(once[dev], [&] {
        DecodeKernel &k = kernels[dev];
        k = DecodeKernel{fn, smem, 0};
        k.threads = threads;
        k.tmap16 = tmap16;
        int n = 0;
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess &&
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) == cudaSuccess)
            k.ctas_per_sm = n;
    });
    return kernels[dev];
}

}  // namespace kvc
