// Rows in the order of what they read, for grids whose rows differ in length: an SM that has several CTAs of long rows,
// or a long row that begins last, ends a launch late.
#pragma once
#include "kvc_decode.cuh"

namespace kvc {

constexpr int kOrderMost = 512;   // rows that are ordered

// Whether a grid of `units` (row, KV head) pairs, c CTAs each, takes its longest rows first: a decoding batch (no more rows
// than sequences) whose CTAs fill the GPU once or a few times.
inline bool longest_first(int64_t rows, int B, int64_t units, int c, int sms)
{
    return rows <= (B < kOrderMost ? B : kOrderMost) && units * c > sms && units <= 8ll * sms;
}

// All threads of a CTA of THREADS: the row of rank r of at most kOrderMost, most blocks first (up to `most` count), in 32
// classes, eight to a factor of two; in a class by number.  Every CTA finds its own row so, from the positions alone (about
// 1 us before its first load of anything else).
template <int THREADS>
__device__ __forceinline__ int row_of_rank(const int32_t *positions, int rows, int bs, int most, int r)
{
    constexpr int PER = kOrderMost / THREADS;
    __shared__ int in_class[32];
    __shared__ __align__(16) uint32_t cls[kOrderMost / 4];   // of every row, in bytes
    const int tid = threadIdx.x, lane = tid & 31;
    int pos[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) pos[u] = tid + THREADS * u < rows ? __ldg(positions + tid + THREADS * u) : -1;
    if (tid < 32) in_class[tid] = 0;
    __syncthreads();
    auto eighths = [](int n) { return static_cast<int>(__float_as_uint(static_cast<float>(n)) >> 20); };   // of octaves
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        const int i = tid + THREADS * u;
        const int n = pos[u] < 0 ? 0 : min(pos[u] / bs, most - 1) + 1;
        const int c = i < rows ? min(eighths(most) - eighths(n), 31) : 32;
        reinterpret_cast<uint8_t *>(cls)[i] = static_cast<uint8_t>(c);
        if (c < 32) atomicAdd(&in_class[c], 1);
    }
    __syncthreads();
    auto before = [&](int n) {   // sum of the lanes before this one
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, sum, o);
            if (lane >= o) sum += y;
        }
        return sum - n;
    };
    // the class that holds rank r, and how many rows of it come before
    const int n = in_class[lane], ahead = before(n);
    const int c = __popc(__ballot_sync(kFull, ahead + n <= r));
    const int left = r - __shfl_sync(kFull, ahead, c);
    // a lane's rows are kOrderMost / 32 neighbours
    constexpr int kWords = kOrderMost / 128;
    uint32_t is[kWords];
    int mine = 0;
#pragma unroll
    for (int w = 0; w < kWords; ++w) {
        is[w] = __vcmpeq4(cls[lane * kWords + w], 0x01010101u * static_cast<uint32_t>(c));
        mine += __popc(is[w]) >> 3;
    }
    int row = 0, k = left - before(mine);   // the k-th of this lane's
    if (k >= 0 && k < mine) {
#pragma unroll
        for (int x = 0; x < kOrderMost / 32; ++x)
            if ((is[x / 4] >> (8 * (x % 4))) & 1u) {
                if (k == 0) row = lane * (kOrderMost / 32) + x;
                --k;
            }
    }
    return __reduce_max_sync(kFull, row);
}

}  // namespace kvc
