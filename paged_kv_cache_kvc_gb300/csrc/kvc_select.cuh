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
    bool longest_first;        // rows are taken in the order of what they read
    uint32_t *err;
};

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelMostBlocks = 262144;
constexpr int kShortList = 128;     // blocks of a list that is ranked from a few candidates
constexpr int kSelKeys = 32768;     // keys that a CTA holds

// Scores as unsigned numbers of the same order; 0 and ~0 are no finite score's.
__device__ __forceinline__ uint32_t score_key(float x)
{
    const uint32_t u = __float_as_uint(x);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float key_score(uint32_t k) { return __uint_as_float((k >> 31) ? (k & 0x7FFFFFFFu) : ~k); }

// Three keys that quarter (lo, hi], lo < hi: lo < m[0] <= m[1] <= m[2] <= hi.  By score, or by the keys themselves.
__device__ __forceinline__ void quarter(uint32_t lo, uint32_t hi, bool by_score, uint32_t (&m)[3])
{
    if (by_score) {
        const float a = key_score(lo), b = key_score(hi);
        m[1] = min(max(score_key(0.5f * a + 0.5f * b), lo + 1u), hi);
        m[0] = min(max(score_key(0.75f * a + 0.25f * b), lo + 1u), m[1]);
        m[2] = min(max(score_key(0.25f * a + 0.75f * b), m[1]), hi);
    } else {
        const uint32_t n = hi - lo;
        m[0] = lo + max(n >> 2, 1u);
        m[1] = max(lo + ((n + 1u) >> 1), m[0]);
        m[2] = max(hi - (n >> 2), m[1]);
    }
}

// What is listed of a set of keys: those above `above`, and the first `equal` of those equal to it.
struct Cut {
    uint32_t above, equal;
};

// One warp: the cut that lists `want` of more than `want` keys that are not 0, S < 32 of them per lane in k (unused: 0).
template <int S>
__device__ __forceinline__ Cut find_cut(const uint32_t (&k)[S], uint32_t want)
{
    uint32_t lo = 0xFFFFFFFFu, hi = 0u, forced = 0u;
#pragma unroll
    for (int u = 0; u < S; ++u) {
        const bool top = k[u] == 0xFFFFFFFFu;
        forced += top;
        lo = min(lo, k[u] == 0u ? 0xFFFFFFFFu : k[u]);
        hi = max(hi, top ? 0u : k[u]);
    }
    forced = __reduce_add_sync(kFull, forced);
    lo = __reduce_min_sync(kFull, lo);
    hi = __reduce_max_sync(kFull, hi);
    if (forced >= want) return {0xFFFFFFFFu, want};   // the forced ones fill the list
    uint32_t n_hi = forced;   // keys > hi: fewer than wanted; keys >= lo: more
    for (int it = 0; lo < hi; ++it) {
        uint32_t m[3], c[3];
        quarter(lo, hi, it < 12, m);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            c[i] = 0u;
#pragma unroll
            for (int u = 0; u < S; ++u) c[i] += k[u] >= m[i];
        }
        const uint32_t all = __reduce_add_sync(kFull, c[0] | (c[1] << 10) | (c[2] << 20));   // 32 S < 1024
        c[0] = all & 1023u;
        c[1] = (all >> 10) & 1023u;
        c[2] = all >> 20;
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (c[i] == want) return {m[i] - 1u, 0u};
        if (c[2] > want) {
            lo = m[2];
        } else if (c[1] > want) {
            lo = m[1];
            hi = m[2] - 1u;
            n_hi = c[2];
        } else if (c[0] > want) {
            lo = m[0];
            hi = m[1] - 1u;
            n_hi = c[1];
        } else {
            hi = m[0] - 1u;
            n_hi = c[0];
        }
    }
    return {lo, want - n_hi};
}

// Keys that a row's list is chosen from, in any order: those at or above a limit that at least top_k keys reach.
constexpr int kCandRow = 256;
constexpr int kCandWords = 2 * kCandRow;   // of a row: keys, then blocks

// One warp: the list of a row from n <= 32 S candidates of `blocks` blocks, the whole of them when n <= top_k.
template <int S>
__device__ __forceinline__ void list_candidates(uint32_t *key, int n, int blocks, int32_t *list, int top_k, int lane)
{
    const int32_t *block = reinterpret_cast<const int32_t *>(key) + kCandRow;
    uint32_t k[S];
    int32_t blk[S];
#pragma unroll
    for (int u = 0; u < S; ++u) {
        const bool in = 32 * u + lane < n;
        k[u] = in ? key[32 * u + lane] : 0u;
        blk[u] = in ? block[32 * u + lane] : 0;
    }
    Cut cut{0u, 0u};
    if (n > top_k) cut = find_cut(k, static_cast<uint32_t>(top_k));
    uint32_t same = 0u;
#pragma unroll
    for (int u = 0; u < S; ++u) same += k[u] != 0u && k[u] == cut.above;
    const bool all_same = __reduce_add_sync(kFull, same) <= cut.equal;
    bool pick[S];
#pragma unroll
    for (int u = 0; u < S; ++u) {
        pick[u] = k[u] > cut.above;
        if (cut.equal != 0u && k[u] != 0u && k[u] == cut.above) {
            uint32_t before = 0u;   // equal ones in lower blocks
            if (!all_same)
                for (int i = 0; i < n; ++i) before += key[i] == cut.above && block[i] < blk[u];
            pick[u] = before < cut.equal;
        }
    }
    __syncwarp();
    const int words = (blocks + 31) / 32, per = (words + 31) / 32;
    int total;
    if (words <= kCandWords) {   // a bit for each block in the candidates' place, then the blocks in order of the bits
        for (int i = lane; i < words; i += 32) key[i] = 0u;
        __syncwarp();
#pragma unroll
        for (int u = 0; u < S; ++u)
            if (pick[u]) atomicOr(&key[blk[u] >> 5], 1u << (blk[u] & 31));
        __syncwarp();
        int mine = 0;
        for (int i = 0; i < per; ++i) mine += lane * per + i < words ? __popc(key[lane * per + i]) : 0;
        int at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, at, o);
            if (lane >= o) at += y;
        }
        total = __shfl_sync(kFull, at, 31);
        at -= mine;
        for (int i = 0; i < per && lane * per + i < words; ++i)
            for (uint32_t w = key[lane * per + i]; w; w &= w - 1u) list[at++] = (lane * per + i) * 32 + __ffs(w) - 1;
    } else {   // too many blocks for that: each listed one counts those before it
        total = 0;
#pragma unroll
        for (int u = 0; u < S; ++u) {
            const uint32_t m = __ballot_sync(kFull, pick[u]);
            if (pick[u]) key[total + __popc(m & ((1u << lane) - 1u))] = static_cast<uint32_t>(blk[u]);
            total += __popc(m);
        }
        __syncwarp();
#pragma unroll
        for (int u = 0; u < S; ++u) {
            int at = 0;
            for (int i = 0; i < total; ++i) at += static_cast<int>(key[i]) < blk[u];
            if (pick[u]) list[at] = blk[u];
        }
    }
    for (int i = total + lane; i < top_k; i += 32) list[i] = -1;
}

// One warp: a limit that at least `want` of the 32 S values reach (0 where fewer are not 0), close to the want-th largest.
template <int S>
__device__ __forceinline__ uint32_t reach_limit(const uint32_t (&v)[S], uint32_t want)
{
    uint32_t lo = 0xFFFFFFFFu, hi = 0u, some = 0u, forced = 0u;   // of the values that are neither 0 nor ~0
#pragma unroll
    for (int u = 0; u < S; ++u) {
        const bool top = v[u] == 0xFFFFFFFFu;
        some += v[u] != 0u;
        forced += top;
        lo = min(lo, v[u] == 0u ? 0xFFFFFFFFu : v[u]);
        hi = max(hi, top ? 0u : v[u]);
    }
    some = __reduce_add_sync(kFull, some | (forced << 16));
    if ((some & 0xFFFFu) < want) return 0u;
    if ((some >> 16) >= want) return 0xFFFFFFFFu;
    lo = __reduce_min_sync(kFull, lo);   // reached by all that are not 0
    hi = __reduce_max_sync(kFull, hi);
    for (int it = 0; it < 20 && lo < hi; ++it) {
        uint32_t m[3], c[3];
        quarter(lo, hi, it < 10, m);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            c[i] = 0u;
#pragma unroll
            for (int u = 0; u < S; ++u) c[i] += v[u] >= m[i];
        }
        const uint32_t all = __reduce_add_sync(kFull, c[0] | (c[1] << 10) | (c[2] << 20));   // 32 S < 1024
        c[0] = all & 1023u;
        c[1] = (all >> 10) & 1023u;
        c[2] = all >> 20;
        uint32_t reached = 0u;
        if (c[2] >= want) lo = m[2], reached = c[2];
        else if (c[1] >= want) lo = m[1], hi = m[2] - 1u, reached = c[1];
        else if (c[0] >= want) lo = m[0], hi = m[1] - 1u, reached = c[0];
        else hi = m[0] - 1u;
        if (reached != 0u && reached <= want + (want >> 2)) break;
    }
    return lo;
}

// A launch that may start while the kernel before it drains, in clusters of `cluster` CTAs along x.
template <typename... P, typename... A>
kvc_status launch(void (*fn)(P...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream, const A &...args)
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, args...);
    if (e != cudaSuccess) return cuda_status(e);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return KVC_OK;
}


// What a list starts with while it waits for select_rest.
constexpr int32_t kUnlisted = -2;

// Scores on the tensor cores for runs of rows of one sequence (kvc_select_tc.cu), lists of up to 128 blocks.  Rows whose
// candidates are too many (equal scores) are left unlisted.
kvc_status select_tiles(const SelectParams &p, int D, int64_t rows, cudaStream_t stream);

}  // namespace kvc
