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

// One warp: the cut that lists `want` of more than `want` keys that are not 0.  count(m, c): this lane's keys >= m[i];
// lo, hi: the least and the largest key below ~0; forced: the number of keys ~0.  SMALL: fewer than 1024 keys.
template <bool SMALL, typename Count>
__device__ __forceinline__ Cut find_cut(uint32_t want, uint32_t forced, uint32_t lo, uint32_t hi, Count count)
{
    if (forced >= want) return {0xFFFFFFFEu, 0u};   // the forced ones fill the list
    uint32_t n_hi = forced;   // keys > hi: fewer than wanted; keys >= lo: more
    for (int it = 0; lo < hi; ++it) {
        uint32_t m[3], c[3];
        quarter(lo, hi, it < 12, m);
        count(m, c);
        if constexpr (SMALL) {
            const uint32_t all = __reduce_add_sync(kFull, c[0] | (c[1] << 10) | (c[2] << 20));
            c[0] = all & 1023u;
            c[1] = (all >> 10) & 1023u;
            c[2] = all >> 20;
        } else {
#pragma unroll
            for (int i = 0; i < 3; ++i) c[i] = __reduce_add_sync(kFull, c[i]);
        }
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
constexpr int kCand = 384;
struct alignas(16) Candidates {
    uint32_t key[kCand];
    int32_t block[kCand];
};
constexpr int kPickMost = 2 * kCand * 32;   // blocks of a row that pick_row serves: a bit each in the candidates' place

// One warp: the list of a row from n candidates, n <= 32 S, of `blocks` blocks, in order of the blocks.
template <int S>
__device__ __forceinline__ void list_candidates(Candidates &s, int n, int blocks, int32_t *list, int top_k, int lane)
{
    uint32_t k[S], forced = 0u, lo = 0xFFFFFFFFu, hi = 0u;
    int32_t blk[S];
#pragma unroll
    for (int u = 0; u < S; ++u) {
        const bool in = 32 * u + lane < n;
        k[u] = in ? s.key[32 * u + lane] : 0u;
        blk[u] = in ? s.block[32 * u + lane] : 0;
        const bool top = k[u] == 0xFFFFFFFFu;
        forced += top;
        lo = min(lo, in ? k[u] : 0xFFFFFFFFu);
        hi = max(hi, top ? 0u : k[u]);
    }
    Cut cut{0u, 0u};
    if (n > top_k)
        cut = find_cut<true>(static_cast<uint32_t>(top_k), __reduce_add_sync(kFull, forced), __reduce_min_sync(kFull, lo),
                             __reduce_max_sync(kFull, hi), [&](const uint32_t (&m)[3], uint32_t (&c)[3]) {
#pragma unroll
                                 for (int i = 0; i < 3; ++i) {
                                     c[i] = 0u;
#pragma unroll
                                     for (int u = 0; u < S; ++u) c[i] += k[u] >= m[i];
                                 }
                             });
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
                for (int i = 0; i < n; ++i) before += s.key[i] == cut.above && s.block[i] < blk[u];
            pick[u] = before < cut.equal;
        }
    }
    // a bit for each block, then the blocks in order of the bits
    __syncwarp();
    uint32_t *bits = s.key;
    const int words = blocks / 32, per = (words + 31) / 32;
    for (int i = lane; i < words; i += 32) bits[i] = 0u;
    __syncwarp();
#pragma unroll
    for (int u = 0; u < S; ++u)
        if (pick[u]) atomicOr(&bits[blk[u] >> 5], 1u << (blk[u] & 31));
    __syncwarp();
    int mine = 0;
    for (int i = 0; i < per; ++i) mine += lane * per + i < words ? __popc(bits[lane * per + i]) : 0;
    int at = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, at, o);
        if (lane >= o) at += y;
    }
    const int total = __shfl_sync(kFull, at, 31);
    at -= mine;
    for (int i = 0; i < per && lane * per + i < words; ++i)
        for (uint32_t w = bits[lane * per + i]; w; w &= w - 1u) list[at++] = (lane * per + i) * 32 + __ffs(w) - 1;
    for (int i = total + lane; i < top_k; i += 32) list[i] = -1;
}

// One warp: the same for n <= 128 candidates by counting, for each, the larger ones and then the listed ones in lower
// blocks: more additions than a search, but no chain of them.
__device__ __forceinline__ void list_few(Candidates &s, int n, int blocks, int32_t *list, int top_k, int lane)
{
    constexpr int S = 4;
    uint32_t k[S];
    int32_t blk[S], larger[S] = {0, 0, 0, 0};
    const int n4 = (n + 3) / 4;
    if (lane < 4 * n4 - n) {   // whole fours: keys of 0, blocks past all
        s.key[n + lane] = 0u;
        s.block[n + lane] = 0x7FFFFFFF;
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < S; ++u) {
        const bool in = 32 * u + lane < n;
        k[u] = in ? s.key[32 * u + lane] : 0xFFFFFFFFu;
        blk[u] = in ? s.block[32 * u + lane] : -1;
    }
    const uint4 *k4 = reinterpret_cast<const uint4 *>(s.key);
#pragma unroll 4
    for (int j = 0; j < n4; ++j) {
        const uint4 v = k4[j];
#pragma unroll
        for (int u = 0; u < S; ++u) larger[u] += (v.x > k[u]) + (v.y > k[u]) + (v.z > k[u]) + (v.w > k[u]);
    }
    bool pick[S];
    int picks = 0;
#pragma unroll
    for (int u = 0; u < S; ++u) {
        pick[u] = blk[u] >= 0 && larger[u] < top_k;
        picks += pick[u];
    }
    if (__reduce_add_sync(kFull, picks) > top_k) {   // equal keys at the border: the lower blocks
        list_candidates<S>(s, n, blocks, list, top_k, lane);
        return;
    }
    __syncwarp();
    int total = 0;
#pragma unroll
    for (int u = 0; u < S; ++u) {   // the listed blocks, in the keys' place
        const uint32_t m = __ballot_sync(kFull, pick[u]);
        if (pick[u]) s.key[total + __popc(m & ((1u << lane) - 1u))] = static_cast<uint32_t>(blk[u]);
        total += __popc(m);
    }
    const int t4 = (total + 3) / 4;
    if (lane < 4 * t4 - total) s.key[total + lane] = 0x7FFFFFFFu;
    __syncwarp();
    int at[S] = {0, 0, 0, 0};
#pragma unroll 4
    for (int j = 0; j < t4; ++j) {
        const uint4 v = k4[j];
#pragma unroll
        for (int u = 0; u < S; ++u)
            at[u] += (static_cast<int>(v.x) < blk[u]) + (static_cast<int>(v.y) < blk[u]) + (static_cast<int>(v.z) < blk[u]) + (static_cast<int>(v.w) < blk[u]);
    }
#pragma unroll
    for (int u = 0; u < S; ++u)
        if (pick[u]) list[at[u]] = blk[u];
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

// One warp: writes the list of a row from its keys k[0 .. n) in shared memory (n a multiple of 128, unused ones 0).
__device__ __forceinline__ void pick_row(const uint32_t *k, int n, Candidates &s, int32_t *list, int top_k, int lane)
{
    const uint4 *k4 = reinterpret_cast<const uint4 *>(k);
    // the largest keys of 256 groups: at least top_k keys reach what top_k of those reach, and not many more
    if (top_k <= 128) {
        uint32_t m[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
#pragma unroll 4
        for (int i = lane; i < n / 4; i += 64) {
            const uint4 v = k4[i], w = i + 32 < n / 4 ? k4[i + 32] : make_uint4(0u, 0u, 0u, 0u);
            m[0] = max(m[0], v.x), m[1] = max(m[1], v.y), m[2] = max(m[2], v.z), m[3] = max(m[3], v.w);
            m[4] = max(m[4], w.x), m[5] = max(m[5], w.y), m[6] = max(m[6], w.z), m[7] = max(m[7], w.w);
        }
        const uint32_t limit = max(reach_limit(m, static_cast<uint32_t>(top_k)), 1u);
        int mine = 0;
#pragma unroll 4
        for (int i = lane; i < n / 4; i += 32) {
            const uint4 v = k4[i];
            mine += (v.x >= limit) + (v.y >= limit) + (v.z >= limit) + (v.w >= limit);
        }
        int at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, at, o);
            if (lane >= o) at += y;
        }
        const int c = __shfl_sync(kFull, at, 31);
        if (c <= kCand) {
            at -= mine;
#pragma unroll 4
            for (int i = lane; i < n / 4; i += 32) {
                const uint4 v = k4[i];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (w[u] >= limit) {
                        s.key[at] = w[u];
                        s.block[at++] = 4 * i + u;
                    }
            }
            __syncwarp();
            if (c <= 128) list_few(s, c, n, list, top_k, lane);
            else list_candidates<kCand / 32>(s, c, n, list, top_k, lane);
            return;
        }
    }
    // long lists, and runs of equal keys: the cut by counting all keys
    uint32_t valid = 0u, forced = 0u, lo = 0xFFFFFFFFu, hi = 0u;
    for (int i = lane; i < n; i += 32) {
        const uint32_t w = k[i];
        const bool top = w == 0xFFFFFFFFu;
        valid += w != 0u;
        forced += top;
        lo = min(lo, w == 0u ? 0xFFFFFFFFu : w);
        hi = max(hi, top ? 0u : w);
    }
    Cut cut{0u, 0u};
    if (__reduce_add_sync(kFull, valid) > static_cast<uint32_t>(top_k))
        cut = find_cut<false>(static_cast<uint32_t>(top_k), __reduce_add_sync(kFull, forced), __reduce_min_sync(kFull, lo),
                              __reduce_max_sync(kFull, hi), [&](const uint32_t (&m)[3], uint32_t (&c)[3]) {
                                  c[0] = c[1] = c[2] = 0u;
                                  for (int i = lane; i < n / 4; i += 32) {
                                      const uint4 v = k4[i];
#pragma unroll
                                      for (int x = 0; x < 3; ++x) c[x] += (v.x >= m[x]) + (v.y >= m[x]) + (v.z >= m[x]) + (v.w >= m[x]);
                                  }
                              });
    const uint32_t below = (1u << lane) - 1u;
    uint32_t g0 = 0u, e0 = 0u;
    for (int i = 0; i < n; i += 32) {
        const uint32_t w = k[i + lane];
        const bool gt = w > cut.above, eq = w != 0u && w == cut.above;
        const uint32_t mg = __ballot_sync(kFull, gt), me = __ballot_sync(kFull, eq);
        if ((mg | me) == 0u) continue;
        const uint32_t ge = g0 + __popc(mg & below), ee = e0 + __popc(me & below);
        if (gt || (eq && ee < cut.equal)) list[ge + min(ee, cut.equal)] = i + lane;
        g0 += __popc(mg);
        e0 += __popc(me);
    }
    for (int i = static_cast<int>(g0 + min(e0, cut.equal)) + lane; i < top_k; i += 32) list[i] = -1;
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
