// Block bounds and the choice of blocks for sparse attention.
//
// Bounds of a block and KV head, over its filled places t:  hi_i = max_t k_ti, lo_i = min_t k_ti, kept as int8
// codes ceil(hi / 2^e), floor(lo / 2^e) with the smallest e in [-100, 100] that fits both into 127.  A power of two
// as the unit makes every step exact but the outward rounding, and with queries rounded to integers Q the score
//   s_j = 2^e_j max_g sum_i Q_gi (Q_gi > 0 ? hi_ji : lo_ji)
// is an integer below 127 * 127 * 128 < 2^21 times a power of two: exact in fp32 whatever the order of the sum.  So
// the blocks chosen depend on the inputs alone, not on the grid, and equal scores go to the lower block.
#include <algorithm>

#include "kvc_order.cuh"
#include "kvc_select.cuh"

namespace kvc {

// ------------------------------------------------------------------ bounds layout
static uint64_t bounds_layer_bytes(const kvc_pool *pool)
{
    const uint64_t n = static_cast<uint64_t>(pool->N) * pool->H_KV * (2 * pool->D + 4);
    return (n + 255) / 256 * 256;
}

__device__ __forceinline__ uint32_t max2_bf16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2_bf16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max2_f16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min2_f16(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

struct BoundsParams {
    const uint8_t *base;
    int64_t N;
    int32_t bs, H_KV, layer;
    const int32_t *slots;
    int64_t rows;
    int32_t rows_per_cta;
    int8_t *codes;             // this layer's [N][H_KV][2][D]
    float *units;              // [N][H_KV]
    const float *s_k;          // this layer's key scales [H_KV][D] or nullptr
    uint32_t *err;
};

constexpr int kBoundsThreads = 256;
constexpr int kBoundsWarps = kBoundsThreads / 32;

// grid (row chunk, heads of a CTA: one for each warp).  A CTA finds the chunk's last rows of blocks, then its warps take a (block, head) each, the next
// one's keys on their way meanwhile: LPR lanes per key row, 16 bytes a lane, 32 / LPR rows at a time; the channels'
// extremes in packed halves.  Across the row's lanes each halving step passes on half the channels, so that every lane
// ends with 2 or 4 channels of its own to round and store.  65 500 tokens of 8 heads take 18 us on an e4m3 pool (76 MB, 4.2
// TB/s: 400 instructions a block and head, warps waiting for the pipe of the conversions and extremes, issue slots 64 % and
// HBM 40 % busy), 27.5 on a bf16 one (143 MB, 5.2 TB/s), 23.6 on an int4 one (42 MB; 565 instructions); with every lane finishing all of its row's channels and each block's address divided out, 31 and more.  64 single tokens 2.2 us.
// With 32 heads a CTA for all of them took 10.1 us for 83 runs of 972 tokens in all (bf16), one for eight 5.5.
template <int D, int KIND>
__global__ void __launch_bounds__(kBoundsThreads, KIND == KV_BF16 && D == 128 ? 3 : 4) bounds_kernel(const BoundsParams p)
{
    constexpr int BITS = KIND == KV_BF16 ? 16 : (KIND == KV_E4M3 ? 8 : 4);
    constexpr int ROW = D * BITS / 8;             // bytes of a key row
    constexpr int LPR = ROW / 16;                 // lanes per row
    constexpr int RPS = 32 / LPR;                 // rows per step
    constexpr int E = D / LPR;                    // channels of a lane's 16 bytes
    constexpr int P = E / 2;                      // packed pairs
    constexpr int KEEP = P / RPS;                 // pairs that a lane finishes
    constexpr int U = 16 / RPS;                   // steps at a time: 16 rows
    __shared__ int2 ends[kBoundsThreads];         // (block, place) of the last rows of this chunk's blocks
    __shared__ int32_t n_ends;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) n_ends = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    const int64_t r = static_cast<int64_t>(blockIdx.x) * p.rows_per_cta + tid;
    if (tid < p.rows_per_cta && r < p.rows) {
        const int32_t slot = __ldg(p.slots + r);
        if (slot < -1 || (slot >= 0 && slot / p.bs >= p.N)) {
            atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
        } else if (slot >= 0) {   // rows of a block ascend, not always by one
            const int32_t blk = slot / p.bs, behind = r + 1 < p.rows ? __ldg(p.slots + r + 1) : -1;
            if (behind < 0 || behind / p.bs != blk) ends[atomicAdd(&n_ends, 1)] = make_int2(blk, slot - blk * p.bs);
        }
    }
    __syncthreads();
    const int c = lane % LPR, sub = lane / LPR;
    const int h0 = blockIdx.y * kBoundsWarps, heads = min(p.H_KV - h0, kBoundsWarps);   // this CTA's; h counts from h0
    const int count = n_ends;
    const uint8_t *layer = p.base + static_cast<int64_t>(p.layer) * p.N * p.H_KV * (2ll * p.bs * ROW) + h0 * (2 * p.bs * ROW) + 16 * c;

    // rows t0 + sub, t0 + sub + RPS, ... of the keys of (end, head); past the last row: the last one again
    auto fetch = [&](int i, int h, int t0, uint4 (&v)[U]) {
        const int2 e = ends[i];
        const uint8_t *keys = layer + (static_cast<int64_t>(e.x) * p.H_KV + h) * (2 * p.bs * ROW);
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = *reinterpret_cast<const uint4 *>(keys + min(t0 + sub + u * RPS, e.y) * ROW);
    };
    auto advance = [&](int &i, int &h) {
        h += kBoundsWarps;
        while (h >= heads) {
            h -= heads;
            ++i;
        }
    };
    int i = 0, h = warp - kBoundsWarps;
    advance(i, h);
    uint4 v[U];
    if (i < count) fetch(i, h, 0, v);
    while (i < count) {
        const int32_t blk = ends[i].x;
        const int n = ends[i].y + 1;
        int i2 = i, h2 = h;
        advance(i2, h2);
        uint32_t hi[P], lo[P];
#pragma unroll
        for (int x = 0; x < P; ++x) {   // -inf, +inf: no key yet
            hi[x] = KIND == KV_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
            lo[x] = KIND == KV_BF16 ? 0x7F807F80u : 0x7C007C00u;
        }
        for (int t0 = 0; t0 < n; t0 += 16) {
            uint4 cur[U];
#pragma unroll
            for (int u = 0; u < U; ++u) cur[u] = v[u];
            if (t0 + 16 < n) fetch(i, h, t0 + 16, v);
            else if (i2 < count) fetch(i2, h2, 0, v);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t w[4] = {cur[u].x, cur[u].y, cur[u].z, cur[u].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if constexpr (KIND == KV_BF16) {
                        hi[k] = max2_bf16(hi[k], w[k]);
                        lo[k] = min2_bf16(lo[k], w[k]);
                    } else if constexpr (KIND == KV_E4M3) {
                        uint32_t a, b;
                        e4m3x4_to_f16x2x2(w[k], a, b);
                        hi[2 * k] = max2_f16(hi[2 * k], a);
                        lo[2 * k] = min2_f16(lo[2 * k], a);
                        hi[2 * k + 1] = max2_f16(hi[2 * k + 1], b);
                        lo[2 * k + 1] = min2_f16(lo[2 * k + 1], b);
                    } else {   // pair m of word k: channels 8k + m and 8k + m + 4
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            const uint32_t a = nibbles_to_f16x2(w[k] >> (4 * m));
                            hi[4 * k + m] = max2_f16(hi[4 * k + m], a);
                            lo[4 * k + m] = min2_f16(lo[4 * k + m], a);
                        }
                    }
                }
            }
        }
        // across the lanes of a channel: keep half the pairs, pass on the other half
        int x0 = 0;
#pragma unroll
        for (int o = 16, m = P; o >= LPR; o >>= 1) {
            m >>= 1;
            const bool up = (lane & o) != 0;
            x0 += up ? m : 0;
#pragma unroll
            for (int x = 0; x < P / 2; ++x) {
                if (x >= m) break;
                const uint32_t a = __shfl_xor_sync(kFull, up ? hi[x] : hi[x + m], o);
                const uint32_t b = __shfl_xor_sync(kFull, up ? lo[x] : lo[x + m], o);
                const uint32_t ka = up ? hi[x + m] : hi[x], kb = up ? lo[x + m] : lo[x];
                hi[x] = KIND == KV_BF16 ? max2_bf16(ka, a) : max2_f16(ka, a);
                lo[x] = KIND == KV_BF16 ? min2_bf16(kb, b) : min2_f16(kb, b);
            }
        }
        // pair x of the lane: channels first + 2 x and the next one; int4: first + x and first + x + 4
        const int first = E * c + (KIND == KV_INT4 ? 8 * (x0 >> 2) + (x0 & 3) : 2 * x0);
        float y[2][KEEP][2];
        uint32_t top = 0u;   // magnitudes as bits: a NaN's are above infinity's
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int x = 0; x < KEEP; ++x) {
                const uint32_t w = which ? lo[x] : hi[x];
                float2 f;
                if constexpr (KIND == KV_BF16) f = make_float2(bf16_lo(w), bf16_hi(w));
                else f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
                if constexpr (KIND != KV_BF16) {
                    const float *sc = p.s_k + static_cast<int64_t>(h0 + h) * D + first + (KIND == KV_INT4 ? x : 2 * x);
                    f.x *= __ldg(sc);
                    f.y *= __ldg(sc + (KIND == KV_INT4 ? 4 : 1));
                }
                y[which][x][0] = f.x;
                y[which][x][1] = f.y;
                top = max(top, max(__float_as_uint(f.x) & 0x7FFFFFFFu, __float_as_uint(f.y) & 0x7FFFFFFFu));
            }
        const int e = unit_exponent(__uint_as_float(__reduce_max_sync(kFull, top)));
        const float inv = exp2_int(-e);
        const int64_t rec = static_cast<int64_t>(blk) * p.H_KV + h0 + h;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            uint32_t code[KEEP][2];
#pragma unroll
            for (int x = 0; x < KEEP; ++x)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    // rounded outward, so that a product that is too small for fp32 still counts as one (inv is a power of two:
                    // all others are exact); a NaN becomes the first bound that it is compared with
                    const float z = which ? __fmul_rd(y[which][x][k], inv) : __fmul_ru(y[which][x][k], inv);
                    code[x][k] = static_cast<uint32_t>(which ? __float2int_rd(fminf(fmaxf(z, -127.f), 127.f))
                                                             : __float2int_ru(fmaxf(fminf(z, 127.f), -127.f))) & 255u;
                }
            int8_t *dst = p.codes + rec * (2 * D) + which * D + first;
            if constexpr (KIND == KV_INT4) {
                static_assert(KIND != KV_INT4 || KEEP == 2, "two neighbours, twice");
                *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(code[0][0] | (code[KEEP - 1][0] << 8));
                *reinterpret_cast<uint16_t *>(dst + 4) = static_cast<uint16_t>(code[0][1] | (code[KEEP - 1][1] << 8));
            } else if constexpr (KEEP == 2) {
                *reinterpret_cast<uint32_t *>(dst) = code[0][0] | (code[0][1] << 8) | (code[1][0] << 16) | (code[1][1] << 24);
            } else {
                static_assert(KIND == KV_INT4 || KEEP <= 2, "whole words");
                *reinterpret_cast<uint16_t *>(dst) = static_cast<uint16_t>(code[0][0] | (code[0][1] << 8));
            }
        }
        if (lane == 0) p.units[rec] = exp2_int(e);
        i = i2;
        h = h2;
    }
}

// ------------------------------------------------------------------ selection
// One row and KV head, by a cluster of cs CTAs (a power of two up to 8).  CTA `rank` scores its part of the row's blocks
// into `keys` in shared memory.  Lists of up to 128 blocks are ranked from a few candidates; for longer ones, and for
// many equal keys, the k-th largest key is found digit by digit over the cluster's histograms, and each CTA writes its
// part of the list in order.
// One row of 512 blocks and 8 KV heads takes 7.1 us back to back: launch, table and codes 4, the groups' maxima, the
// limit, the candidates and their ranks a barrier each (10.2 with the digits alone).  16 rows of 8192 blocks (273 MB) 59
// us: the scores stream at 7 TB/s, then every CTA of the one wave ranks at once.  The next records copied to shared memory
// during the products left room for fewer CTAs (73 us).
template <int D>
__device__ __forceinline__ void select_row(const SelectParams &p, const int64_t row, const int h, const int cs, const int rank, uint32_t *keys)
{
    constexpr int LPR = D / 16;          // lanes per record: 16 channels each
    constexpr int RPS = 32 / LPR;        // records per step
    constexpr int U = 4;                 // steps at a time
    __shared__ __align__(16) uint32_t qw[32][2][D / 4];   // the group's queries: positive parts, negative parts, int8
    __shared__ __align__(16) uint32_t hist[2][256], sum[256];
    __shared__ __align__(16) uint32_t cand_key[kCandRow + 4];
    __shared__ int32_t cand_block[kCandRow];
    __shared__ uint32_t n_cand, limit;
    __shared__ uint32_t top_bits, pick_bin, pick_above, n_valid, n_gt, n_eq;
    __shared__ uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int seq = p.seqs ? __ldg(p.seqs + row) : static_cast<int>(row);
    const int pos = __ldg(p.positions + row);
    uint4 x[2];   // the group's queries: 16 bytes of each thread, twice
    const int chunks = p.g * D / 8;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = tid + u * kSelThreads;
        x[u] = i < chunks ? __ldg(reinterpret_cast<const uint4 *>(p.q + (row * p.H_Q + static_cast<int64_t>(h) * p.g) * D) + i)
                          : make_uint4(0u, 0u, 0u, 0u);
    }
    if (seq == -1 || pos == -1) return;   // padding: the whole cluster leaves
    int32_t *list = p.lists + (row * p.H_KV + h) * p.top_k;
    if (seq < 0 || seq >= p.B || pos < 0 || pos / p.bs >= p.max_blocks) {
        if (rank == 0 && h == 0 && tid == 0) atomicOr(p.err, KVC_EBIT_RANGE);
        for (int i = rank * kSelThreads + tid; i < p.top_k; i += cs * kSelThreads) list[i] = -1;
        return;
    }
    if (cs > 1) cluster_arrive();
    const int nb = pos / p.bs + 1;
    const int per = (nb + cs - 1) / cs;
    const int j0 = min(nb, rank * per), n = min(nb, j0 + per) - j0;   // this CTA's blocks
    const int32_t *bt = p.bt + static_cast<int64_t>(seq) * p.max_blocks;
    const bool all = nb <= p.top_k;   // every block is listed: no score needed

    // ---- the group's queries as integers
    if (tid == 0) {
        top_bits = 0u;
        n_valid = n_gt = n_eq = n_cand = limit = 0u;
    }
    __syncthreads();
    if (!all) {
        float m = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));   // NaNs drop out
        }
        const uint32_t bits = __reduce_max_sync(kFull, __float_as_uint(m));   // not negative: ordered as integers
        if (lane == 0) atomicMax(&top_bits, bits);
        __syncthreads();
        const float inv = exp2_int(-unit_exponent(__uint_as_float(top_bits)));
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = tid + u * kSelThreads;
            if (i >= chunks) continue;
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            uint32_t pw[2] = {0u, 0u}, nw[2] = {0u, 0u};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float f = (k & 1) ? bf16_hi(w[k >> 1]) : bf16_lo(w[k >> 1]);
                const int z = isnan(f) ? 0 : static_cast<int>(fminf(fmaxf(rintf(f * inv), -127.f), 127.f));
                pw[k >> 2] |= (static_cast<uint32_t>(max(z, 0)) & 255u) << (8 * (k & 3));
                nw[k >> 2] |= (static_cast<uint32_t>(min(z, 0)) & 255u) << (8 * (k & 3));
            }
            const int head = 8 * i / D, word = (8 * i % D) / 4;
            qw[head][0][word] = pw[0];
            qw[head][0][word + 1] = pw[1];
            qw[head][1][word] = nw[0];
            qw[head][1][word + 1] = nw[1];
        }
        __syncthreads();
    }

    // ---- scores of this CTA's blocks, 32 blocks a warp at a time
    const int c = lane % LPR, sub = lane / LPR;
    int next_phys = warp * 32 + lane < n ? __ldg(bt + j0 + warp * 32 + lane) : -1;
    for (int t0 = warp * 32; t0 < n; t0 += kSelThreads) {
        const int j = j0 + t0 + lane;
        const bool in = t0 + lane < n;
        int phys = next_phys;
        next_phys = t0 + kSelThreads + lane < n ? __ldg(bt + j + kSelThreads) : -1;
        if (in && (phys < 0 || static_cast<int64_t>(phys) >= p.N)) {
            if (h == 0) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
            phys = -1;
        }
        const bool forced = j < p.sink || j >= nb - p.recent || all;
        if (all) {
            if (in) keys[t0 + lane] = phys < 0 ? 0u : 0xFFFFFFFFu;
            continue;
        }
        const float unit = phys < 0 ? 0.f : __ldg(p.units + static_cast<int64_t>(phys) * p.H_KV + h);
#pragma unroll
        for (int it = 0; it < 32; it += U * RPS) {
            if (t0 + it >= n) break;
            uint4 hi[U], lo[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int blk = __shfl_sync(kFull, phys, it + u * RPS + sub);
                const int8_t *rec = p.codes + (static_cast<int64_t>(max(blk, 0)) * p.H_KV + h) * (2 * D) + 16 * c;
                hi[u] = __ldg(reinterpret_cast<const uint4 *>(rec));
                lo[u] = __ldg(reinterpret_cast<const uint4 *>(rec + D));
            }
            int best = INT32_MIN;
            for (int g = 0; g < p.g; ++g) {
                const uint4 a = *reinterpret_cast<const uint4 *>(&qw[g][0][4 * c]);
                const uint4 b = *reinterpret_cast<const uint4 *>(&qw[g][1][4 * c]);
                int acc[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    int x = __dp4a(static_cast<int>(hi[u].x), static_cast<int>(a.x), 0);
                    x = __dp4a(static_cast<int>(hi[u].y), static_cast<int>(a.y), x);
                    x = __dp4a(static_cast<int>(hi[u].z), static_cast<int>(a.z), x);
                    x = __dp4a(static_cast<int>(hi[u].w), static_cast<int>(a.w), x);
                    x = __dp4a(static_cast<int>(lo[u].x), static_cast<int>(b.x), x);
                    x = __dp4a(static_cast<int>(lo[u].y), static_cast<int>(b.y), x);
                    x = __dp4a(static_cast<int>(lo[u].z), static_cast<int>(b.z), x);
                    acc[u] = __dp4a(static_cast<int>(lo[u].w), static_cast<int>(b.w), x);
                }
                // sum over the record's lanes, each lane keeping fewer of the U records: record 2 x + y ends in the
                // lanes whose highest two bits (of the record's LPR lanes) are x, y
                constexpr int o1 = LPR / 2, o2 = LPR / 4;
                const bool b1 = (c & o1) != 0, b2 = (c & o2) != 0;
                const int s0 = b1 ? acc[0] : acc[2], s1 = b1 ? acc[1] : acc[3];
                int k0 = b1 ? acc[2] : acc[0], k1 = b1 ? acc[3] : acc[1];
                k0 += __shfl_xor_sync(kFull, s0, o1);
                k1 += __shfl_xor_sync(kFull, s1, o1);
                int v = (b2 ? k1 : k0) + __shfl_xor_sync(kFull, b2 ? k0 : k1, o2);
                if constexpr (LPR == 8) v += __shfl_xor_sync(kFull, v, 1);
                best = max(best, v);
            }
            const int u = (c & (LPR / 2) ? 2 : 0) + (c & (LPR / 4) ? 1 : 0);
            const int at = it + u * RPS + sub;   // of the warp's 32 blocks
            const float un = __shfl_sync(kFull, unit, at);
            const int ph = __shfl_sync(kFull, phys, at);
            const bool fo = __shfl_sync(kFull, static_cast<int>(forced), at) != 0;
            if ((LPR == 4 || (c & 1) == 0) && t0 + at < n)
                keys[t0 + at] = ph < 0 ? 0u : (fo ? 0xFFFFFFFFu : score_key(static_cast<float>(best) * un));
        }
    }
    __syncthreads();
    if (cs > 1) cluster_wait();

    // ---- short lists: the largest keys of 256 groups over the cluster; at least top_k keys reach what top_k of those
    // reach, and not many more.  The first CTA ranks those few by counting.
    if (p.top_k <= kShortList) {
        uint32_t m = 0u;
        for (int i = tid; i < n; i += kSelThreads) m = max(m, keys[i]);
        for (int o = 1; o < cs; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));   // cs a power of two: 256 / cs groups
        const int groups = kSelThreads / cs;
        // lane tid mod cs of a group's threads tells CTA tid mod cs
        cluster_st(cluster_addr(smem_u32(&sum[rank * groups + tid / cs]), tid % cs), m);
        if (cs > 1) cluster_sync();
        else __syncthreads();
        if (warp == 0) {
            uint32_t v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = sum[32 * u + lane];
            const uint32_t lim = reach_limit(v, static_cast<uint32_t>(p.top_k));
            if (lane == 0) limit = lim;
        }
        __syncthreads();
        const uint32_t lim = max(limit, 1u);
        int mine = 0;
        for (int i = tid; i < n; i += kSelThreads) mine += keys[i] >= lim;
        int at = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kFull, at, o);
            if (lane >= o) at += y;
        }
        // every CTA counts all candidates; the first one's count gives them their places, in its shared memory
        const uint32_t warp_has = __shfl_sync(kFull, at, 31);
        uint32_t base = 0u;
        if (lane < cs && warp_has > 0u) base = cluster_add(cluster_addr(smem_u32(&n_cand), lane), warp_has);
        at += static_cast<int>(__shfl_sync(kFull, base, 0)) - mine;
        if (mine > 0)
            for (int i = tid; i < n; i += kSelThreads) {
                const uint32_t k = keys[i];
                if (k >= lim) {
                    if (at < kCandRow) {
                        cluster_st(cluster_addr(smem_u32(&cand_key[at]), 0), k);
                        cluster_st(cluster_addr(smem_u32(&cand_block[at]), 0), static_cast<uint32_t>(j0 + i));
                    }
                    ++at;
                }
            }
        if (cs > 1) cluster_sync();
        else __syncthreads();
        static_assert(kCandRow == kSelThreads, "a thread ranks a candidate");
        if (n_cand <= kCandRow) {
            if (rank == 0) {
                const int c = static_cast<int>(n_cand);
                if (tid < 4) cand_key[c + tid] = 0u;   // whole fours
                __syncthreads();
                const uint32_t k = tid < c ? cand_key[tid] : 0xFFFFFFFFu;
                const int blk = tid < c ? cand_block[tid] : -1;
                const uint4 *k4 = reinterpret_cast<const uint4 *>(cand_key);
                int larger = 0;
#pragma unroll 8
                for (int i = 0; i < (c + 3) / 4; ++i) {
                    const uint4 v = k4[i];
                    larger += (v.x > k) + (v.y > k) + (v.z > k) + (v.w > k);
                }
                bool pick = tid < c && larger < p.top_k;
                if (__syncthreads_count(pick) > p.top_k) {   // equal keys at the border: the lower blocks
                    if (pick)
                        for (int i = 0; i < c; ++i) larger += cand_key[i] == k && cand_block[i] < blk;
                    pick = pick && larger < p.top_k;
                }
                sum[tid] = pick ? static_cast<uint32_t>(blk) : 0x7FFFFFFFu;
                const int picks = __syncthreads_count(pick);
                const int4 *b4 = reinterpret_cast<const int4 *>(sum);
                int place = 0;
#pragma unroll 8
                for (int i = 0; i < (c + 3) / 4; ++i) {
                    const int4 v = b4[i];
                    place += (v.x < blk) + (v.y < blk) + (v.z < blk) + (v.w < blk);
                }
                if (pick) list[place] = blk;
                for (int i = picks + tid; i < p.top_k; i += kSelThreads) list[i] = -1;
            }
            return;
        }
        __syncthreads();   // many equal keys: all of them are counted below
    }

    // ---- the k-th largest key
    {
        uint32_t valid = 0u;
        for (int i = tid; i < n; i += kSelThreads) valid += keys[i] != 0u;
        valid = __reduce_add_sync(kFull, valid);
        if (lane == 0) atomicAdd(&n_valid, valid);
    }
    for (int i = tid; i < 512; i += kSelThreads) (&hist[0][0])[i] = 0u;
    if (cs > 1) cluster_sync();
    else __syncthreads();
    uint32_t valid_in_all = 0u;
    for (int r = 0; r < cs; ++r) valid_in_all += cluster_ld(cluster_addr(smem_u32(&n_valid), r));
    uint32_t threshold = 0u, want = 0u;   // keys above the threshold are listed, and `want` keys equal to it
    if (valid_in_all > static_cast<uint32_t>(p.top_k)) {
        want = static_cast<uint32_t>(p.top_k);
        uint32_t mask = 0u;
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
            const int shift = 24 - 8 * pass;
            uint32_t *hs = hist[pass & 1];
            for (int i = tid; i < n; i += kSelThreads) {
                const uint32_t k = keys[i];
                if (k != 0u && (k & mask) == threshold) atomicAdd(&hs[(k >> shift) & 255u], 1u);
            }
            if (cs > 1) cluster_sync();
            else __syncthreads();
            uint32_t s = 0u;
            for (int r = 0; r < cs; ++r) s += cluster_ld(cluster_addr(smem_u32(&hs[tid]), r));
            sum[tid] = s;
            __syncthreads();
            if (warp == 0) {   // lane l: bins 255 - 8 l downwards
                uint32_t mine = 0u;
#pragma unroll
                for (int x = 0; x < 8; ++x) mine += sum[255 - 8 * lane - x];
                uint32_t inc = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t y = __shfl_up_sync(kFull, inc, o);
                    if (lane >= o) inc += y;
                }
                uint32_t above = inc - mine;
                if (above < want && inc >= want)
                    for (int x = 0; x < 8; ++x) {
                        const uint32_t s1 = sum[255 - 8 * lane - x];
                        if (above + s1 >= want) {
                            pick_bin = static_cast<uint32_t>(255 - 8 * lane - x);
                            pick_above = above;
                            break;
                        }
                        above += s1;
                    }
            }
            __syncthreads();
            threshold |= pick_bin << shift;
            mask |= 255u << shift;
            want -= pick_above;
            hist[(pass + 1) & 1][tid] = 0u;   // last read, by any CTA, before this pass's barrier
            __syncthreads();
        }
    }

    // ---- the list, in order of the blocks
    {
        uint32_t gt = 0u, eq = 0u;
        for (int i = tid; i < n; i += kSelThreads) {
            const uint32_t k = keys[i];
            gt += k > threshold;
            eq += k != 0u && k == threshold;
        }
        gt = __reduce_add_sync(kFull, gt);
        eq = __reduce_add_sync(kFull, eq);
        if (lane == 0) {
            atomicAdd(&n_gt, gt);
            atomicAdd(&n_eq, eq);
        }
    }
    if (cs > 1) cluster_sync();
    else __syncthreads();
    uint32_t gt_before = 0u, eq_before = 0u, listed = 0u, eq_all = 0u;
    for (int r = 0; r < cs; ++r) {
        const uint32_t a = cluster_ld(cluster_addr(smem_u32(&n_gt), r)), b = cluster_ld(cluster_addr(smem_u32(&n_eq), r));
        if (r < rank) {
            gt_before += a;
            eq_before += b;
        }
        listed += a;
        eq_all += b;
    }
    listed += min(eq_all, want);
    for (int base = 0; base < n; base += kSelThreads) {
        const int i = base + tid;
        const uint32_t k = i < n ? keys[i] : 0u;
        const bool gt = k > threshold, eq = k != 0u && k == threshold;
        const uint32_t mg = __ballot_sync(kFull, gt), me = __ballot_sync(kFull, eq);
        if (lane == 0) {
            warp_gt[warp] = __popc(mg);
            warp_eq[warp] = __popc(me);
        }
        __syncthreads();
        uint32_t g0 = gt_before, e0 = eq_before;
        for (int w = 0; w < kSelWarps; ++w) {
            if (w < warp) {
                g0 += warp_gt[w];
                e0 += warp_eq[w];
            }
            gt_before += warp_gt[w];
            eq_before += warp_eq[w];
        }
        const uint32_t below = (1u << lane) - 1u;
        g0 += __popc(mg & below);
        e0 += __popc(me & below);
        if (gt || (eq && e0 < want)) list[g0 + min(e0, want)] = j0 + i;
        __syncthreads();
    }
    for (int i = static_cast<int>(listed) + rank * kSelThreads + tid; i < p.top_k; i += cs * kSelThreads) list[i] = -1;
    if (cs > 1) cluster_sync();   // a CTA's shared memory stays until the others have read it
}

// grid (C x rows, KV head), clusters of C CTAs along x
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p)
{
    extern __shared__ uint32_t keys[];
    const unsigned cs = cluster_size();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    int row = static_cast<int>(blockIdx.x / cs), h = blockIdx.y;
    if (p.longest_first) {
        const int unit = static_cast<int>((blockIdx.y * gridDim.x + blockIdx.x) / cs);
        h = unit % gridDim.y;
        row = row_of_rank<kSelThreads>(p.positions, gridDim.x / cs, p.bs, p.max_blocks, unit / gridDim.y);
    }
    select_row<D>(p, row, h, static_cast<int>(cs), static_cast<int>(cluster_rank()), keys);
}

// The rows that select_tiles left unlisted.  grid (8 rows, KV head)
constexpr int kRestRows = 8;
template <int D>
__global__ void __launch_bounds__(kSelThreads) select_rest_kernel(const SelectParams p, const int64_t rows)
{
    extern __shared__ uint32_t keys[];
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRestRows;
    const int lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t r = r0 + lane;
    const bool mine = lane < kRestRows && r < rows && p.lists[(r * p.H_KV + blockIdx.y) * p.top_k] == kUnlisted;
    uint32_t todo = __ballot_sync(kFull, mine);
    __syncthreads();   // no row is written before every warp has looked
    for (; todo; todo &= todo - 1u) {
        select_row<D>(p, r0 + __ffs(todo) - 1, blockIdx.y, 1, 0, keys);
        __syncthreads();
    }
}

static bool aligned(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

// Whether rows are scored together.  Alone, a row's cost per block is its group's int8 products, and at least the
// bounds' way out of L2 (that of four heads); together, a tile of rows walks all blocks once per sequence it holds, one
// tile to an SM at a time, whatever it holds.  Measured at 2048 blocks, 8 KV heads of 4 query heads: 64 rows 41 us
// alone, 62 together; 128 rows 69 and 63; 512 rows 244 and 64.  One query head per KV head, 32 of them, 128 rows: 168
// and 110; groups that do not divide 32 columns (3, 5), 128 rows: 62 and 79 alone, 147 and 152 together.
// The host does not know which sequence has how many rows, and B counts the table's.  So a chunk and decoding rows in one
// call are planned for the worse of both: a 512-row chunk (65 us alone) takes 334 us with 7 single rows of other sequences
// and 710 with 15 (a tile's sequences are walked one after another), 303 with 63 (every row goes alone).  Two calls take 81,
// 86 and 120.
static bool rows_together(const SelectParams &p, int64_t rows, int sms)
{
    const int64_t RT = std::min(32, 128 / p.g);
    const int64_t walks = std::min(rows, (rows + RT - 1) / RT + p.B - 1) * p.H_KV;
    const int64_t waves = (walks + sms - 1) / sms;
    const bool whole = p.g == 2 || p.g == 4 || p.g == 8;
    return rows * p.H_KV * std::max(p.g, 4) >= waves * (whole ? 4000 : (p.g == 1 ? 6500 : 10000));
}

template <int D>
static kvc_status launch_rest(const SelectParams &p, int64_t rows, cudaStream_t stream)
{
    struct Tag {};
    const DecodeKernel k = configured<Tag>(reinterpret_cast<const void *>(&select_rest_kernel<D>), 4 * kSelKeys, kSelThreads, false);
    if (k.ctas_per_sm <= 0) return KVC_ERR_CUDA;
    return launch(&select_rest_kernel<D>, dim3(static_cast<unsigned>((rows + kRestRows - 1) / kRestRows), p.H_KV), kSelThreads,
                  4 * static_cast<size_t>(p.max_blocks), 1, stream, p, rows);
}

template <int D>
static kvc_status launch_select(const SelectParams &p, int64_t rows, int sms, cudaStream_t stream)
{
    struct Tag {};
    const DecodeKernel k = configured<Tag>(reinterpret_cast<const void *>(&select_kernel<D>), 4 * kSelKeys, kSelThreads, false);
    if (k.ctas_per_sm <= 0) return KVC_ERR_CUDA;
    const int64_t units = rows * p.H_KV;
    // CTAs of a row: one up to 256 blocks (its barriers are cheaper than the cluster's), else so many that each has 256
    // blocks while they fill the GPU twice over, or 128 while they leave half of it free.  Measured, 8 KV heads: one row
    // of 256 blocks 6.1 us with one CTA, 6.6 with two; 512 blocks 8.2, 7.1 and 6.7 with one, two and four; 8 rows of 512
    // blocks 8.0 with two, 8.5 with four; 16 rows of 8192 blocks 57.5 with four, 61.4 with eight.
    // A CTA has 4096 blocks at most, or 2048 while they fill the GPU four times over: it takes 13 us for 1024 blocks, so one
    // long row would outlast the others.  64 rows of up to 8192 blocks, with one, two and four: 100, 59 and 61 us (all of
    // them long: 212, 192 and 201); 32 rows, with two and four: 54 and 35 (100 and 105).
    int c = 1;
    auto more = [&] {
        return (units * c < 2ll * sms && p.max_blocks > 256 * c) ||
               (units * c * 2 <= sms && p.max_blocks > 256 && p.max_blocks > 128 * c) ||
               (units * c < 4ll * sms && p.max_blocks > 2048 * c) || p.max_blocks > 4096 * c;
    };
    while (c < 8 && more()) c *= 2;
    // Measured by number and longest first: 64 rows of up to 8192 blocks 72 and 59 us, 32 rows 44 and 35; 128 rows of up to
    // 2048 blocks 42 and 34; 64 rows of up to 512 blocks 12.2 and 10.9 (all long: 20.3 and 21.8); 16 rows of 8192 blocks
    // 59.5 and 60.6.
    SelectParams sp = p;
    sp.longest_first = longest_first(rows, p.B, units, c, sms);
    if (rows * c > 0x7FFFFFFF) return KVC_ERR_UNSUPPORTED;
    const int per = (p.max_blocks + c - 1) / c;
    return launch(&select_kernel<D>, dim3(static_cast<unsigned>(rows * c), p.H_KV), kSelThreads, 4 * static_cast<size_t>(per), c,
                  stream, sp);
}

template <int D, int KIND>
static kvc_status launch_bounds(const kvc_pool *pool, BoundsParams &p, cudaStream_t stream)
{
    // Few rows are a decoding batch's, nearly each the last one of its block: as many CTAs as rows, until there are four
    // for every SM.
    const int64_t per_chunk = (p.H_KV + kBoundsWarps - 1) / kBoundsWarps, most = std::max<int64_t>(4 * pool->num_sms / per_chunk, 1);
    p.rows_per_cta = static_cast<int32_t>(std::min<int64_t>((p.rows + most - 1) / most, kBoundsThreads));
    const int64_t chunks = (p.rows + p.rows_per_cta - 1) / p.rows_per_cta;
    return launch(&bounds_kernel<D, KIND>, dim3(static_cast<unsigned>(chunks), static_cast<unsigned>(per_chunk)), kBoundsThreads, 0, 1,
                  stream, p);
}

}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_bounds_bytes(const kvc_pool *pool, uint64_t *bytes)
{
    if (!pool || !bytes) return KVC_ERR_ARG;
    *bytes = bounds_layer_bytes(pool) * pool->L;
    return KVC_OK;
}

extern "C" kvc_status kvc_update_bounds(kvc_pool *pool, int32_t layer, const int32_t *slots, int64_t n_rows,
                                        void *bounds, uint64_t bounds_bytes, kvc_stream_t stream)
{
    if (!pool || n_rows < 0 || n_rows > 0x7FFFFFFF || layer < 0 || layer >= pool->L) return KVC_ERR_ARG;
    if (!bounds || !aligned(bounds, 256) || bounds_bytes < bounds_layer_bytes(pool) * pool->L) return KVC_ERR_ARG;
    if (n_rows == 0) return KVC_OK;
    if (!slots || !aligned(slots, 4)) return KVC_ERR_ARG;
    const kvc_status st = check_device(pool);
    if (st != KVC_OK) return st;
    BoundsParams p{};
    p.base = pool->base;
    p.N = pool->N;
    p.bs = pool->bs;
    p.H_KV = pool->H_KV;
    p.layer = layer;
    p.slots = slots;
    p.rows = n_rows;
    p.codes = static_cast<int8_t *>(bounds) + bounds_layer_bytes(pool) * layer;
    p.units = reinterpret_cast<float *>(p.codes + static_cast<size_t>(pool->N) * pool->H_KV * 2 * pool->D);
    p.s_k = pool->scales ? pool->scales + static_cast<size_t>(layer) * 2 * pool->H_KV * pool->D : nullptr;
    p.err = pool->err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (pool->dtype == KVC_FP8_E4M3) return launch_bounds<128, KV_E4M3>(pool, p, s);
    if (pool->dtype == KVC_INT4) return launch_bounds<128, KV_INT4>(pool, p, s);
    return pool->D == 64 ? launch_bounds<64, KV_BF16>(pool, p, s) : launch_bounds<128, KV_BF16>(pool, p, s);
}

extern "C" kvc_status kvc_select_blocks(kvc_pool *pool, int32_t layer, const void *bounds, uint64_t bounds_bytes,
                                        const void *q, int32_t num_q_heads, const int32_t *block_tables,
                                        int32_t max_blocks, int32_t B, const int32_t *seq_ids,
                                        const int32_t *positions, int64_t n_rows, int32_t top_k, int32_t sink,
                                        int32_t recent, int32_t *selected, kvc_stream_t stream)
{
    if (!pool || B < 0 || n_rows < 0 || n_rows > 0x7FFFFFFF || num_q_heads <= 0 || num_q_heads % pool->H_KV != 0)
        return KVC_ERR_ARG;
    if (sink < 0 || recent < 1 || top_k > 65536 || static_cast<int64_t>(sink) + recent > top_k) return KVC_ERR_ARG;
    if (num_q_heads / pool->H_KV > 32) return KVC_ERR_UNSUPPORTED;
    if (!bounds || !aligned(bounds, 256) || bounds_bytes < bounds_layer_bytes(pool) * pool->L) return KVC_ERR_ARG;
    if (n_rows == 0) return KVC_OK;
    if (layer < 0 || layer >= pool->L || max_blocks <= 0 || (!seq_ids && n_rows > B)) return KVC_ERR_ARG;
    if (max_blocks > kSelMostBlocks) return KVC_ERR_UNSUPPORTED;
    if (!q || !block_tables || !positions || !selected || !aligned(q, 16) || !aligned(block_tables, 4) ||
        !aligned(positions, 4) || !aligned(seq_ids, 4) || !aligned(selected, 4))
        return KVC_ERR_ARG;
    const kvc_status st = check_device(pool);
    if (st != KVC_OK) return st;
    SelectParams p{};
    p.codes = static_cast<const int8_t *>(bounds) + bounds_layer_bytes(pool) * layer;
    p.units = reinterpret_cast<const float *>(p.codes + static_cast<size_t>(pool->N) * pool->H_KV * 2 * pool->D);
    p.q = static_cast<const uint16_t *>(q);
    p.H_Q = num_q_heads;
    p.H_KV = pool->H_KV;
    p.g = num_q_heads / pool->H_KV;
    p.bs = pool->bs;
    p.N = pool->N;
    p.bt = block_tables;
    p.max_blocks = max_blocks;
    p.B = B;
    p.seqs = seq_ids;
    p.positions = positions;
    p.top_k = top_k;
    p.sink = sink;
    p.recent = recent;
    p.lists = selected;
    p.err = pool->err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (seq_ids && top_k <= kShortList && max_blocks <= kSelKeys && rows_together(p, n_rows, pool->num_sms)) {
        const kvc_status tiled = select_tiles(p, pool->D, n_rows, s);
        if (tiled != KVC_OK) return tiled;
        return pool->D == 64 ? launch_rest<64>(p, n_rows, s) : launch_rest<128>(p, n_rows, s);
    }
    return pool->D == 64 ? launch_select<64>(p, n_rows, pool->num_sms, s) : launch_select<128>(p, n_rows, pool->num_sms, s);
}
