// Block selection for chunks: many rows of one sequence score the same blocks, so the scores are a matrix product,
// on the fifth-generation tensor cores.
//
// Mathematics.  With the positive and the negative parts of the whole-numbered queries side by side, a score is one
// product of length 2 d:  sum_i Q_i (Q_i > 0 ? hi_i : lo_i) = <(Q+, Q-), (hi, lo)>.  Codes and queries are integers
// up to 127, exact in f16; products are below 2^14 and sums below 2^21, exact in the fp32 accumulator in any order.
//
// A cluster of C CTAs takes RT rows of one KV head; the CTAs share the blocks in tiles of 128 (tile t to CTA t mod C).
// Per tile: D[128 blocks x RT g query columns] = A[128 x 2d] B[2d x RT g].  The blocks are the M rows, so that a
// thread of the epilogue holds one block's products with every query head and takes their maximum without a shuffle.
// B (the queries) stays in shared memory; A is read as int8 into registers while the tile before is multiplied,
// widened to f16 and stored in the 128-byte swizzle.  The keys stay in shared memory, and each row is finished by one
// warp: it gathers the row's keys from the cluster, narrows the k-th largest by counting, and writes the list.
//
// A tile of rows may hold several sequences (runs): they are done one after the other.
#include <algorithm>

#include "kvc_select.cuh"
#include "kvc_tc.cuh"

namespace kvc {

constexpr int kStThreads = 512;
constexpr int kStWarps = kStThreads / 32;
constexpr int kStTile = 128;       // blocks per MMA
constexpr int kStCols = 128;       // query columns at most
constexpr int kStRows = 32;        // rows at most
constexpr int kStPick = 8;         // warps that finish rows

template <int D>
struct StCfg {
    static constexpr int K = 2 * D;
    static constexpr int BANDS = K / 64;            // 128-byte bands of f16
    static constexpr int BAND = 128 * 128;          // bytes of a band of 128 rows
    static constexpr int A = BANDS * BAND;          // bytes
    static constexpr int KEYS = 2 * A;              // offset of the keys: after A and B
    static constexpr int CPR = K / 16;              // 16-byte chunks per record
    static constexpr int STEP = kStThreads / CPR;   // records per pass of the CTA's threads
    static constexpr int U = kStTile / STEP;        // passes per tile
};

struct SelectTileParams {
    SelectParams s;
    int64_t rows;
    int32_t RT;            // rows per tile
    int32_t tiles;         // tiles of blocks per CTA that the keys have room for
};

// Two pairs of f16 from four int8 codes, exact.
__device__ __forceinline__ uint2 s8x4_to_f16(uint32_t x)
{
    x ^= 0x80808080u;   // 0 .. 255: as a mantissa under 1024's exponent, minus 1024 + 128
    uint2 r;
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r.x) : "r"(__byte_perm(x, 0x64646464u, 0x4140)), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(r.y) : "r"(__byte_perm(x, 0x64646464u, 0x4342)), "r"(0x64806480u));
    return r;
}

// grid (C x row tiles, KV head), clusters of C CTAs along x; one CTA per SM.
// G: query heads per KV head where that divides 32 and is at most 8, else 0 (any).
template <int D, int G>
__global__ void __launch_bounds__(kStThreads, 1) select_tile_kernel(const SelectTileParams tp)
{
    using C = StCfg<D>;
    const SelectParams &p = tp.s;
    extern __shared__ uint8_t st_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(st_raw) + 1023) & ~uintptr_t(1023));
    Candidates *cand = reinterpret_cast<Candidates *>(smem + C::KEYS);                     // [kStPick]
    int32_t *phys_s = reinterpret_cast<int32_t *>(smem + C::KEYS + kStPick * sizeof(Candidates));   // [tile of this CTA][128]
    float *unit_s = reinterpret_cast<float *>(phys_s + tp.tiles * kStTile);                // [tile of this CTA][128]
    uint32_t *keys = reinterpret_cast<uint32_t *>(unit_s + tp.tiles * kStTile);            // [row][tile of this CTA][128]
    __shared__ int32_t row_seq[kStRows], row_nb[kStRows];            // sequence (-1: no work), blocks of the row
    __shared__ uint64_t bar;
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
    const int cs = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const int64_t r0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(cs)) * tp.RT;
    const int cols = (tp.RT * p.g + 15) & ~15;
    const int stride = tp.tiles * kStTile;   // keys of a row
    if (warp == 0) {
        tmem_alloc(smem_u32(&tmem_base), 2 * kStCols);
        tmem_relinquish();
    }
    if (tid == 0) {
        mbar_init(smem_u32(&bar), 1);
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid < tp.RT) {
        const int64_t r = r0 + tid;
        int seq = -1, nb = 0;
        if (r < tp.rows) {
            seq = __ldg(p.seqs + r);
            const int pos = __ldg(p.positions + r);
            if (seq == -1 || pos == -1) {
                seq = -1;
            } else if (seq < 0 || seq >= p.B || pos < 0 || pos / p.bs >= p.max_blocks) {
                if (rank == 0 && h == 0) atomicOr(p.err, KVC_EBIT_RANGE);
                seq = -2;   // lists nothing
            } else {
                nb = pos / p.bs + 1;
            }
        }
        row_seq[tid] = seq;
        row_nb[tid] = nb;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    const uint32_t a_base = smem_u32(smem), b_base = a_base + C::A;

    // the first run's table entries, ahead of their use
    int early = -1;
    {
        const int s = lane < tp.RT ? row_seq[lane] : -1;
        const uint32_t live = __ballot_sync(kFull, s >= 0);
        const int j = (rank + (tid / kStTile) * cs) * kStTile + tid % kStTile;
        if (live) {
            const int64_t at = static_cast<int64_t>(__shfl_sync(kFull, s, __ffs(live) - 1)) * p.max_blocks;
            if (j < p.max_blocks) early = __ldg(p.bt + at + j);
        }
    }

    // ---- the rows' queries as whole numbers, positive parts then negative ones: a warp per row
    constexpr int KEEP = 2;   // chunks of a lane that stay in registers between the two passes
    const int chunks = p.g * (D / 8);
    auto source = [&](int r) {
        return reinterpret_cast<const uint4 *>(p.q + ((r0 + r) * p.H_Q + static_cast<int64_t>(h) * p.g) * D);
    };
    auto fetch = [&](int r, uint4 (&x)[KEEP]) {
#pragma unroll
        for (int u = 0; u < KEEP; ++u) {
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (r < tp.RT && row_seq[r] >= 0 && lane + 32 * u < chunks) x[u] = __ldg(source(r) + lane + 32 * u);
        }
    };
    uint4 next[KEEP];
    fetch(warp, next);
    for (int r = warp; r < tp.RT; r += kStWarps) {
        uint4 kept[KEEP];
#pragma unroll
        for (int u = 0; u < KEEP; ++u) kept[u] = next[u];
        fetch(r + kStWarps, next);
        if (row_seq[r] == -2) {
            int32_t *list = p.lists + ((r0 + r) * p.H_KV + h) * p.top_k;
            for (int i = rank * 32 + lane; i < p.top_k; i += 32 * cs) list[i] = -1;
        }
        if (row_seq[r] < 0) continue;
        float m = 0.f;
        auto largest = [&](const uint4 &x) {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) m = fmaxf(m, fmaxf(fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k]))));   // NaNs drop out
        };
#pragma unroll
        for (int u = 0; u < KEEP; ++u) largest(kept[u]);
        for (int i = lane + 32 * KEEP; i < chunks; i += 32) largest(__ldg(source(r) + i));
        const float inv = exp2_int(-unit_exponent(__uint_as_float(__reduce_max_sync(kFull, __float_as_uint(m)))));
        auto place = [&](int i, const uint4 &x) {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            uint32_t pos[4], neg[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float z[2] = {bf16_lo(w[k]), bf16_hi(w[k])};
#pragma unroll
                for (int u = 0; u < 2; ++u) z[u] = isnan(z[u]) ? 0.f : fminf(fmaxf(rintf(z[u] * inv), -127.f), 127.f);
                pos[k] = pack_f16(fmaxf(z[0], 0.f), fmaxf(z[1], 0.f));
                neg[k] = pack_f16(fminf(z[0], 0.f), fminf(z[1], 0.f));
            }
            const int n = r * p.g + i / (D / 8), ch = i % (D / 8);
            const uint32_t at = b_base + (ch >> 3) * C::BAND + sw128(n, ch & 7);
            sts128(at, make_uint4(pos[0], pos[1], pos[2], pos[3]));
            sts128(at + (D / 64) * C::BAND, make_uint4(neg[0], neg[1], neg[2], neg[3]));
        };
#pragma unroll
        for (int u = 0; u < KEEP; ++u)
            if (lane + 32 * u < chunks) place(lane + 32 * u, kept[u]);
        for (int i = lane + 32 * KEEP; i < chunks; i += 32) place(i, __ldg(source(r) + i));
    }
    __syncthreads();

    const uint32_t idesc = tc_idesc_f16(128, cols, false, false, false);
    const uint64_t desc_a = tc_smem_desc(a_base, 16, 1024, kSwizzle128B), desc_b = tc_smem_desc(b_base, 16, 1024, kSwizzle128B);
    const int chunk = tid % C::CPR, rec0 = tid / C::CPR;
    uint32_t phase = 0u;
    bool begun = false;

    const int lane_seq = lane < tp.RT ? row_seq[lane] : -3, lane_nb = lane < tp.RT ? row_nb[lane] : 0;   // RT <= 32
    for (int first = 0; first < tp.RT;) {   // runs of rows of one sequence
        const int seq = __shfl_sync(kFull, lane_seq, first);
        const uint32_t others = __ballot_sync(kFull, lane_seq != seq) & (0xFFFFFFFFu << first);
        const int end = others ? __ffs(others) - 1 : 32;
        if (seq < 0) {
            first = end;
            continue;
        }
        const bool mine_row = lane >= first && lane < end;
        const int most = __reduce_max_sync(kFull, mine_row ? lane_nb : 0), least = __reduce_min_sync(kFull, mine_row ? lane_nb : 0x7FFFFFFF);
        const int32_t *bt = p.bt + static_cast<int64_t>(seq) * p.max_blocks;
        const int n_tiles = (most + kStTile - 1) / kStTile;
        const int mine = n_tiles > rank ? (n_tiles - rank + cs - 1) / cs : 0;

        // the blocks and units of this CTA's tiles
        for (int i = tid; i < mine * kStTile; i += kStThreads) {
            const int j = (rank + (i / kStTile) * cs) * kStTile + i % kStTile;
            int phys = j >= most ? -1 : (begun || i != tid ? __ldg(bt + j) : early);
            if (j < most && (phys < 0 || static_cast<int64_t>(phys) >= p.N)) {
                if (h == 0) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
                phys = -1;
            }
            phys_s[i] = phys;
            unit_s[i] = phys < 0 ? 0.f : __ldg(p.units + static_cast<int64_t>(phys) * p.H_KV + h);
        }
        begun = true;
        __syncthreads();

        // this thread's 16 bytes of U records of a tile
        uint4 raw[C::U];
        auto load = [&](int t) {
#pragma unroll
            for (int u = 0; u < C::U; ++u) {
                const int phys = phys_s[t * kStTile + u * C::STEP + rec0];
                raw[u] = make_uint4(0u, 0u, 0u, 0u);
                if (phys >= 0)
                    raw[u] = __ldg(reinterpret_cast<const uint4 *>(p.codes + (static_cast<int64_t>(phys) * p.H_KV + h) * (2 * D)) + chunk);
            }
        };
        auto widen = [&] {   // to A; the upper half of a 128-byte band's writers store their second chunk first: no conflicts
#pragma unroll
            for (int u = 0; u < C::U; ++u) {
                const uint2 x0 = s8x4_to_f16(raw[u].x), x1 = s8x4_to_f16(raw[u].y), x2 = s8x4_to_f16(raw[u].z),
                            x3 = s8x4_to_f16(raw[u].w);
                const uint4 v0 = make_uint4(x0.x, x0.y, x1.x, x1.y), v1 = make_uint4(x2.x, x2.y, x3.x, x3.y);
                const int row = u * C::STEP + rec0, band = chunk >> 2, c0 = 2 * (chunk & 3), flip = band & 1;
                const uint32_t base = a_base + band * C::BAND;
                sts128(base + sw128(row, c0 + flip), flip ? v1 : v0);
                sts128(base + sw128(row, c0 + 1 - flip), flip ? v0 : v1);
            }
        };
        auto multiply = [&](int t) {
            fence_proxy_async_smem();
            tc_fence_before();
            __syncthreads();
            if (warp == 0) {
                tc_fence_after();
                const uint32_t d = tmem + (t & 1) * kStCols;
#pragma unroll
                for (int kk = 0; kk < C::K / 16; ++kk)
                    tc_mma_f16_warp(d, tc_desc_advance(desc_a, (kk >> 2) * C::BAND + (kk & 3) * 32),
                                    tc_desc_advance(desc_b, (kk >> 2) * C::BAND + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
                tc_commit_warp(smem_u32(&bar));
            }
        };
        if (mine > 0) {
            load(0);
            widen();
            multiply(0);
        }
        for (int t = 0; t < mine; ++t) {
            if (t + 1 < mine) load(t + 1);
            if (!mbar_wait_bounded(smem_u32(&bar), phase) && lane == 0) atomicOr(p.err, KVC_EBIT_TIMEOUT);
            phase ^= 1u;
            tc_fence_after();
            if (t + 1 < mine) {
                widen();
                multiply(t + 1);
            }
            // a lane holds a block; warps w, w + 4, ... of its quarter take a part of the run's rows each
            const int place = t * kStTile + 32 * (warp & 3) + lane, j = (rank + t * cs) * kStTile + 32 * (warp & 3) + lane;
            const int phys = phys_s[place];
            const float unit = unit_s[place];
            // tiles between the forced blocks of every row look at no row's length
            const bool plain = (rank + t * cs) * kStTile >= p.sink && (rank + t * cs + 1) * kStTile <= least - p.recent;
            auto keep = [&](int r, float best) {
                uint32_t key = score_key(best * unit);
                if (!plain) {
                    const int nb = row_nb[r];
                    if (j < p.sink || j >= nb - p.recent) key = 0xFFFFFFFFu;
                    if (j >= nb) key = 0u;
                }
                keys[r * stride + place] = phys < 0 ? 0u : key;
            };
            const uint32_t d = tmem + (t & 1) * kStCols + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
            if constexpr (G > 0) {   // 32 columns are whole rows
                constexpr int RPC = 32 / G;
                for (int r = (first / RPC + (warp >> 2)) * RPC; r < end; r += (kStWarps / 4) * RPC) {
                    uint32_t v[32];
                    tmem_ld32(d + r * G, v);
                    tmem_ld_wait(v);
#pragma unroll
                    for (int x = 0; x < RPC; ++x) {
                        float best = __uint_as_float(v[x * G]);
#pragma unroll
                        for (int y = 1; y < G; ++y) best = fmaxf(best, __uint_as_float(v[x * G + y]));
                        if (r + x >= first && r + x < end) keep(r + x, best);
                    }
                }
            } else {
                const int part = (end - first + kStWarps / 4 - 1) / (kStWarps / 4);
                const int ra = min(end, first + (warp >> 2) * part), rb = min(end, ra + part);
                float best = -INFINITY;
                int r = ra, left = p.g;
                for (int c0 = (ra * p.g) & ~31; c0 < rb * p.g; c0 += 32) {
                    uint32_t v[32];
                    tmem_ld32(d + c0, v);
                    tmem_ld_wait(v);
#pragma unroll
                    for (int x = 0; x < 32; ++x) {
                        if (c0 + x < ra * p.g || r >= rb) continue;   // warp-uniform
                        best = fmaxf(best, __uint_as_float(v[x]));
                        if (--left == 0) {
                            keep(r, best);
                            best = -INFINITY;
                            left = p.g;
                            ++r;
                        }
                    }
                }
            }
            tc_fence_before();
        }
        if (cs > 1) cluster_sync();
        else __syncthreads();

        // ---- a warp per row: gather its keys into A's place, choose, write
        const int n4 = n_tiles * kStTile;
        const int lanes_of = min(kStPick, C::A / 4 / n4);   // rows at a time
        if (warp < lanes_of) {
            uint32_t *mine_k = reinterpret_cast<uint32_t *>(smem) + warp * n4;
            for (int r = first + rank + cs * warp; r < end; r += cs * lanes_of) {
                constexpr int UG = 8;
                for (int i0 = lane; i0 < n4 / 4; i0 += 32 * UG) {
                    float4 v[UG];
#pragma unroll
                    for (int u = 0; u < UG; ++u) {
                        const int i = min(i0 + 32 * u, n4 / 4 - 1), t = i / (kStTile / 4);
                        const uint32_t a = smem_u32(keys + r * stride + (t / cs) * kStTile + 4 * (i % (kStTile / 4)));
                        v[u] = cluster_ld4(cluster_addr(a, t % cs));
                    }
#pragma unroll
                    for (int u = 0; u < UG; ++u)
                        if (i0 + 32 * u < n4 / 4) reinterpret_cast<float4 *>(mine_k)[i0 + 32 * u] = v[u];
                }
                __syncwarp();
                pick_row(mine_k, n4, cand[warp], p.lists + ((r0 + r) * p.H_KV + h) * p.top_k, p.top_k, lane);
                __syncwarp();
            }
        }
        if (cs > 1) cluster_sync();   // the others have read this CTA's keys
        else __syncthreads();
        first = end;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kStCols);
    }
}

// Largest shared memory that the kernel is launched with, beside its static variables.
constexpr int kStRoom = 226 * 1024;

template <int D, int G>
static kvc_status launch_tile_kernel(const SelectTileParams &tp, dim3 grid, size_t smem, int c, cudaStream_t stream)
{
    struct Tag {};
    const DecodeKernel k = configured<Tag>(reinterpret_cast<const void *>(&select_tile_kernel<D, G>), kStRoom, kStThreads, false);
    if (k.ctas_per_sm <= 0) return KVC_ERR_CUDA;
    return launch(&select_tile_kernel<D, G>, grid, kStThreads, smem, c, stream, tp);
}

template <int D>
static kvc_status launch_tiles(SelectTileParams &tp, int sms, cudaStream_t stream)
{
    using C = StCfg<D>;
    const SelectParams &p = tp.s;
    constexpr int kFixed = 1024 + C::KEYS + kStPick * static_cast<int>(sizeof(Candidates));
    constexpr int kTiles = (kStRoom - kFixed) / (4 * kStTile);      // runs of 128 words that there is room for
    const int blocks = (p.max_blocks + kStTile - 1) / kStTile;      // tiles of the widest row
    tp.RT = std::min(kStRows, kStCols / p.g);
    int c = 1;
    auto room = [&] { return (blocks + c - 1) / c * (tp.RT + 2) <= kTiles; };   // keys, blocks and units
    while (c < 8 && !room()) c *= 2;
    while (tp.RT > 4 && !room()) tp.RT /= 2;
    if (!room() || blocks * kStTile > C::A / 4 || blocks * kStTile > kPickMost) return KVC_ERR_UNSUPPORTED;
    const int64_t row_tiles = (tp.rows + tp.RT - 1) / tp.RT;
    while (c < 8 && c < blocks && row_tiles * p.H_KV * c < sms) c *= 2;
    tp.tiles = (blocks + c - 1) / c;
    if (row_tiles * c > 0x7FFFFFFF) return KVC_ERR_UNSUPPORTED;
    // At least 80 KB: no more than two CTAs to an SM, whose tensor memory holds two allocations.  (A CTA that waited for
    // tensor memory while its cluster waits for it could wait for a CTA of another cluster that does the same.)
    const size_t smem = std::max<size_t>(80 * 1024, kFixed + static_cast<size_t>(4) * kStTile * tp.tiles * (tp.RT + 2));
    const dim3 grid(static_cast<unsigned>(row_tiles * c), p.H_KV);
    switch (p.g) {
    case 1: return launch_tile_kernel<D, 1>(tp, grid, smem, c, stream);
    case 2: return launch_tile_kernel<D, 2>(tp, grid, smem, c, stream);
    case 4: return launch_tile_kernel<D, 4>(tp, grid, smem, c, stream);
    case 8: return launch_tile_kernel<D, 8>(tp, grid, smem, c, stream);
    }
    return launch_tile_kernel<D, 0>(tp, grid, smem, c, stream);
}

kvc_status select_tiles(const SelectParams &p, int D, int64_t rows, int sms, cudaStream_t stream)
{
    SelectTileParams tp{};
    tp.s = p;
    tp.rows = rows;
    return D == 64 ? launch_tiles<64>(tp, sms, stream) : launch_tiles<128>(tp, sms, stream);
}

}  // namespace kvc
