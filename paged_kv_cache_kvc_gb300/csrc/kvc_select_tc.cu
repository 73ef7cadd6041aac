// Block selection for chunks: many rows of one sequence score the same blocks, so the scores are a matrix product,
// on the fifth-generation tensor cores.
//
// Mathematics.  With the positive and the negative parts of the whole-numbered queries side by side, a score is one
// product of length 2 d:  sum_i Q_i (Q_i > 0 ? hi_i : lo_i) = <(Q+, Q-), (hi, lo)>.  Codes and queries are integers
// up to 127, exact in f16; products are below 2^14 and sums below 2^21, exact in the fp32 accumulator in any order.
//
// A CTA takes RT rows of one KV head and walks all blocks in tiles of 128, twice:
//   D[128 blocks x RT g query columns] = A[128 x 2d] B[2d x RT g].
// The blocks are the M rows, so that a thread of the epilogue holds one block's products with every query head and
// takes their maximum without a shuffle.  Keeping a score for every row and block would fill shared memory and keep
// the rest of the SM idle while rows are finished; multiplying again costs little.  So the first walk only keeps the
// largest score of 256 groups of blocks per row: the top_k-th of those is a limit that at least top_k blocks reach.
// The second walk collects the few blocks that reach it, and a warp per row ranks them by counting.
// B (the queries) stays in shared memory.  A goes through tensor memory: with both operands in shared memory the
// products alone would take all of its bandwidth (8 KB in 68 cycles), and every warp can stage, widen and store its own
// part without a barrier: 32 blocks and a quarter of the 2 d channels, by copies two tiles ahead.
//
// 512 rows of 2048 blocks, 8 KV heads of 4 query heads: 64 us (273 scored row by row; 181 and then 92 with the scores
// of all blocks kept in shared memory of a cluster, 76 with A in shared memory).  A tile costs 1.1 us in the first walk
// and 1.35 in the second: each warp's chain of copies, widening (110 instructions), barrier, products and maxima (70), with
// 16 warps to hide it in (issue slots 54 % busy); the products themselves are 0.56 (tensor pipe 20 %).  15 us are code that runs once: queries, limits, ranks.
// Reading and widening by warps of their own was slower (126 us: half the warps for each, loads of TMEM one after
// another).
//
// A tile of rows may hold several sequences (runs): they are done one after the other, each with two walks of its own.
#include <algorithm>
#include <cstdlib>

#include "kvc_select.cuh"
#include "kvc_tc.cuh"

namespace kvc {

constexpr int kStThreads = 512;   // the threads that widen and read; one warp more issues the products
constexpr int kStWarps = kStThreads / 32;
constexpr int kStCta = kStThreads + 32;
constexpr int kStTile = 128;       // blocks per MMA
constexpr int kStCols = 128;       // query columns at most
constexpr int kStRows = 32;        // rows at most
constexpr int kStChunk = 16;       // tiles whose table entries and units are looked up at a time
constexpr int kStGroups = 256;     // per row: a lane's place in its tile, even and odd tiles apart

template <int D>
struct StCfg {
    static constexpr int K = 2 * D;
    static constexpr int BANDS = K / 64;            // 128-byte bands of f16
    static constexpr int BAND = 128 * 128;          // bytes of a band of 128 rows
    static constexpr int B = BANDS * BAND;          // bytes of the queries
    static constexpr int SEG = K / 4;               // bytes of a record that a warp widens
    static constexpr int CH = SEG / 16;             // in 16-byte chunks: 4 or 2
    static constexpr int STAGE = 32 * SEG;          // bytes of a warp's stage
    static constexpr int STAGES = 2;
    static constexpr int STAGED = B;                // offset of the stages
    static constexpr int CAND = STAGED + kStWarps * STAGES * STAGE;   // groups' maxima, then candidates
    static constexpr int ROW_CAND = kCandWords * 4;
    static constexpr int PHYS = CAND + kStRows * ROW_CAND;   // blocks of a chunk's tiles
    static constexpr int UNIT = PHYS + kStChunk * kStTile * 4;
    static constexpr int SMEM = 1024 /* alignment */ + UNIT + kStChunk * kStTile * 4;
    static constexpr int A_COLS = K / 2;            // columns of A in tensor memory
    static constexpr int A_TMEM = 2 * kStCols;      // A's two buffers, after the products' two
    static_assert(ROW_CAND >= kStGroups * 4, "the groups' maxima lie in the candidates' place");
};
constexpr int kStTmem = 512;   // columns: all of them

struct SelectTileParams {
    SelectParams s;
    int64_t rows;
    int32_t RT;            // rows per tile
    uint32_t stall_from;   // test hook: tiles of a CTA from this one on are never announced, so that the waits run out
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

// grid (row tiles, KV head); one CTA per SM.
// G: query heads per KV head where that divides 32 and is at most 8, else 0 (any).
template <int D, int G>
__global__ void __launch_bounds__(kStCta, 1) select_tile_kernel(const SelectTileParams tp)
{
    using C = StCfg<D>;
    const SelectParams &p = tp.s;
    extern __shared__ uint8_t st_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(st_raw) + 1023) & ~uintptr_t(1023));
    uint32_t *groups = reinterpret_cast<uint32_t *>(smem + C::CAND);     // [row][kStGroups]
    int32_t *phys_s = reinterpret_cast<int32_t *>(smem + C::PHYS);       // [tile of the chunk][128]
    float *unit_s = reinterpret_cast<float *>(smem + C::UNIT);
    auto cand = [&](int r) { return reinterpret_cast<uint32_t *>(smem + C::CAND + r * C::ROW_CAND); };   // keys, blocks
    __shared__ int32_t row_seq[kStRows], row_nb[kStRows];                // sequence (< 0: no work), blocks of the row
    __shared__ float row_limit[kStRows];
    __shared__ int32_t row_count[kStRows];                               // candidates
    __shared__ uint64_t full_bar[2], done_bar[2];   // a buffer of A is written; its products are there (and it is free)
    __shared__ uint32_t tmem_base;
    __shared__ int32_t expired;   // a wait ran out: written between a walk's barriers only, so all threads read the same
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, h = blockIdx.y;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * tp.RT;
    const int cols = (tp.RT * p.g + 15) & ~15;
    if (warp == 0) {
        tmem_alloc(smem_u32(&tmem_base), kStTmem);
        tmem_relinquish();
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&full_bar[i]), kStWarps);
            mbar_init(smem_u32(&done_bar[i]), 1);
        }
        expired = 0;
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
                if (h == 0) atomicOr(p.err, KVC_EBIT_RANGE);
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
    const uint32_t b_base = smem_u32(smem);

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
    if (warp < kStWarps) fetch(warp, next);
    for (int r = warp; r < tp.RT && warp < kStWarps; r += kStWarps) {
        uint4 kept[KEEP];
#pragma unroll
        for (int u = 0; u < KEEP; ++u) kept[u] = next[u];
        fetch(r + kStWarps, next);
        if (row_seq[r] == -2) {
            int32_t *list = p.lists + ((r0 + r) * p.H_KV + h) * p.top_k;
            for (int i = lane; i < p.top_k; i += 32) list[i] = -1;
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
    fence_proxy_async_smem();   // the tensor cores read the queries through the async proxy, which the barrier alone does not order
    __syncthreads();

    const uint32_t idesc = tc_idesc_f16(128, cols, false, false, false);
    const uint64_t desc_b = tc_smem_desc(b_base, 16, 1024, kSwizzle128B);
    const int quarter = warp & 3, part = (warp >> 2) & 3;   // this warp's 32 blocks of a tile, and its part of the channels
    const uint32_t stage = b_base + C::STAGED + (warp & (kStWarps - 1)) * (C::STAGES * C::STAGE);
    // where chunk c of row r stands in a stage, so that eight rows' chunks c are free of conflicts
    auto staged = [](int r, int c) { return static_cast<uint32_t>(r * C::SEG + ((c ^ ((C::CH == 4 ? r >> 1 : r >> 2) & (C::CH - 1))) << 4)); };
    const int8_t *codes = p.codes + h * (2 * D) + part * C::SEG;
    const uint32_t record_stride = static_cast<uint32_t>(p.H_KV) * (2 * D);   // H_KV is at most 256
    uint32_t tile_no = 0u;   // tiles of this CTA so far: the barriers' phases
    uint32_t issued = 0u;    // tiles whose products have begun (the last warp's)
    // A wait that runs out ends the walk for its warp, and the kernel after the next barrier: the other warps' waits run out
    // with it or one tile later.
    auto wait = [&](uint64_t &b, uint32_t parity) {
        const bool ok = __all_sync(kFull, mbar_wait_bounded(smem_u32(&b), parity & 1u));
        if (!ok && lane == 0) {
            atomicOr(p.err, KVC_EBIT_TIMEOUT);
            expired = 1;
        }
        return ok;
    };

    const int lane_seq = lane < tp.RT ? row_seq[lane] : -3, lane_nb = lane < tp.RT ? row_nb[lane] : 0;   // RT <= 32
    int first = 0;
    while (first < tp.RT) {   // runs of rows of one sequence
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
        int t0 = 0;   // the chunk's first tile

        // this warp's part of tile t to its stage: CH lanes a record
        auto copy = [&](int t) {
            const uint32_t to = stage + (t & 1) * C::STAGE;
            const int c = lane % C::CH;
#pragma unroll
            for (int i = 0; i < C::CH; ++i) {
                const int r = i * (32 / C::CH) + lane / C::CH;
                // no block: block 0's, whose scores are not used
                const uint32_t phys = static_cast<uint32_t>(max(phys_s[t * kStTile + 32 * quarter + r], 0));
                cp_async16(to + staged(r, c), codes + static_cast<uint64_t>(phys) * record_stride + 16 * c);
            }
            cp_async_commit();
        };
        // from there to A's buffer in tensor memory, widened: lane = block
        auto widen = [&](int t, uint32_t buf) {
            uint32_t w[32];
#pragma unroll
            for (int c = 0; c < C::CH; ++c) {
                const uint4 x = lds128(stage + (t & 1) * C::STAGE + staged(lane, c));
                const uint2 x0 = s8x4_to_f16(x.x), x1 = s8x4_to_f16(x.y), x2 = s8x4_to_f16(x.z), x3 = s8x4_to_f16(x.w);
                w[8 * c + 0] = x0.x, w[8 * c + 1] = x0.y, w[8 * c + 2] = x1.x, w[8 * c + 3] = x1.y;
                w[8 * c + 4] = x2.x, w[8 * c + 5] = x2.y, w[8 * c + 6] = x3.x, w[8 * c + 7] = x3.y;
            }
            const uint32_t to = tmem + C::A_TMEM + buf * C::A_COLS + part * (C::A_COLS / 4) + (static_cast<uint32_t>(32 * quarter) << 16);
            if constexpr (C::CH == 4) {
                tmem_st32(to, w);
            } else {
                uint32_t w16[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) w16[i] = w[i];
                tmem_st16(to, w16);
            }
            tmem_st_wait();
            tc_fence_before();   // and what this warp read of tensor memory it has read
            __syncwarp();
            if (lane == 0 && tile_no + t < tp.stall_from) mbar_arrive(smem_u32(&full_bar[buf]));
        };

        // One walk over the blocks.  read(t, d): the epilogue of tile t, whose products stand at d in tensor memory.
        auto walk = [&](bool report, auto read) {
            for (t0 = 0; t0 < n_tiles; t0 += kStChunk) {
                const int nt = min(kStChunk, n_tiles - t0);
                __syncthreads();   // the chunk before is done with its table entries
                if (expired) break;
                // a single chunk's are still there in the second walk
                for (int i = tid; i < nt * kStTile && (report || n_tiles > kStChunk); i += kStCta) {
                    const int j = t0 * kStTile + i;
                    int phys = j < most ? __ldg(bt + j) : -1;
                    if (j < most && (phys < 0 || static_cast<int64_t>(phys) >= p.N)) {
                        if (report && h == 0) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
                        phys = -1;
                    }
                    phys_s[i] = phys;
                    unit_s[i] = phys < 0 ? 0.f : __ldg(p.units + static_cast<int64_t>(phys) * p.H_KV + h);
                }
                __syncthreads();
                // Barrier phases: tile i of the CTA is use i / 2 of buffer i mod 2.
                if (warp == kStWarps) {
                    for (int t = 0; t < nt; ++t) {
                        const uint32_t i = tile_no + t, buf = i & 1u;
                        if (!wait(full_bar[buf], i >> 1)) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < C::K / 16; ++kk)
                            tc_mma_f16_tmem_a_warp(tmem + buf * kStCols, tmem + C::A_TMEM + buf * C::A_COLS + kk * 8,
                                                   tc_desc_advance(desc_b, (kk >> 2) * C::BAND + (kk & 3) * 32), idesc, kk > 0 ? 1u : 0u);
                        tc_commit_warp(smem_u32(&done_bar[buf]));
                        issued = i + 1u;
                    }
                } else {
                    copy(0);
                    if (nt > 1) copy(1);
                    else cp_async_commit();
                    cp_async_wait<1>();
                    __syncwarp();
                    widen(0, tile_no & 1u);
                    for (int t = 0; t < nt; ++t) {
                        const uint32_t i = tile_no + t, buf = i & 1u;
                        __syncwarp();   // stage t mod 2 has been read
                        if (t + 2 < nt) copy(t + 2);
                        else cp_async_commit();   // a group each time, so that the wait below counts
                        if (t + 1 < nt) {   // A's other buffer is free: tile t - 1's products were waited for
                            cp_async_wait<1>();
                            __syncwarp();
                            widen(t + 1, buf ^ 1u);
                        }
                        if (!wait(done_bar[buf], i >> 1)) break;
                        tc_fence_after();
                        read(t, tmem + buf * kStCols + (static_cast<uint32_t>(32 * quarter) << 16));
                    }
                }
                tile_no += nt;
            }
            tc_fence_before();
            __syncthreads();
        };

        // A lane holds a block of the tile; warps w, w + 4, ... of its quarter take a part of the rows each.  score(x, s):
        // the score of row (warp / 4) RPC + x, -inf where the block is none of the row's, +inf where it is always listed.
        constexpr int RPC = G > 1 ? 32 / G : 1;   // rows of 32 columns
        const int in_tile = 32 * (warp & 3) + lane, row0 = (warp >> 2) * RPC;
        auto scores = [&](int t, uint32_t d, auto score) {
            const int j = (t0 + t) * kStTile + in_tile;
            const float unit = unit_s[t * kStTile + in_tile], none = phys_s[t * kStTile + in_tile] < 0 ? -INFINITY : 0.f;
            // tiles between the forced blocks of every row look at no row's length
            const bool plain = (t0 + t) * kStTile >= p.sink && (t0 + t + 1) * kStTile <= least - p.recent;
            auto edge = [&](int r, float s) {
                const int nb = row_nb[r];
                return j >= nb ? -INFINITY : (none == 0.f && (j < p.sink || j >= nb - p.recent) ? INFINITY : s);
            };
            if constexpr (G > 1) {
                if (row0 >= tp.RT) return;   // warp-uniform
                uint32_t v[32];
                tmem_ld32(d + row0 * G, v);
                tmem_ld_wait(v);
#pragma unroll
                for (int x = 0; x < RPC; ++x) {
                    float best = __uint_as_float(v[x * G]);
#pragma unroll
                    for (int y = 1; y < G; ++y) best = fmaxf(best, __uint_as_float(v[x * G + y]));
                    float s = fmaf(best, unit, none);   // 0, never -0
                    if (!plain) s = edge(min(row0 + x, kStRows - 1), s);
                    score(x, s);
                }
            } else {   // any group: x is the row itself
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
                            float s = fmaf(best, unit, none);
                            if (!plain) s = edge(r, s);
                            score(r, s);
                            best = -INFINITY;
                            left = p.g;
                            ++r;
                        }
                    }
                }
            }
        };
        auto to_key = [](float s) { return s == -INFINITY ? 0u : (s == INFINITY ? 0xFFFFFFFFu : score_key(s)); };

        // ---- the largest key of every group, and of those the limit that top_k blocks reach
        if constexpr (G > 1) {
            float most_of[2][RPC];   // even and odd tiles
#pragma unroll
            for (int x = 0; x < RPC; ++x) most_of[0][x] = most_of[1][x] = -INFINITY;
            walk(true, [&](int t, uint32_t d) {
                const bool odd = (t & 1) != 0;
                scores(t, d, [&](int x, float s) {
                    if (odd) most_of[1][x] = fmaxf(most_of[1][x], s);
                    else most_of[0][x] = fmaxf(most_of[0][x], s);
                });
            });
#pragma unroll
            for (int x = 0; x < RPC; ++x)
                if (warp < kStWarps && row0 + x >= first && row0 + x < end) {
                    groups[(row0 + x) * kStGroups + in_tile] = to_key(most_of[0][x]);
                    groups[(row0 + x) * kStGroups + kStTile + in_tile] = to_key(most_of[1][x]);
                }
        } else {
            for (int i = first * kStGroups + tid; i < end * kStGroups; i += kStCta) groups[i] = 0u;
            walk(true, [&](int t, uint32_t d) {   // begins with a barrier; each place is this lane's own
                scores(t, d, [&](int r, float s) {
                    uint32_t *g = groups + r * kStGroups + (t & 1) * kStTile + in_tile;
                    *g = max(*g, to_key(s));
                });
            });
        }
        if (expired) break;
        __syncthreads();
        for (int r = first + warp; r < end && warp < kStWarps; r += kStWarps) {
            uint32_t v[kStGroups / 32];
#pragma unroll
            for (int u = 0; u < kStGroups / 32; ++u) v[u] = groups[r * kStGroups + 32 * u + lane];
            const uint32_t limit = reach_limit(v, static_cast<uint32_t>(p.top_k));
            if (lane == 0) {
                row_limit[r] = limit == 0u ? -FLT_MAX : (limit == 0xFFFFFFFFu ? INFINITY : key_score(limit));
                row_count[r] = 0;
            }
        }
        __syncthreads();

        // ---- the blocks that reach it
        auto append = [&](int r, uint32_t count, float s, float limit, int j) {   // if s reaches the limit; no branch
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t.reg .u32 at, a;\n\t"
                "setp.ge.f32 p, %0, %1;\n\tmov.u32 at, 0xffffffff;\n\t"
                "@p atom.shared.add.u32 at, [%2], 1;\n\t"
                "setp.lt.u32 q, at, %5;\n\tshl.b32 a, at, 2;\n\tadd.u32 a, a, %3;\n\t"
                "@q st.shared.f32 [a], %0;\n\t@q st.shared.u32 [a + %6], %4;\n\t}"
                ::"f"(s), "f"(limit), "r"(count), "r"(smem_u32(cand(r))), "r"(j), "n"(kCandRow), "n"(4 * kCandRow)
                : "memory");
        };
        if constexpr (G > 1) {
            float limit[RPC];
#pragma unroll
            for (int x = 0; x < RPC; ++x)   // nothing reaches a NaN: the rows of other runs
                limit[x] = row0 + x >= first && row0 + x < end ? row_limit[row0 + x] : __uint_as_float(0x7FFFFFFFu);
            const uint32_t counts = smem_u32(&row_count[row0 < kStRows ? row0 : 0]);
            walk(false, [&](int t, uint32_t d) {
                scores(t, d, [&](int x, float s) { append(row0 + x, counts + 4 * x, s, limit[x], (t0 + t) * kStTile + in_tile); });
            });
        } else {
            walk(false, [&](int t, uint32_t d) {
                scores(t, d, [&](int r, float s) { append(r, smem_u32(&row_count[r]), s, row_limit[r], (t0 + t) * kStTile + in_tile); });
            });
        }
        if (expired) break;
        for (int r = first + warp; r < end && warp < kStWarps; r += kStWarps) {   // a warp per row
            int32_t *list = p.lists + ((r0 + r) * p.H_KV + h) * p.top_k;
            const int n = row_count[r];
            for (int i = lane; i < min(n, kCandRow); i += 32) cand(r)[i] = to_key(__uint_as_float(cand(r)[i]));   // keys from here on
            __syncwarp();
            if (n <= 128) list_candidates<4>(cand(r), n, most, list, p.top_k, lane);
            else if (n <= kCandRow) list_candidates<kCandRow / 32>(cand(r), n, most, list, p.top_k, lane);
            else if (lane == 0) list[0] = kUnlisted;   // many equal keys
        }
        __syncthreads();
        first = end;
    }
    if (expired) {   // what is on its way lands; this run's rows and those behind it list nothing
        cp_async_wait<0>();
        if (issued > 0u) (void)mbar_wait_bounded(smem_u32(&done_bar[(issued - 1u) & 1u]), ((issued - 1u) >> 1) & 1u);
        for (int r = first + warp; r < tp.RT; r += kStCta / 32) {
            if (row_seq[r] < 0) continue;
            int32_t *list = p.lists + ((r0 + r) * p.H_KV + h) * p.top_k;
            for (int i = lane; i < p.top_k; i += 32) list[i] = -1;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, kStTmem);
    }
}

template <int D, int G>
static kvc_status launch_tile_kernel(const SelectTileParams &tp, cudaStream_t stream)
{
    constexpr int kSmem = StCfg<D>::SMEM;
    static_assert(2 * kSmem > 228 * 1024, "one CTA to an SM, whose tensor memory it takes whole");
    struct Tag {};
    const DecodeKernel k = configured<Tag>(reinterpret_cast<const void *>(&select_tile_kernel<D, G>), kSmem, kStCta, false);
    if (k.ctas_per_sm <= 0) return KVC_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>((tp.rows + tp.RT - 1) / tp.RT), tp.s.H_KV);
    return launch(&select_tile_kernel<D, G>, grid, kStCta, kSmem, 1, stream, tp);
}

template <int D>
static kvc_status launch_tiles(const SelectTileParams &tp, cudaStream_t stream)
{
    switch (tp.s.g) {
    case 1: return launch_tile_kernel<D, 1>(tp, stream);
    case 2: return launch_tile_kernel<D, 2>(tp, stream);
    case 4: return launch_tile_kernel<D, 4>(tp, stream);
    case 8: return launch_tile_kernel<D, 8>(tp, stream);
    }
    return launch_tile_kernel<D, 0>(tp, stream);
}

kvc_status select_tiles(const SelectParams &p, int D, int64_t rows, cudaStream_t stream)
{
    SelectTileParams tp{};
    tp.s = p;
    tp.rows = rows;
    tp.RT = std::min(kStRows, kStCols / p.g);
    const char *stall = std::getenv("KVC_TEST_STALL");   // "n": from the n-th tile of every CTA on
    tp.stall_from = stall ? static_cast<uint32_t>(std::max(std::atoi(stall), 1) - 1) : 0xFFFFFFFFu;
    return D == 64 ? launch_tiles<64>(tp, stream) : launch_tiles<128>(tp, stream);
}

}  // namespace kvc
