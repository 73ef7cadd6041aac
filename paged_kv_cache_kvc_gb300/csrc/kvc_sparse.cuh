// Sparse attention: per query row and KV head, attention over a list of blocks.
//
// Mathematics, for a row at position p, a KV head h and each of its g query heads:
//   softmax over t in { j bs + i : j listed, i < bs, t <= p } of scale <q, k_t>, times v_t.
// A listed block is bs / 16 tiles of 16 positions; each tile is one step of the online softmax of kvc_mod.cuh
// (scores of the tile on tensor cores with the positions as rows, running maximum and sum in registers, weights
// into the value product).
//
// Decomposition: a cluster of C CTAs (1, 2, 4 or 8) per (row, KV head), W = 4 or 2 warps each; warp w of CTA c takes
// tiles c + C (w + W i), T of them at a time (32 positions, for up to 16 query heads), through a ring of TMA stages of its
// own.  A step's instructions wait on one another (products, maximum, exponentials, products), so what counts is how
// much a step does: two tiles to a step share the maximum over lanes, the rescaling and the loop.  The warps of a CTA
// merge in shared memory and the CTAs through distributed shared memory: no partial goes to global memory, so a call
// needs no workspace and one launch, and two calls share nothing.
//
// Measured, 8 KV heads of 4 query heads of 128: one row of 64 blocks (bf16) 5.3 us back to back, a chain of list, table,
// tile and merge; 64 ragged rows of up to 128 e4m3 blocks (160 MB) 35 us, 4.6 TB/s, with the longest first (38 in their own
// order); 512 rows of 64 blocks (2.15 GB out of L2) 128 us, 17 TB/s, with 12 warps an SM.  One tile to a step takes 33 and
// 143 us: a chunk gains more by two than the decoding batch loses.  The CTAs' sums read one by one took 3 us more for the
// single row.
#pragma once
#include "kvc_cluster.cuh"
#include "kvc_mod.cuh"
#include "kvc_order.cuh"

namespace kvc {

struct SparseParams {
    ModParams m;               // d.q, d.bt, d.bt_stride, d.max_blocks, d.B (sequences), heads, layer, N, scales, lse, out
    const int32_t *seqs;       // [rows] or nullptr: row r is sequence r
    const int32_t *positions;  // [rows]
    const int32_t *lists;      // [rows][H_KV][top_k]
    int32_t top_k;
    int32_t sub;               // tiles per block: bs / 16
    bool longest_first;        // rows are taken in the order of what they read
};

constexpr int kSparseMost = 8;   // CTAs of a cluster

// W: warps of a CTA
template <int D, int NT, int KIND, int W>
struct SparseCfg {
    using C = DecodeCfg<D, KIND>;
    static constexpr int T = NT == 4 ? 1 : 2;          // tiles per step (more columns leave no registers for two)
    // tiles in flight per warp: the next step's, on their way while other warps compute.  More cost shared memory, and with
    // it warps or cache, or places that change from step to step: 64 e4m3 rows of 128 blocks 48.0 us with two, 49.4 with
    // three, 61.6 with four; int4 50.3 with two, 49.1 with four, 51.9 with six, ragged 38.6, 37.9 and 39.1.  With 9 to 16
    // heads per KV head registers leave room for four (64 ragged e4m3 rows 41.2 us with three, 39.4; int4 would gain too:
    // even rows 80.9 with two, 73.9 with four, ragged 48.2 and 46.0).
    static constexpr int R = KIND == KV_E4M3 && NT > 1 ? 4 : 2;
    static constexpr int RING = W * R * C::STAGE;
    static constexpr int QW = NT * 8;
    // The warps' partials, in the ring's place.  A column has a row of COL floats, so long that the lanes of one store
    // spread over all banks: four lanes hold columns of neighbouring places and eight hold channels, one each in a row of
    // eight (bf16) or four each at 16 apart (the others).
    static constexpr int COL = D + (KIND == KV_BF16 ? 8 : 4);
    static constexpr int MERGE = (W * QW * 2 + W * QW * COL) * 4;
    static constexpr int BARS = RING > MERGE ? RING : MERGE;                // offset of the barriers
    // Warps that an SM keeps, for the compiler: a register more may cost a whole CTA.  With bounds and without, 512 rows of
    // one sequence: bf16 128 us and 131, with 16 heads per KV head 185 and 221, e4m3 105 and 116; with 64 channels, as many
    // warps as for 128 would do (16 and not 24), 79 us instead of 72.
    static constexpr int CTAS = (D == 64 ? (NT == 1 ? 24 : (NT == 2 ? 16 : 12)) : (NT == 1 ? 16 : (NT == 2 ? 12 : 8))) / W;
    static constexpr int SMEM = 1024 /* alignment */ + BARS + W * R * 8;
};

// One step of a warp's running softmax: T tiles of 16 positions at st[t], of which the first valid[t] are read (all of
// them when full).  Operand layouts as in kvc_decode.cuh.  Value rows that are not read hold finite numbers.
template <int D, int NT, int KIND, bool PSPLIT, int T>
__device__ __forceinline__ void tiles_update(float scale_log2, const uint32_t (&st)[T], const uint32_t (&qf)[NT][D / 16][2],
                                             float (&m_run)[NT][2], float (&l_run)[NT][2], float (&oacc)[D / 16][NT][4],
                                             bool full, const int (&valid)[T], int lane)
{
    using C = DecodeCfg<D, KIND>;
    constexpr bool INT4 = KIND == KV_INT4, QUANT = KIND != KV_BF16;
    constexpr int NACC = NT == 1 ? 2 : 1;   // with one column tile, even and odd k-steps accumulate apart
    const int gq = lane >> 2, tg = lane & 3;
    float sc[T][NT][4], sc2[T][NT][4];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int jn = 0; jn < NT; ++jn)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[t][jn][c] = sc2[t][jn][c] = 0.f;
    auto acc = [&](int t, int jn, int kk) -> float(&)[4] { return (NACC == 2 && (kk & 1)) ? sc2[t][jn] : sc[t][jn]; };
    // ---- S^T = K Q^T
    if constexpr (!QUANT) {
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS; ++kk)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                uint32_t a[4];
                ldsm_x4(a, st[t] + swz((lane & 7) + ((lane >> 3) & 1) * 8, 2 * kk + (lane >> 4)));
#pragma unroll
                for (int jn = 0; jn < NT; ++jn) mma_bf16(acc(t, jn, kk), a, qf[jn][kk]);
            }
    } else if constexpr (INT4) {
        uint4 kw[T][2];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) kw[t][r] = lds128(st[t] + swz64(gq + 8 * r, tg));
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS; ++kk)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const uint32_t k0[4] = {kw[t][0].x, kw[t][0].y, kw[t][0].z, kw[t][0].w};
                const uint32_t k1[4] = {kw[t][1].x, kw[t][1].y, kw[t][1].z, kw[t][1].w};
                const int sh = 8 * (kk & 1);
                const uint32_t w0 = k0[kk >> 1] >> sh, w1 = k1[kk >> 1] >> sh;
                const uint32_t a[4] = {nibbles_to_f16x2(w0), nibbles_to_f16x2(w1), nibbles_hi_to_f16x2(w0), nibbles_hi_to_f16x2(w1)};
#pragma unroll
                for (int jn = 0; jn < NT; ++jn) mma_f16(acc(t, jn, kk), a, qf[jn][kk]);
            }
    } else {
        uint32_t kw[T][2][D / 16];
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int u = 0; u < D / 64; ++u) {
                    const uint4 v = lds128(st[t] + swz(gq + 8 * r, (D / 64) * tg + u));
                    kw[t][r][4 * u + 0] = v.x;
                    kw[t][r][4 * u + 1] = v.y;
                    kw[t][r][4 * u + 2] = v.z;
                    kw[t][r][4 * u + 3] = v.w;
                }
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS; ++kk)
#pragma unroll
            for (int t = 0; t < T; ++t) {
                uint32_t a[4];
                e4m3x4_to_f16x2x2(kw[t][0][kk], a[0], a[2]);
                e4m3x4_to_f16x2x2(kw[t][1][kk], a[1], a[3]);
#pragma unroll
                for (int jn = 0; jn < NT; ++jn) mma_f16(acc(t, jn, kk), a, qf[jn][kk]);
            }
    }

    // ---- scale, mask, and the online softmax (log2 units; reference maxima move only past the slack)
    uint32_t pb[T][NT][2], pl[T][NT][2];
    float alpha[NT][2];
    bool moved = false;
#pragma unroll
    for (int jn = 0; jn < NT; ++jn) {
#pragma unroll
        for (int t = 0; t < T; ++t)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float x = sc[t][jn][c];
                if constexpr (NACC == 2) x += sc2[t][jn][c];
                x *= scale_log2;
                sc[t][jn][c] = full || gq + 8 * (c >> 1) < valid[t] ? x : -INFINITY;
            }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float bm = fmaxf(sc[0][jn][c], sc[0][jn][c + 2]);
#pragma unroll
            for (int t = 1; t < T; ++t) bm = fmaxf(bm, fmaxf(sc[t][jn][c], sc[t][jn][c + 2]));
            bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 4));
            bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 8));
            bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 16));
            const bool up = bm > m_run[jn][c] + kRescaleSlack;   // false while nothing has been read
            alpha[jn][c] = up ? fast_exp2(m_run[jn][c] - bm) : 1.f;
            m_run[jn][c] = up ? bm : m_run[jn][c];
            moved |= up;
            const float mref = m_run[jn][c] == -INFINITY ? 0.f : m_run[jn][c];
            float sum = 0.f;
#pragma unroll
            for (int t = 0; t < T; ++t) {
                const float p0 = fast_exp2(sc[t][jn][c] - mref), p1 = fast_exp2(sc[t][jn][c + 2] - mref);
                sum += p0 + p1;
                sc[t][jn][c] = p0;
                sc[t][jn][c + 2] = p1;
            }
            l_run[jn][c] = fmaf(l_run[jn][c], alpha[jn][c], sum);
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {   // weights as operands: bf16 (as a pair: 16 bits), or f16 beside widened codes
            if constexpr (!QUANT) {
                const uint32_t h0 = pack_bf16(sc[t][jn][0], sc[t][jn][1]), h1 = pack_bf16(sc[t][jn][2], sc[t][jn][3]);
                pb[t][jn][0] = movmatrix_trans(h0);
                pb[t][jn][1] = movmatrix_trans(h1);
                if constexpr (PSPLIT) {
                    pl[t][jn][0] = movmatrix_trans(pack_bf16(sc[t][jn][0] - bf16_lo(h0), sc[t][jn][1] - bf16_hi(h0)));
                    pl[t][jn][1] = movmatrix_trans(pack_bf16(sc[t][jn][2] - bf16_lo(h1), sc[t][jn][3] - bf16_hi(h1)));
                }
            } else {
                pb[t][jn][0] = movmatrix_trans(pack_f16(sc[t][jn][0], sc[t][jn][1]));
                pb[t][jn][1] = movmatrix_trans(pack_f16(sc[t][jn][2], sc[t][jn][3]));
            }
        }
    }
    if (__any_sync(kFull, moved)) {
#pragma unroll
        for (int jn = 0; jn < NT; ++jn)
#pragma unroll
            for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    oacc[mt][jn][c] *= alpha[jn][c];
                    oacc[mt][jn][c + 2] *= alpha[jn][c];
                }
    }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const uint32_t sv = st[t];
        if constexpr (!QUANT) {
#pragma unroll
            for (int mt = 0; mt < C::MT; ++mt) {
                uint32_t a[4];
                ldsm_x4_trans(a, sv + swz(kBS + (lane & 7) + ((lane >> 4) & 1) * 8, 2 * mt + ((lane >> 3) & 1)));
#pragma unroll
                for (int jn = 0; jn < NT; ++jn) {
                    mma_bf16(oacc[mt][jn], a, pb[t][jn]);
                    if constexpr (PSPLIT) mma_bf16(oacc[mt][jn], a, pl[t][jn]);
                }
            }
        } else if constexpr (INT4) {
            const uint32_t par = static_cast<uint32_t>(tg & 1);
            uint32_t vw[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = kBS + 2 * tg + ((r & 1) ^ static_cast<int>(par)) + (r >> 1) * 8;
                const uint32_t a = sv + swz64(row, gq >> 1) + 8 * (gq & 1);
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(vw[r][0]), "=r"(vw[r][1]) : "r"(a));
            }
            const uint32_t sel0 = par ? 0x0044u : 0x4400u;
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t sel = sel0 + 0x1111u * static_cast<uint32_t>(k);
                    const uint32_t x01 = __byte_perm(vw[0][w], vw[1][w], sel);
                    const uint32_t x89 = __byte_perm(vw[2][w], vw[3][w], sel);
                    const uint32_t a[4] = {nibbles_to_f16x2(x01), nibbles_hi_to_f16x2(x01), nibbles_to_f16x2(x89), nibbles_hi_to_f16x2(x89)};
#pragma unroll
                    for (int jn = 0; jn < NT; ++jn) mma_f16(oacc[4 * w + k][jn], a, pb[t][jn]);
                }
        } else {
            uint32_t vw[4][D / 32];
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int u = 0; u < D / 128; ++u) {
                    const uint4 v = lds128(sv + swz(kBS + 2 * tg + (r & 1) + (r >> 1) * 8, (D / 128) * gq + u));
                    vw[r][4 * u + 0] = v.x;
                    vw[r][4 * u + 1] = v.y;
                    vw[r][4 * u + 2] = v.z;
                    vw[r][4 * u + 3] = v.w;
                }
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint32_t x01 = __byte_perm(vw[0][w], vw[1][w], 0x5140);
                const uint32_t y01 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
                const uint32_t x89 = __byte_perm(vw[2][w], vw[3][w], 0x5140);
                const uint32_t y89 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
                uint32_t a0[4], a1[4];
                e4m3x4_to_f16x2x2(x01, a0[0], a0[1]);
                e4m3x4_to_f16x2x2(x89, a0[2], a0[3]);
                e4m3x4_to_f16x2x2(y01, a1[0], a1[1]);
                e4m3x4_to_f16x2x2(y89, a1[2], a1[3]);
#pragma unroll
                for (int jn = 0; jn < NT; ++jn) {
                    mma_f16(oacc[2 * w][jn], a0, pb[t][jn]);
                    mma_f16(oacc[2 * w + 1][jn], a1, pb[t][jn]);
                }
            }
        }
    }
}

// grid (C x rows, KV head), clusters of C CTAs along x
template <int D, int NT, int KIND, bool PSPLIT, int W>
__global__ void __launch_bounds__(32 * W, SparseCfg<D, NT, KIND, W>::CTAS) sparse_kernel(const __grid_constant__ CUtensorMap tmap, const SparseParams sp)
{
    using S = SparseCfg<D, NT, KIND, W>;
    using C = DecodeCfg<D, KIND>;
    constexpr bool INT4 = KIND == KV_INT4, QUANT = KIND != KV_BF16;
    constexpr int QW = S::QW, T = S::T, R = S::R;
    const ModParams &mp = sp.m;
    const DecodeParams &p = mp.d;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ float2 part[QW];   // this CTA's (maximum, sum) of every column
    const int cs = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(cs)), h = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tg = lane & 3;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + S::BARS) + warp * R;   // this warp's
    if (lane == 0) {
        for (int i = 0; i < R; ++i) mbar_init(smem_u32(&bars[i]), 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) prefetch_tensormap(&tmap);
    grid_dependency_wait();
    if (sp.longest_first) {
        const int unit = (blockIdx.y * gridDim.x + blockIdx.x) / cs;
        h = unit % gridDim.y;
        row = row_of_rank<32 * W>(sp.positions, gridDim.x / cs, sp.sub * kBS, sp.top_k, unit / gridDim.y);
    }
    const size_t orow = static_cast<size_t>(row) * p.H_Q + static_cast<size_t>(h) * p.g;   // of the group's first head

    // What is known from the row alone is on its way before the first answer: sequence, position, this lane's list
    // entries and the queries.
    const int seq = sp.seqs ? __ldg(sp.seqs + row) : row;
    const int pos = __ldg(sp.positions + row);
    const int32_t *list = sp.lists + (static_cast<size_t>(row) * p.H_KV + h) * sp.top_k;
    const int first = rank + cs * warp, step = cs * W, listed = sp.top_k * sp.sub;   // this warp's tiles
    auto load_entry = [&](int jj) {
        const int t = first + step * jj;
        return t < listed ? __ldg(list + t / sp.sub) : -1;
    };
    const int e_cur = load_entry(lane), e_next = load_entry(32 + lane);

    // ---- query fragments, see kvc_decode.cuh.  Quantised pools: codes are exact in f16, so the queries are f16 too, with the
    // key scales in them: of the output's norm that rounding is 3.4e-4 (e4m3) and 3.8e-4 (int4), the f16 weights' 1.2e-4, the
    // output's own to bf16 1.7e-3 (2048 positions).
    uint32_t qf[NT][C::KSTEPS][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int qi = 8 * j + gq;
        const bool real = qi < p.g;
        const uint16_t *qrow = p.q + (orow + (real ? qi : 0)) * D;
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS; ++kk) {
            if constexpr (!QUANT) {
                qf[j][kk][0] = real ? *reinterpret_cast<const uint32_t *>(qrow + 16 * kk + 2 * tg) : 0u;
                qf[j][kk][1] = real ? *reinterpret_cast<const uint32_t *>(qrow + 16 * kk + 8 + 2 * tg) : 0u;
            } else if constexpr (INT4) {
                const int base = 32 * tg + 8 * (kk >> 1) + 2 * (kk & 1);
                const float *sk = p.s_k + static_cast<size_t>(h) * D;
                auto qv = [&](int c) {
                    const uint16_t raw = real ? qrow[c] : uint16_t(0);
                    return __uint_as_float(static_cast<uint32_t>(raw) << 16) * __ldg(sk + c);
                };
                qf[j][kk][0] = pack_f16(qv(base), qv(base + 4));
                qf[j][kk][1] = pack_f16(qv(base + 1), qv(base + 5));
            } else {
                const int c0 = (D / 4) * tg + 4 * kk;
                const uint2 raw = real ? *reinterpret_cast<const uint2 *>(qrow + c0) : make_uint2(0u, 0u);
                const float *sk = p.s_k + static_cast<size_t>(h) * D + c0;
                qf[j][kk][0] = pack_f16(bf16_lo(raw.x) * __ldg(sk + 0), bf16_hi(raw.x) * __ldg(sk + 1));
                qf[j][kk][1] = pack_f16(bf16_lo(raw.y) * __ldg(sk + 2), bf16_hi(raw.y) * __ldg(sk + 3));
            }
        }
    }

    if (seq == -1 || pos == -1) return;   // padding: the whole cluster leaves
    int len = pos + 1;                    // positions that the row may read
    if (seq < 0 || seq >= p.B || pos < 0 || static_cast<int64_t>(pos) >= static_cast<int64_t>(p.max_blocks) * sp.sub * kBS) {
        if (rank == 0 && threadIdx.x == 0) atomicOr(p.err, KVC_EBIT_RANGE);
        len = 0;
    }
    __syncwarp();   // the barriers are this warp's own

    const int tiles = len > 0 ? listed : 0;
    int nmine = tiles > first ? (tiles - first + step - 1) / step : 0;
    const int32_t *bt_row = p.bt + static_cast<int64_t>(seq) * p.bt_stride;
    const uint32_t st_base = smem_u32(smem + warp * R * C::STAGE);
    const uint32_t bar_base = smem_u32(bars);
    const int own = pos / (sp.sub * kBS);

    // This warp's tiles, 32 at a time in registers: (positions to read, the keys' row of the map), 0 and -1: nothing to read.
    constexpr int rows_per_tile = C::BOX_ROWS / 2;   // map rows (int4: 128-byte lines) of 16 positions
    const int64_t first_head = static_cast<int64_t>(p.layer) * p.N * p.H_KV + h;
    auto load_tile = [&](int jj, int j) -> int2 {
        if (jj >= nmine || j == -1) return make_int2(0, -1);
        const int t = first + step * jj, part = t - t / sp.sub * sp.sub;
        if (j < 0 || j > own) {
            atomicOr(p.err, KVC_EBIT_RANGE);
            return make_int2(0, -1);
        }
        const int tok0 = (j * sp.sub + part) * kBS;
        if (tok0 >= len) return make_int2(0, -1);   // past the query in its own block
        const int phys = __ldg(bt_row + j);
        if (phys < 0 || static_cast<int64_t>(phys) >= p.N) {
            atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
            return make_int2(0, -1);
        }
        const int64_t y = (first_head + static_cast<int64_t>(phys) * p.H_KV) * (2 * rows_per_tile * sp.sub) + part * rows_per_tile;
        return make_int2(min(kBS, len - tok0), static_cast<int>(y));
    };
    int2 t_cur = load_tile(lane, e_cur), t_next = load_tile(32 + lane, e_next);
    // The map's row of tile jj, which may differ from lane to lane: the lane asked cannot know which of its two the asker wants.
    auto row_of = [&](int jj, int jbase) {
        const int from = (jj - jbase) & 31;
        const int a = __shfl_sync(kFull, t_cur.y, from), b = __shfl_sync(kFull, t_next.y, from);
        return jj - jbase < 32 ? a : b;
    };
    // A lane copies tile j, whose keys stand at y, to a stage of the ring: keys, then the values behind them, a box each per
    // 128-byte band, or one for both where they are a whole block.
    auto issue = [&](int j, int y, int stage) {
        if (j >= nmine || p.stall_loads) return;
        const uint32_t bar = bar_base + 8u * static_cast<uint32_t>(stage);
        if (y < 0) {
            mbar_arrive(bar);   // complete the phase without data; the consumer skips it
            return;
        }
        const uint32_t dst = st_base + static_cast<uint32_t>(stage * C::STAGE);
        mbar_arrive_expect_tx(bar, C::STAGE);
#pragma unroll
        for (int band = 0; band < C::BANDS; ++band) {
            tma_load_2d(dst + band * C::BOX_BYTES, &tmap, bar, band * C::BOX_X, y);
            if (sp.sub > 1)
                tma_load_2d(dst + band * C::BOX_BYTES + C::BOX_BYTES / 2, &tmap, bar, band * C::BOX_X, y + rows_per_tile * sp.sub);
        }
    };
    {
        const int y = row_of(lane, 0);
        if (lane < R) issue(lane, y, lane);
    }

    // The tiles end with the last that reads anything: lists of rows shorter than top_k end with empty entries.
    uint32_t last = 0u;
    int tail = (nmine - 1) & ~31;
    for (; tail >= 64; tail -= 32)
        if ((last = __ballot_sync(kFull, tail + lane < nmine && load_entry(tail + lane) != -1)) != 0u) break;
    if (tail == 32) {
        last = __ballot_sync(kFull, t_next.y >= 0);
        if (last == 0u) tail = 0;
    }
    if (tail == 0) last = __ballot_sync(kFull, t_cur.y >= 0);
    nmine = last ? tail + 32 - __clz(last) : 0;
    const int nsteps = (nmine + T - 1) / T;

    float m_run[NT][2], l_run[NT][2];
    float oacc[C::MT][NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        m_run[j][0] = m_run[j][1] = -INFINITY;
        l_run[j][0] = l_run[j][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) oacc[mt][j][0] = oacc[mt][j][1] = oacc[mt][j][2] = oacc[mt][j][3] = 0.f;
    }

    // Tile j is stage j % R of the ring, and its use j / R.
    int i = 0, stage = 0;
    uint32_t use = 0u;
    bool timed_out = false;
    for (; i < nsteps; ++i) {
        const int j = i * T, jbase = j & ~31;
        if (j > 0 && (j & 31) == 0) {
            t_cur = t_next;
            t_next = load_tile(j + 32 + lane, load_entry(j + 32 + lane));
        }
        uint32_t st[T];
        bool ok = true;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const bool wrap = stage + t >= R;   // T <= R
            const int at = wrap ? stage + t - R : stage + t;
            st[t] = st_base + static_cast<uint32_t>(at * C::STAGE);
            if (j + t < nmine) ok &= mbar_wait_bounded(bar_base + 8u * static_cast<uint32_t>(at), (use + (wrap ? 1u : 0u)) & 1u);
        }
        if (!__all_sync(kFull, ok)) {
            timed_out = true;
            break;
        }
        int valid[T];
        bool full = true, some = false;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            valid[t] = __shfl_sync(kFull, t_cur.x, (j + t) & 31);
            full &= valid[t] == kBS;
            some |= valid[t] > 0;
        }
        if (some) {
            // value rows past the query, or of no tile, may hold anything (NaN included): zero them
            // (every int4 nibble is a finite value, and its weight there is 0)
            if (!INT4 && !full) {
#pragma unroll
                for (int t = 0; t < T; ++t) {
                    const int nz = (kBS - valid[t]) * C::BANDS * 8;
                    for (int z = lane; z < nz; z += 32)
                        sts128_zero(st[t] + swz(kBS + valid[t] + z / (C::BANDS * 8), z % (C::BANDS * 8)));
                }
            }
            __syncwarp();
            tiles_update<D, NT, KIND, PSPLIT, T>(p.scale_log2, st, qf, m_run, l_run, oacc, full, valid, lane);
        }
        __syncwarp();
        if (j + R < nmine) {   // the next ones into the places of these
            const int y = row_of(j + R + lane, jbase);
            if (lane < T) {
                fence_proxy_async_smem();
                issue(j + R + lane, y, stage + lane >= R ? stage + lane - R : stage + lane);
            }
        }
        stage += T;
        if (stage >= R) {
            stage -= R;
            ++use;
        }
    }
    if (timed_out) {   // record, then let copies already in flight land before the CTA exits
        if (lane == 0) {
            atomicOr(p.err, KVC_EBIT_TIMEOUT);
            for (int x = i * T; x < min(nmine, i * T + R); ++x)
                (void)mbar_wait_bounded(bar_base + 8u * (x % R), static_cast<uint32_t>((x / R) & 1), 100000000ull);
        }
        __syncwarp();
    }

#pragma unroll
    for (int jn = 0; jn < NT; ++jn)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float l = l_run[jn][c];
            l += __shfl_xor_sync(kFull, l, 4);
            l += __shfl_xor_sync(kFull, l, 8);
            l += __shfl_xor_sync(kFull, l, 16);
            l_run[jn][c] = l;
        }

    // ---- the warps' partials to shared memory (the ring is free), then one sum per CTA, then one per cluster
    __syncthreads();
    float *cm = reinterpret_cast<float *>(smem);
    float *cl = cm + W * QW;
    float *co = cl + W * QW;   // [warp][place of column][COL]
    constexpr int COL = S::COL;
    auto place = [](int qi) { return (qi & ~7) + 4 * (qi & 1) + ((qi & 7) >> 1); };   // even columns first: a lane has two
#pragma unroll
    for (int jn = 0; jn < NT; ++jn)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int qi = 8 * jn + 2 * tg + c;
            if (qi >= p.g) continue;
            if (gq == 0) {
                cm[warp * QW + qi] = m_run[jn][c];
                cl[warp * QW + qi] = l_run[jn][c];
            }
            float *col = co + (warp * QW + place(qi)) * COL;
            if constexpr (QUANT) {   // channels gq D/8 + 2 mt and the one behind it
#pragma unroll
                for (int mt = 0; mt < C::MT; mt += 2)
                    *reinterpret_cast<float4 *>(col + gq * (D / 8) + 2 * mt) =
                        make_float4(oacc[mt][jn][c], oacc[mt][jn][c + 2], oacc[mt + 1][jn][c], oacc[mt + 1][jn][c + 2]);
            } else {   // 16 mt + gq and the one 8 behind it
#pragma unroll
                for (int mt = 0; mt < C::MT; ++mt) {
                    col[16 * mt + gq] = oacc[mt][jn][c];
                    col[16 * mt + gq + 8] = oacc[mt][jn][c + 2];
                }
            }
        }
    __syncthreads();
    for (int i = threadIdx.x; i < p.g * (D / 2); i += 32 * W) {
        const int qi = i / (D / 2), d = 2 * (i - qi * (D / 2));
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, cm[w * QW + qi]);
        const float Mref = M == -INFINITY ? 0.f : M;
        float L = 0.f, O0 = 0.f, O1 = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float e = fast_exp2(cm[w * QW + qi] - Mref);   // warps that read nothing: exp2(-inf) = 0
            const float2 o = *reinterpret_cast<const float2 *>(co + (w * QW + place(qi)) * COL + d);
            L += e * cl[w * QW + qi];
            O0 += e * o.x;
            O1 += e * o.y;
        }
        if constexpr (QUANT) {
            const float *sv = p.s_v + static_cast<size_t>(h) * D + d;
            O0 *= __ldg(sv);
            O1 *= __ldg(sv + 1);
        }
        if (cs == 1) {
            const float inv = L == 0.f ? 0.f : 1.f / L;
            *reinterpret_cast<uint32_t *>(mp.out + (orow + qi) * D + d) = pack_bf16(O0 * inv, O1 * inv);
            if (d == 0 && p.lse) p.lse[orow + qi] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
        } else {   // in the first warp's place, which no other thread reads
            *reinterpret_cast<float2 *>(co + place(qi) * COL + d) = make_float2(O0, O1);
            if (d == 0) part[qi] = make_float2(M, L);
        }
    }
    if (cs == 1) return;

    // CTA `rank` finishes its part of the group's channels from all CTAs' sums
    cluster_sync();
    for (int i = rank * 32 * W + threadIdx.x; i < p.g * (D / 4); i += cs * 32 * W) {
        const int qi = i / (D / 4), d = 4 * (i - qi * (D / 4));
        float2 ml[kSparseMost];
        float4 o[kSparseMost];
#pragma unroll
        for (int r = 0; r < kSparseMost; ++r) {
            ml[r] = make_float2(-INFINITY, 0.f);
            o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < cs) {
                ml[r] = cluster_ld2(cluster_addr(smem_u32(part + qi), r));
                o[r] = cluster_ld4(cluster_addr(smem_u32(co + place(qi) * COL + d), r));
            }
        }
        float M = -INFINITY;
#pragma unroll
        for (int r = 0; r < kSparseMost; ++r) M = fmaxf(M, ml[r].x);
        const float Mref = M == -INFINITY ? 0.f : M;
        float L = 0.f;
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < kSparseMost; ++r) {
            const float e = fast_exp2(ml[r].x - Mref);
            L = fmaf(e, ml[r].y, L);
            sum.x = fmaf(e, o[r].x, sum.x);
            sum.y = fmaf(e, o[r].y, sum.y);
            sum.z = fmaf(e, o[r].z, sum.z);
            sum.w = fmaf(e, o[r].w, sum.w);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint2 *>(mp.out + (orow + qi) * D + d) =
            make_uint2(pack_bf16(sum.x * inv, sum.y * inv), pack_bf16(sum.z * inv, sum.w * inv));
        if (d == 0 && p.lse) p.lse[orow + qi] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
    cluster_sync();   // a CTA's shared memory stays until the others have read it
}

struct SparseKernel {
    void (*fn)(const CUtensorMap, const SparseParams);
    DecodeKernel k;
};

template <int D, int NT, int KIND, bool PSPLIT, int W>
SparseKernel sparse_instance()
{
    struct Tag {};
    return {&sparse_kernel<D, NT, KIND, PSPLIT, W>,
            configured<Tag>(reinterpret_cast<const void *>(&sparse_kernel<D, NT, KIND, PSPLIT, W>), SparseCfg<D, NT, KIND, W>::SMEM,
                            32 * W, false)};
}

SparseKernel select_sparse_bf16(int D, int g, int warps);
SparseKernel select_sparse_fp8(int g, int warps);
SparseKernel select_sparse_int4(int g, int warps);

}  // namespace kvc
