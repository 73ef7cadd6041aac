// Attention with modified scores over a block table: tanh-capped scores, a
// bias linear in the distance, a sliding window with leading sink positions,
// a bidirectional prefix, packed documents.
//
// Mathematics, for a query at position p of query head hq:
//   x_t = scale * <q, k_t>
//   x_t <- cap * tanh(x_t / cap)                       (cap > 0)
//   x_t <- x_t - slope[hq] * |p - t|                   (alibi)
//   read t:  t in [lo, p]  or  t in [d, e)             (both below the length)
//     d  = the query's document start (0 without documents)
//     lo = max(d, p - window + 1)                      (d without a window)
//     e  = max(min(d + sink, p + 1) with a window, prefix), d when neither
//   out = sum softmax(x)_t v_t,  lse = ln sum exp(x_t); nothing read: 0, -inf.
// Scores live in log2 units.  tanh(u) = 1 - 2 / (1 + 2^(2 u log2 e)): one
// exponential and one reciprocal, its error (about 2^-23 of cap) absolute, so
// the weights are off by no more than fp32 scores of size cap are anyway;
// the hardware's tanh approximation (2^-11) would move weights by percents.
//
// Every query of a unit (a CTA's query columns) reads a union of at most two
// runs of positions, so a unit visits blocks [b0, b0 + n0) and [b1, ...): a
// window skips the blocks between them, whose table entries are never looked
// at (a serving engine frees them).  Blocks that some column may not read in
// full mask per column; the other blocks mask nothing.
#pragma once
#include "kvc_configured.cuh"
#include "kvc_decode.cuh"

namespace kvc {

struct ModParams {
    DecodeParams d;            // as in the plain kernels; d.out is unused
    uint16_t *out;             // bf16 [n_pos][H_Q][D]
    const float *alibi;        // [H_Q] slopes or nullptr
    const int32_t *doc_start;  // [n_pos] (prefill) or nullptr
    int32_t window, sink, prefix;
    int32_t capped;
    float cap_in;              // 2 scale log2(e) / cap
    float cap_out;             // cap log2(e)
};

// The positions query position p reads: [lo, p] and [d, e); lo > p and e = d where nothing is.
struct Range {
    int32_t lo, hi, d, e;
};

__device__ __forceinline__ Range query_range(const ModParams &p, int pos, int total, int doc)
{
    Range r;
    r.d = doc > 0 ? doc : 0;
    r.hi = pos + 1;
    r.lo = p.window > 0 ? max(r.d, r.hi - p.window) : r.d;
    r.e = r.d;
    if (p.window > 0) r.e = max(r.d, static_cast<int32_t>(min(static_cast<int64_t>(r.d) + p.sink, static_cast<int64_t>(r.hi))));
    if (p.prefix > 0) r.e = max(r.e, min(p.prefix, total));
    return r;
}

// A unit's blocks: [b0, b0 + n0), then [b1, b1 + n - n0); virtual block j is the j-th of them.
struct BlockRuns {
    int32_t b0, n0, b1, n;
    __device__ __forceinline__ int at(int j) const { return j < n0 ? b0 + j : b1 + (j - n0); }
};

// Blocks covering positions [e0, e1) and [a0, a1) (either may be empty).
__device__ __forceinline__ BlockRuns block_runs(int e0, int e1, int a0, int a1)
{
    BlockRuns r;
    const bool he = e1 > e0, ha = a1 > a0;
    const int eb0 = e0 / kBS, eb1 = (e1 + kBS - 1) / kBS, ab0 = a0 / kBS, ab1 = (a1 + kBS - 1) / kBS;
    if (he && ha && (ab0 <= eb1 && eb0 <= ab1)) {   // they meet: one run
        r.b0 = min(eb0, ab0);
        r.n0 = max(eb1, ab1) - r.b0;
        r.b1 = 0;
        r.n = r.n0;
    } else {
        r.b0 = he ? eb0 : 0;
        r.n0 = he ? eb1 - eb0 : 0;
        r.b1 = ab0;
        r.n = r.n0 + (ha ? ab1 - ab0 : 0);
    }
    return r;
}

// Modified score in log2 units of a raw dot product.
__device__ __forceinline__ float modified(const ModParams &p, float dot)
{
    if (!p.capped) return dot * p.d.scale_log2;
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + fast_exp2(dot * p.cap_in)));
    return fmaf(-2.f * p.cap_out, r, p.cap_out);
}

// What a query column needs when it masks or biases.
struct Column {
    Range r;
    float slope;   // log2 units per position
    int32_t pos;
};

template <int D, int NT, int KIND>
__host__ __device__ constexpr int mod_smem_bytes()
{
    return decode_smem_bytes<D, NT, KIND>() + 32 * static_cast<int>(sizeof(Column));
}

// The running softmax of a warp over its 16-token blocks, see kvc_decode.cuh for the
// operand layouts.  full: every column reads the whole block.
template <int D, int NT, int KIND, bool PSPLIT>
__device__ __forceinline__ void mod_block_update(const ModParams &p, uint32_t st, const uint32_t (&qf)[NT][D / 16][2],
                                                 float (&m_run)[NT][2], float (&l_run)[NT][2],
                                                 float (&oacc)[D / 16][NT][4], bool full, int tok0,
                                                 const Column *cols, int lane)
{
    using C = DecodeCfg<D, KIND>;
    constexpr bool INT4 = KIND == KV_INT4, QUANT = KIND != KV_BF16;
    const int gq = lane >> 2, tg = lane & 3;
    constexpr int NACC = NT == 1 ? 2 : 1;
    float sc[NT][4], sc2[NT][4];
#pragma unroll
    for (int jn = 0; jn < NT; ++jn)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[jn][c] = sc2[jn][c] = 0.f;
    auto acc = [&](int jn, int kk) -> float(&)[4] { return (NACC == 2 && (kk & 1)) ? sc2[jn] : sc[jn]; };
    // ---- S^T = K Q^T
    if constexpr (!QUANT) {
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS; ++kk) {
            uint32_t a[4];
            ldsm_x4(a, st + swz((lane & 7) + ((lane >> 3) & 1) * 8, 2 * kk + (lane >> 4)));
#pragma unroll
            for (int jn = 0; jn < NT; ++jn) mma_bf16(acc(jn, kk), a, qf[jn][kk]);
        }
    } else if constexpr (INT4) {
        uint4 kw[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) kw[r] = lds128(st + swz64(gq + 8 * r, tg));
        const uint32_t k0[4] = {kw[0].x, kw[0].y, kw[0].z, kw[0].w}, k1[4] = {kw[1].x, kw[1].y, kw[1].z, kw[1].w};
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS; ++kk) {
            const int sh = 8 * (kk & 1);
            const uint32_t w0 = k0[kk >> 1] >> sh, w1 = k1[kk >> 1] >> sh;
            const uint32_t a[4] = {nibbles_to_f16x2(w0), nibbles_to_f16x2(w1), nibbles_hi_to_f16x2(w0),
                                   nibbles_hi_to_f16x2(w1)};
#pragma unroll
            for (int jn = 0; jn < NT; ++jn) mma_f16(acc(jn, kk), a, qf[jn][kk]);
        }
    } else {
        uint32_t kw[2][D / 16];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int u = 0; u < D / 64; ++u) {
                const uint4 v = lds128(st + swz(gq + 8 * r, (D / 64) * tg + u));
                kw[r][4 * u + 0] = v.x;
                kw[r][4 * u + 1] = v.y;
                kw[r][4 * u + 2] = v.z;
                kw[r][4 * u + 3] = v.w;
            }
#pragma unroll
        for (int kk = 0; kk < C::KSTEPS; ++kk) {
            uint32_t a[4];
            e4m3x4_to_f16x2x2(kw[0][kk], a[0], a[2]);
            e4m3x4_to_f16x2x2(kw[1][kk], a[1], a[3]);
#pragma unroll
            for (int jn = 0; jn < NT; ++jn) mma_f16(acc(jn, kk), a, qf[jn][kk]);
        }
    }
    if constexpr (NACC == 2)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[0][c] += sc2[0][c];

    // ---- modify, mask, and the online softmax (log2 units; reference maxima move only past the slack)
    uint32_t pb[NT][2], pl[NT][2];
    float alpha[NT][2];
    bool moved = false;
#pragma unroll
    for (int jn = 0; jn < NT; ++jn) {
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[jn][c] = modified(p, sc[jn][c]);
        if (p.alibi) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const Column &k = cols[8 * jn + 2 * tg + c];
                const float slope = k.slope;
                const int pos = k.pos, t = tok0 + gq;
                sc[jn][c] = fmaf(-slope, static_cast<float>(abs(pos - t)), sc[jn][c]);
                sc[jn][c + 2] = fmaf(-slope, static_cast<float>(abs(pos - t - 8)), sc[jn][c + 2]);
            }
        }
        if (!full) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const Range r = cols[8 * jn + 2 * tg + c].r;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int t = tok0 + gq + 8 * u;
                    const bool seen = (t >= r.lo && t < r.hi) || (t >= r.d && t < r.e);
                    sc[jn][c + 2 * u] = seen ? sc[jn][c + 2 * u] : -INFINITY;
                }
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float bm = fmaxf(sc[jn][c], sc[jn][c + 2]);
            bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 4));
            bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 8));
            bm = fmaxf(bm, __shfl_xor_sync(kFull, bm, 16));
            const bool up = bm > m_run[jn][c] + kRescaleSlack;   // false while nothing has been read
            alpha[jn][c] = up ? fast_exp2(m_run[jn][c] - bm) : 1.f;
            m_run[jn][c] = up ? bm : m_run[jn][c];
            moved |= up;
            const float mref = m_run[jn][c] == -INFINITY ? 0.f : m_run[jn][c];
            const float p0 = fast_exp2(sc[jn][c] - mref), p1 = fast_exp2(sc[jn][c + 2] - mref);
            l_run[jn][c] = l_run[jn][c] * alpha[jn][c] + p0 + p1;
            sc[jn][c] = p0;
            sc[jn][c + 2] = p1;
        }
        if constexpr (!QUANT) {
            const uint32_t h0 = pack_bf16(sc[jn][0], sc[jn][1]), h1 = pack_bf16(sc[jn][2], sc[jn][3]);
            pb[jn][0] = movmatrix_trans(h0);
            pb[jn][1] = movmatrix_trans(h1);
            if constexpr (PSPLIT) {
                pl[jn][0] = movmatrix_trans(pack_bf16(sc[jn][0] - bf16_lo(h0), sc[jn][1] - bf16_hi(h0)));
                pl[jn][1] = movmatrix_trans(pack_bf16(sc[jn][2] - bf16_lo(h1), sc[jn][3] - bf16_hi(h1)));
            }
        } else {
            pb[jn][0] = movmatrix_trans(pack_f16(sc[jn][0], sc[jn][1]));
            pb[jn][1] = movmatrix_trans(pack_f16(sc[jn][2], sc[jn][3]));
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
    if constexpr (!QUANT) {
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) {
            uint32_t a[4];
            ldsm_x4_trans(a, st + swz(kBS + (lane & 7) + ((lane >> 4) & 1) * 8, 2 * mt + ((lane >> 3) & 1)));
#pragma unroll
            for (int jn = 0; jn < NT; ++jn) {
                mma_bf16(oacc[mt][jn], a, pb[jn]);
                if constexpr (PSPLIT) mma_bf16(oacc[mt][jn], a, pl[jn]);
            }
        }
    } else if constexpr (INT4) {
        const uint32_t par = static_cast<uint32_t>(tg & 1);
        uint32_t vw[4][2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = kBS + 2 * tg + ((r & 1) ^ static_cast<int>(par)) + (r >> 1) * 8;
            const uint32_t a = st + swz64(row, gq >> 1) + 8 * (gq & 1);
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
                const uint32_t a[4] = {nibbles_to_f16x2(x01), nibbles_hi_to_f16x2(x01), nibbles_to_f16x2(x89),
                                       nibbles_hi_to_f16x2(x89)};
#pragma unroll
                for (int jn = 0; jn < NT; ++jn) mma_f16(oacc[4 * w + k][jn], a, pb[jn]);
            }
    } else {
        uint32_t vw[4][D / 32];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int u = 0; u < D / 128; ++u) {
                const uint4 v = lds128(st + swz(kBS + 2 * tg + (r & 1) + (r >> 1) * 8, (D / 128) * gq + u));
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
                mma_f16(oacc[2 * w][jn], a0, pb[jn]);
                mma_f16(oacc[2 * w + 1][jn], a1, pb[jn]);
            }
        }
    }
}

// grid (split, KV head, unit), 128 threads: the split kernel's decomposition (kvc_decode.cuh).
// A unit is ppu consecutive query positions x the g query heads of a KV head (decode: ppu = 1).
// Splits share a unit's virtual blocks evenly in runs of `chunk`; a split without blocks leaves
// (-inf, 0) for the merge, a unit of one split writes its outputs at once and leaves (-inf, -1).
template <int D, int NT, int KIND, bool PSPLIT, bool TILE>
__global__ void __launch_bounds__(kThreads) mod_kernel(const __grid_constant__ CUtensorMap tmap, const ModParams mp)
{
    using C = DecodeCfg<D, KIND>;
    constexpr bool INT4 = KIND == KV_INT4, QUANT = KIND != KV_BF16;
    const DecodeParams &p = mp.d;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int split = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tg = lane & 3;
    const int hq0 = h * p.g;
    const int rows = TILE ? p.ppu * p.g : p.g;
    // Only this call's own merge may start early (it waits for this grid): the chunk's kernel of kvc_mixed_step
    // starts without waiting for the kernel before the step, whose outputs it may overwrite.
    if (p.part_ml && !p.counters) allow_dependent_launch();
    grid_dependency_wait();

    auto col_pos = [&](int qi) { return TILE ? b * p.ppu + qi / p.g : b; };   // row of q: chunk position or sequence
    auto col_real = [&](int qi) { return qi < rows && (!TILE || col_pos(qi) < p.n_pos); };
    auto col_orow = [&](int qi) { return static_cast<size_t>(col_pos(qi)) * p.H_Q + hq0 + (TILE ? qi % p.g : qi); };

    constexpr int kBars = decode_smem_bytes<D, NT, KIND>() - 1024 - kWarps * C::R * 8;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kBars);
    Column *cols = reinterpret_cast<Column *>(smem + kBars + kWarps * C::R * 8);
    if (lane == 0) {
        for (int s = 0; s < C::R; ++s) mbar_init(smem_u32(&bars[warp * C::R + s]), 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) prefetch_tensormap(&tmap);

    // ---- what the columns read, and the unit's blocks (every warp computes the same)
    int total;
    BlockRuns br;
    int full_lo, full_hi, lead_lo, lead_hi;   // every column reads [full_lo, full_hi) and [lead_lo, lead_hi)
    {
        Range r{0, 0, 0, 0};
        bool real = false;
        int pos = 0;
        if constexpr (TILE) {
            total = p.len_base + p.n_pos;
            const int i = b * p.ppu + lane;   // lane = position of the unit (ppu <= 32)
            real = lane < p.ppu && i < p.n_pos;
            pos = p.len_base + i;
            if (real) r = query_range(mp, pos, total, mp.doc_start ? __ldg(mp.doc_start + i) : 0);
        } else {
            total = __ldg(p.lens + b);
            if (total < 0 || static_cast<int64_t>(total) > static_cast<int64_t>(p.max_blocks) * kBS) {
                if (split == 0 && threadIdx.x == 0) atomicOr(p.err, KVC_EBIT_RANGE);
                total = 0;
            }
            real = total > 0;   // the same for every lane
            pos = total - 1;
            if (real) r = query_range(mp, pos, total, 0);
        }
        const bool ha = real && r.hi > r.lo, he = real && r.e > r.d;
        const int a0 = __reduce_min_sync(kFull, ha ? r.lo : 0x7FFFFFFF), a1 = __reduce_max_sync(kFull, ha ? r.hi : 0);
        const int e0 = __reduce_min_sync(kFull, he ? r.d : 0x7FFFFFFF), e1 = __reduce_max_sync(kFull, he ? r.e : 0);
        br = block_runs(e1 > 0 ? e0 : 0, e1, a1 > 0 ? a0 : 0, a1);
        full_lo = __reduce_max_sync(kFull, real ? r.lo : 0);
        full_hi = __reduce_min_sync(kFull, real ? r.hi : 0x7FFFFFFF);   // a row with lo >= hi leaves nothing full
        lead_lo = __reduce_max_sync(kFull, real ? r.d : 0);
        lead_hi = __reduce_min_sync(kFull, real ? r.e : 0x7FFFFFFF);
        if (warp == 0) {
            for (int qi = lane; qi < 32; qi += 32) {
                Column k;
                const int src = TILE ? min(qi / p.g, 31) : 0;
                k.r.lo = __shfl_sync(kFull, r.lo, src);
                k.r.hi = __shfl_sync(kFull, r.hi, src);
                k.r.d = __shfl_sync(kFull, r.d, src);
                k.r.e = __shfl_sync(kFull, r.e, src);
                k.pos = __shfl_sync(kFull, pos, src);
                const bool cr = col_real(qi) && total > 0;
                if (!cr) k.r = Range{0, 0, 0, 0};
                k.slope = (cr && mp.alibi) ? __ldg(mp.alibi + hq0 + (TILE ? qi % p.g : qi)) * 1.4426950408889634f : 0.f;
                cols[qi] = k;
            }
        }
    }
    __syncthreads();

    const int ns = min((br.n + p.chunk - 1) / p.chunk, p.max_splits);
    auto mark = [&](float l) {   // this split's (m, l) of every row: nothing read (l = 0) or finished elsewhere (-1)
        if (p.part_ml && !p.counters && threadIdx.x < rows && col_real(threadIdx.x))
            p.part_ml[col_orow(threadIdx.x) * p.max_splits + split] = make_float2(-INFINITY, l);
    };
    if (br.n == 0) {   // nothing to read: zero output, lse = -inf
        if (split == 0) {
            for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads)
                if (col_real(i / (D / 2)))
                    reinterpret_cast<uint32_t *>(mp.out + col_orow(i / (D / 2)) * D)[i % (D / 2)] = 0u;
            if (p.lse && threadIdx.x < rows && col_real(threadIdx.x)) p.lse[col_orow(threadIdx.x)] = -INFINITY;
        }
        mark(-1.f);
        return;
    }
    const int blk0 = split * p.chunk;
    if (blk0 >= br.n) {
        mark(ns == 1 ? -1.f : 0.f);
        return;
    }
    const int nloc = (split == p.max_splits - 1 ? br.n : min(br.n, blk0 + p.chunk)) - blk0;
    const int32_t *bt_row = p.bt + static_cast<int64_t>(TILE ? 0 : b) * p.bt_stride;

    const int nmine = nloc > warp ? (nloc - warp + kWarps - 1) / kWarps : 0;   // this warp's blocks
    const uint32_t st_base = smem_u32(smem + warp * C::R * C::STAGE);
    const uint32_t bar_base = smem_u32(&bars[warp * C::R]);
    const int64_t row_layer = static_cast<int64_t>(p.layer) * p.N;

    auto load_entry = [&](int jj) -> int32_t {
        return jj < nmine ? __ldg(bt_row + br.at(blk0 + warp + kWarps * jj)) : -1;
    };
    int32_t t_cur = load_entry(lane), t_next = load_entry(32 + lane);
    auto entry = [&](int jj, int jbase) -> int32_t {
        const int32_t v = (jj - jbase < 32) ? t_cur : t_next;
        return __shfl_sync(kFull, v, (jj - jbase) & 31);
    };
    auto issue = [&](int jj, int jbase) {   // warp-collective; lane 0 issues
        const int32_t phys = entry(jj, jbase);
        if (lane == 0 && !p.stall_loads) {
            const uint32_t bar = bar_base + 8u * static_cast<uint32_t>(jj % C::R);
            if (phys < 0 || static_cast<int64_t>(phys) >= p.N) {
                const int t = br.at(blk0 + warp + kWarps * jj) * kBS;   // an error only if some column reads it
                for (int qi = 0; qi < rows; ++qi) {
                    const Range r = cols[qi].r;
                    if ((t < r.hi && t + kBS > r.lo && r.hi > r.lo) || (t < r.e && t + kBS > r.d && r.e > r.d)) {
                        atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
                        break;
                    }
                }
                mbar_arrive(bar);   // complete the phase without data; the consumer skips it
            } else {
                const int32_t y = static_cast<int32_t>(((row_layer + phys) * p.H_KV + h) * C::BOX_ROWS);
                const uint32_t dst = st_base + static_cast<uint32_t>((jj % C::R) * C::STAGE);
                mbar_arrive_expect_tx(bar, C::STAGE);
#pragma unroll
                for (int band = 0; band < C::BANDS; ++band)
                    tma_load_2d(dst + band * C::BOX_BYTES, &tmap, bar, band * C::BOX_X, y);
            }
        }
    };
    for (int jj = 0; jj < min(C::R, nmine); ++jj) issue(jj, 0);

    // ---- query fragments (B operand, k = channel, n = query column)
    uint32_t qf[NT][C::KSTEPS][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int qi = 8 * j + gq;
        const bool real = col_real(qi);
        const uint16_t *qrow = p.q + (real ? col_orow(qi) : static_cast<size_t>(0)) * D;
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

    float m_run[NT][2], l_run[NT][2];
    float oacc[C::MT][NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        m_run[j][0] = m_run[j][1] = -INFINITY;
        l_run[j][0] = l_run[j][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt) oacc[mt][j][0] = oacc[mt][j][1] = oacc[mt][j][2] = oacc[mt][j][3] = 0.f;
    }

    int j = 0;
    bool timed_out = false;
    for (; j < nmine; ++j) {
        const int jbase = j & ~31;
        if (j > 0 && (j & 31) == 0) {
            t_cur = t_next;
            t_next = load_entry(j + 32 + lane);
        }
        const int s = j % C::R;
        const bool ok = mbar_wait_bounded(bar_base + 8u * s, static_cast<uint32_t>((j / C::R) & 1));
        if (!__all_sync(kFull, ok)) {
            timed_out = true;
            break;
        }
        const int32_t phys = entry(j, jbase);
        if (phys >= 0 && static_cast<int64_t>(phys) < p.N) {
            const uint32_t st = st_base + static_cast<uint32_t>(s * C::STAGE);
            const int tok0 = br.at(blk0 + warp + kWarps * j) * kBS;
            const bool full = (tok0 >= full_lo && tok0 + kBS <= full_hi) || (tok0 >= lead_lo && tok0 + kBS <= lead_hi);
            // value rows that no column reads may hold anything (NaN included): zero them
            // (every int4 nibble is a finite value, and its weight there is 0)
            if (!INT4 && !full) {
                uint32_t used = 0u;   // bit t: some column reads the block's row t
                if (lane < rows) {
                    const Range r = cols[lane].r;
#pragma unroll
                    for (int t = 0; t < kBS; ++t)
                        used |= ((tok0 + t >= r.lo && tok0 + t < r.hi) || (tok0 + t >= r.d && tok0 + t < r.e)) ? 1u << t : 0u;
                }
                used = __reduce_or_sync(kFull, used);
                for (int i = lane; i < kBS * C::BANDS * 8; i += 32)
                    if (!(used >> (i / (C::BANDS * 8)) & 1u))
                        sts128_zero(st + swz(kBS + i / (C::BANDS * 8), i % (C::BANDS * 8)));
            }
            __syncwarp();
            mod_block_update<D, NT, KIND, PSPLIT>(mp, st, qf, m_run, l_run, oacc, full, tok0, cols, lane);
        }
        __syncwarp();
        if (j + C::R < nmine) {
            if (lane == 0) fence_proxy_async_smem();
            issue(j + C::R, jbase);
        }
    }
    if (timed_out) {   // record, then let copies already in flight land before the CTA exits
        if (lane == 0) {
            atomicOr(p.err, KVC_EBIT_TIMEOUT);
            for (int jj = j; jj < min(nmine, j + C::R); ++jj)
                (void)mbar_wait_bounded(bar_base + 8u * (jj % C::R), static_cast<uint32_t>((jj / C::R) & 1), 100000000ull);
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

    // ---- combine the four warps (the rings' memory reused), then write
    __syncthreads();
    constexpr int QW = NT * 8;
    float *cm = reinterpret_cast<float *>(smem);
    float *cl = cm + kWarps * QW;
    float *co = cl + kWarps * QW;
#pragma unroll
    for (int jn = 0; jn < NT; ++jn) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
            if (gq == 0) {
                cm[warp * QW + 8 * jn + 2 * tg + c] = m_run[jn][c];
                cl[warp * QW + 8 * jn + 2 * tg + c] = l_run[jn][c];
            }
#pragma unroll
        for (int mt = 0; mt < C::MT; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int qi = 8 * jn + 2 * tg + (c & 1);
                const int dim = QUANT ? gq * (D / 8) + 2 * mt + (c >> 1) : 16 * mt + gq + 8 * (c >> 1);
                co[(warp * QW + qi) * D + dim] = oacc[mt][jn][c];
            }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 2); i += kThreads) {
        const int qi = i / (D / 2), d = 2 * (i % (D / 2));
        if (!col_real(qi)) continue;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, cm[w * QW + qi]);
        const float Mref = M == -INFINITY ? 0.f : M;
        float L = 0.f, O0 = 0.f, O1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float e = fast_exp2(cm[w * QW + qi] - Mref);   // warps that read nothing: exp2(-inf) = 0
            L += e * cl[w * QW + qi];
            O0 += e * co[(w * QW + qi) * D + d];
            O1 += e * co[(w * QW + qi) * D + d + 1];
        }
        if constexpr (QUANT) {
            O0 *= __ldg(p.s_v + static_cast<size_t>(h) * D + d);
            O1 *= __ldg(p.s_v + static_cast<size_t>(h) * D + d + 1);
        }
        const size_t bq = col_orow(qi);
        if (ns == 1) {
            const bool none = L == 0.f;   // a row that reads nothing
            *reinterpret_cast<uint32_t *>(mp.out + bq * D + d) = none ? 0u : pack_bf16(O0 / L, O1 / L);
            if (d == 0 && p.lse) p.lse[bq] = none ? -INFINITY : (M + log2f(L)) * kLn2;
        } else {
            const size_t pi = bq * p.max_splits + split;
            *reinterpret_cast<float2 *>(p.part_o + pi * D + d) = make_float2(O0, O1);
            if (d == 0) p.part_ml[pi] = make_float2(M, L);
        }
    }
    if (ns == 1) {
        mark(-1.f);
        return;
    }
    if (!p.counters) return;   // without counters the host launches the merge kernel

    // ---- split merge by the last split CTA of the unit to finish
    __shared__ uint32_t last_flag;
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t prev = atomicAdd(p.counters + static_cast<size_t>(b) * p.H_KV + h, 1u);
        last_flag = (prev == static_cast<uint32_t>(ns - 1)) ? 1u : 0u;
    }
    __syncthreads();
    if (!last_flag) return;
    __threadfence();
    float *wsm = reinterpret_cast<float *>(smem);   // [rows][ns] weights, then [rows] 1/L
    float *linv = wsm + rows * ns;
    for (int qi = warp; qi < rows; qi += kWarps) {
        if (!col_real(qi)) continue;   // warp-uniform
        const size_t bq = col_orow(qi);
        const float2 *ml = p.part_ml + bq * p.max_splits;
        float m = -INFINITY;
        for (int sp = lane; sp < ns; sp += 32) m = fmaxf(m, __ldcg(&ml[sp].x));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        const float Mref = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        for (int sp = lane; sp < ns; sp += 32) {
            const float2 v = __ldcg(ml + sp);
            const float e = fast_exp2(v.x - Mref);
            wsm[qi * ns + sp] = e;
            l += e * v.y;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
        if (lane == 0) {
            linv[qi] = l == 0.f ? 0.f : 1.f / l;   // 0: the row reads nothing, its partials count nothing
            if (p.lse) p.lse[bq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        }
    }
    __syncthreads();
    constexpr int D4 = D / 4;
    for (int i = threadIdx.x; i < rows * D4; i += kThreads) {
        const int qi = i / D4, d4 = i - qi * D4;
        if (!col_real(qi)) continue;
        const size_t bq = col_orow(qi);
        const float4 *po = reinterpret_cast<const float4 *>(p.part_o + bq * p.max_splits * D) + d4;
        const float *w = wsm + qi * ns;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int sp = 0; sp < ns; ++sp) {
            const float4 o = __ldcg(po + static_cast<size_t>(sp) * D4);
            const float e = w[sp];
            if (e == 0.f) continue;   // a split that read nothing for this row
            acc.x = fmaf(e, o.x, acc.x);
            acc.y = fmaf(e, o.y, acc.y);
            acc.z = fmaf(e, o.z, acc.z);
            acc.w = fmaf(e, o.w, acc.w);
        }
        const float inv = linv[qi];
        *reinterpret_cast<uint2 *>(mp.out + bq * D + 4 * d4) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
    if (threadIdx.x == 0) p.counters[static_cast<size_t>(b) * p.H_KV + h] = 0u;   // ready for the next call
}

template <int D, int NT, int KIND, bool PSPLIT, bool TILE>
DecodeKernel mod_instance()
{
    struct Tag {};
    return configured<Tag>(reinterpret_cast<const void *>(&mod_kernel<D, NT, KIND, PSPLIT, TILE>),
                           mod_smem_bytes<D, NT, KIND>(), kThreads, false);
}

// The split kernel's instance for a pool kind, head width and columns per unit (fn = nullptr: none).
DecodeKernel select_mod_bf16(int D, int cols, bool tile);
DecodeKernel select_mod_fp8(int cols, bool tile);
DecodeKernel select_mod_int4(int cols, bool tile);

}  // namespace kvc
