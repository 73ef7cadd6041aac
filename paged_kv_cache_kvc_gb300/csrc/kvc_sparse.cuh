// Sparse attention: per query row and KV head, attention over a list of blocks.
//
// Mathematics, for a row at position p, a KV head h and each of its g query heads:
//   softmax over t in { j bs + i : j listed, i < bs, t <= p } of scale <q, k_t>, times v_t.
// A listed block is bs / 16 tiles of 16 positions; each tile is one step of the online softmax of kvc_mod.cuh
// (scores of the tile on tensor cores with the positions as rows, running maximum and sum in registers, weights
// into the value product).
//
// Decomposition: a cluster of C CTAs (1, 2, 4 or 8) per (row, KV head), 4 warps each; warp w of CTA c takes tiles
// c + C (w + 4 i), each warp through a ring of TMA stages of its own.  The warps of a CTA merge in shared memory and
// the CTAs through distributed shared memory: no partial goes to global memory, so a call needs no workspace and
// one launch, and two calls share nothing.
#pragma once
#include "kvc_cluster.cuh"
#include "kvc_mod.cuh"

namespace kvc {

struct SparseParams {
    ModParams m;               // d.q, d.bt, d.bt_stride, d.max_blocks, d.B (sequences), heads, layer, N, scales, lse, out
    const int32_t *seqs;       // [rows] or nullptr: row r is sequence r
    const int32_t *positions;  // [rows]
    const int32_t *lists;      // [rows][H_KV][top_k]
    int32_t top_k;
    int32_t sub;               // tiles per block: bs / 16
};

constexpr int kSparseMost = 8;   // CTAs of a cluster

template <int D, int NT, int KIND>
__host__ __device__ constexpr int sparse_smem_bytes()
{
    return mod_smem_bytes<D, NT, KIND>();
}

// grid (C x rows, KV head), clusters of C CTAs along x
template <int D, int NT, int KIND, bool PSPLIT>
__global__ void __launch_bounds__(kThreads) sparse_kernel(const __grid_constant__ CUtensorMap tmap, const SparseParams sp)
{
    using C = DecodeCfg<D, KIND>;
    constexpr bool INT4 = KIND == KV_INT4, QUANT = KIND != KV_BF16;
    constexpr int QW = NT * 8;
    const ModParams &mp = sp.m;
    const DecodeParams &p = mp.d;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ float2 part[QW];   // this CTA's (maximum, sum) of every column
    const int cs = static_cast<int>(cluster_size()), rank = static_cast<int>(cluster_rank());
    const int row = static_cast<int>(blockIdx.x / static_cast<unsigned>(cs)), h = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, tg = lane & 3;
    const size_t orow = static_cast<size_t>(row) * p.H_Q + static_cast<size_t>(h) * p.g;   // of the group's first head

    constexpr int kBars = decode_smem_bytes<D, NT, KIND>() - 1024 - kWarps * C::R * 8;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kBars);
    Column *cols = reinterpret_cast<Column *>(smem + kBars + kWarps * C::R * 8);
    if (lane == 0) {
        for (int s = 0; s < C::R; ++s) mbar_init(smem_u32(&bars[warp * C::R + s]), 1);
        fence_barrier_init();
    }
    if (threadIdx.x == 0) prefetch_tensormap(&tmap);
    grid_dependency_wait();

    // What is known from the row alone is on its way before the first answer: sequence, position, this lane's list
    // entries and the queries.
    const int seq = sp.seqs ? __ldg(sp.seqs + row) : row;
    const int pos = __ldg(sp.positions + row);
    const int32_t *list = sp.lists + (static_cast<size_t>(row) * p.H_KV + h) * sp.top_k;
    const int first = rank + cs * warp, step = cs * kWarps, listed = sp.top_k * sp.sub;   // this warp's tiles
    auto load_entry = [&](int jj) {
        const int t = first + step * jj;
        return t < listed ? __ldg(list + t / sp.sub) : -1;
    };
    const int e_cur = load_entry(lane), e_next = load_entry(32 + lane);

    // ---- query fragments, see kvc_decode.cuh
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
    for (int qi = threadIdx.x; qi < 32; qi += kThreads) {
        Column k;
        k.r = Range{0, qi < p.g ? len : 0, 0, 0};
        k.slope = 0.f;
        k.pos = pos;
        cols[qi] = k;
    }
    __syncthreads();

    const int tiles = len > 0 ? listed : 0;
    const int nmine = tiles > first ? (tiles - first + step - 1) / step : 0;
    const int32_t *bt_row = p.bt + static_cast<int64_t>(seq) * p.bt_stride;
    const uint32_t st_base = smem_u32(smem + warp * C::R * C::STAGE);
    const uint32_t bar_base = smem_u32(&bars[warp * C::R]);
    const int own = pos / (sp.sub * kBS);

    // This warp's tiles, 32 at a time in registers: (first position, block), block -1: nothing to read.
    auto load_tile = [&](int jj, int j) -> int2 {
        if (jj >= nmine || j == -1) return make_int2(0, -1);
        const int t = first + step * jj, part = t - t / sp.sub * sp.sub;
        if (j < 0 || j > own) {
            atomicOr(p.err, KVC_EBIT_RANGE);
            return make_int2(0, -1);
        }
        const int tok0 = (j * sp.sub + part) * kBS;
        if (tok0 >= len) return make_int2(0, -1);   // past the query in its own block
        int phys = __ldg(bt_row + j);
        if (phys < 0 || static_cast<int64_t>(phys) >= p.N) {
            atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
            phys = -1;
        }
        return make_int2(tok0, phys);
    };
    int2 t_cur = load_tile(lane, e_cur), t_next = load_tile(32 + lane, e_next);
    auto entry = [&](int jj, int jbase) -> int2 {
        const int2 v = (jj - jbase < 32) ? t_cur : t_next;
        return make_int2(__shfl_sync(kFull, v.x, (jj - jbase) & 31), __shfl_sync(kFull, v.y, (jj - jbase) & 31));
    };
    const int64_t layer_row = static_cast<int64_t>(p.layer) * p.N;
    auto issue = [&](int jj, int jbase) {   // warp-collective; lane 0 issues
        const int2 e = entry(jj, jbase);
        if (lane == 0 && !p.stall_loads) {
            const uint32_t bar = bar_base + 8u * static_cast<uint32_t>(jj % C::R);
            if (e.y < 0) {
                mbar_arrive(bar);   // complete the phase without data; the consumer skips it
            } else {
                const uint32_t dst = st_base + static_cast<uint32_t>((jj % C::R) * C::STAGE);
                const int64_t blk = (layer_row + e.y) * p.H_KV + h;
                mbar_arrive_expect_tx(bar, C::STAGE);
                // keys, then the values behind them in the same stage, one box per 128-byte band each
                constexpr int rows_per_tile = C::BOX_ROWS / 2;   // map rows (int4: 128-byte lines) of 16 positions
                const int part = (e.x / kBS) % sp.sub;
                const int32_t y = static_cast<int32_t>(blk * (2 * rows_per_tile) * sp.sub) + part * rows_per_tile;
#pragma unroll
                for (int band = 0; band < C::BANDS; ++band) {
                    tma_load_2d(dst + band * C::BOX_BYTES, &tmap, bar, band * C::BOX_X, y);
                    tma_load_2d(dst + band * C::BOX_BYTES + C::BOX_BYTES / 2, &tmap, bar, band * C::BOX_X,
                                y + rows_per_tile * sp.sub);
                }
            }
        }
    };
    for (int jj = 0; jj < min(C::R, nmine); ++jj) issue(jj, 0);

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
            t_next = load_tile(j + 32 + lane, load_entry(j + 32 + lane));
        }
        const int s = j % C::R;
        const bool ok = mbar_wait_bounded(bar_base + 8u * s, static_cast<uint32_t>((j / C::R) & 1));
        if (!__all_sync(kFull, ok)) {
            timed_out = true;
            break;
        }
        const int2 e = entry(j, jbase);
        if (e.y >= 0) {
            const uint32_t st = st_base + static_cast<uint32_t>(s * C::STAGE);
            const int valid = min(kBS, len - e.x);
            // value rows past the query may hold anything (NaN included): zero them
            if (!INT4 && valid < kBS) {
                const int nz = (kBS - valid) * C::BANDS * 8;
                for (int i = lane; i < nz; i += 32)
                    sts128_zero(st + swz(kBS + valid + i / (C::BANDS * 8), i % (C::BANDS * 8)));
            }
            __syncwarp();
            mod_block_update<D, NT, KIND, PSPLIT>(mp, st, qf, m_run, l_run, oacc, valid == kBS, e.x, cols, lane);
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

    // ---- the warps' partials to shared memory (the ring is free), then one sum per CTA, then one per cluster
    __syncthreads();
    float *cm = reinterpret_cast<float *>(smem);
    float *cl = cm + kWarps * QW;
    float *co = cl + kWarps * QW;   // [warp][column][D]
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
    for (int i = threadIdx.x; i < p.g * (D / 2); i += kThreads) {
        const int qi = i / (D / 2), d = 2 * (i - qi * (D / 2));
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, cm[w * QW + qi]);
        const float Mref = M == -INFINITY ? 0.f : M;
        float L = 0.f, O0 = 0.f, O1 = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float e = fast_exp2(cm[w * QW + qi] - Mref);   // warps that read nothing: exp2(-inf) = 0
            const float2 o = *reinterpret_cast<const float2 *>(co + (w * QW + qi) * D + d);
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
            *reinterpret_cast<float2 *>(co + qi * D + d) = make_float2(O0, O1);
            if (d == 0) part[qi] = make_float2(M, L);
        }
    }
    if (cs == 1) return;

    // CTA `rank` finishes its part of the group's channels from all CTAs' sums
    cluster_sync();
    for (int i = rank * kThreads + threadIdx.x; i < p.g * (D / 4); i += cs * kThreads) {
        const int qi = i / (D / 4), d = 4 * (i - qi * (D / 4));
        float2 ml[kSparseMost];
        float4 o[kSparseMost];
#pragma unroll
        for (int r = 0; r < kSparseMost; ++r) {
            ml[r] = make_float2(-INFINITY, 0.f);
            o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < cs) {
                ml[r] = cluster_ld2(cluster_addr(smem_u32(part + qi), r));
                o[r] = cluster_ld4(cluster_addr(smem_u32(co + qi * D + d), r));
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

template <int D, int NT, int KIND, bool PSPLIT>
SparseKernel sparse_instance()
{
    struct Tag {};
    return {&sparse_kernel<D, NT, KIND, PSPLIT>,
            configured<Tag>(reinterpret_cast<const void *>(&sparse_kernel<D, NT, KIND, PSPLIT>), sparse_smem_bytes<D, NT, KIND>(),
                            kThreads, false)};
}

SparseKernel select_sparse_bf16(int D, int g);
SparseKernel select_sparse_fp8(int g);
SparseKernel select_sparse_int4(int g);

}  // namespace kvc
