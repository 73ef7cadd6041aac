// Attention with modified scores on the fifth-generation tensor cores (tcgen05), scores, weights
// and outputs in tensor memory (TMEM).  The mathematics and the masks are kvc_mod.cuh's.
//
// A unit is KV head h and 256 query rows: 2 x 128 / g consecutive chunk positions x the g query
// heads of h, as two tiles of 128 rows (row r of a tile = position r / g, head h g + r mod g).  A
// staged tile of 64 keys and values serves both.  Each query tile is its own chain
//     S[128 x 64] = Q K^T  ->  softmax warps: P over S in TMEM  ->  O += P V
// with two score buffers, so that a step's scores are there when the softmax warps are done with the
// step before.  (One 128-key buffer per query tile measured 1.7x slower: the two chains fell into
// step, both computing weights, then both waiting for the tensor cores.)  384 threads:
//   warps 0..3, 4..7  softmax of tile 0, 1; thread = query row (TMEM lane)
//   warps 8, 9        bring the key and the value tiles into rings; warp 9 also zeroes value rows that
//                     no row of the unit reads (a zero weight times NaN is NaN)
//   warps 10, 11      MMA issuers of tile 0, 1
// bf16 pools: warps 8 and 9 issue one 16-row TMA box per block and 128-byte band (one warp's boxes
// issue ~40 ns apart, hence two warps).  e4m3 and int4 pools: 512 threads, warp 8 issues whole blocks of
// codes into a third ring, warps 12 and 13 widen the landed keys and 14 and 15 the values to f16,
// exactly (one warp for each of the two took 800 and 2 000 cycles a tile, against 1 000 for the rest of
// the work on it), and the softmax warps take registers over from the others.  The
// queries are then q times the key scales, rounded to f16 (as in the split kernel), and the value
// scales multiply the outputs.  int4 codes widen in the order 0, 4, 1, 5, 2, 6, 3, 7 of every eight
// channels (two nibbles 16 bits apart are one mask): the queries are staged in that order, and the
// outputs' registers are read in it.
//
// Work split.  The unit's key tiles (only those that some row reads, kvc_mod.cuh) of every head and
// unit form one line of W tiles; CTA c of G takes tiles [c W / G, (c + 1) W / G), whatever units they
// belong to, so every SM gets the same work to within a tile: a late chunk of few long rows, a long
// triangular one and a ragged decode batch alike.  A unit that lies in one CTA is written at once; a
// unit's start and end cost about eight tiles (its queries staged, the first scores, its outputs written:
// 9 us against 1.1 us a tile), so the line gives every unit kMtStart tiles more than it has.  A
// unit cut by CTA borders leaves fp32 partials for mod_tc_merge_kernel, which adds them in CTA order; a
// CTA leaves pieces of two units at most (kvc_mod_line.cuh).  (Merged by the unit's last CTA instead, 600
// queries of 1800 positions took 43 us, 20 pieces of a 5-query chunk 9 us of its 36: one SM's loads against
// all SMs'.)
//
// Short units (little more than the start and the merge they would cost) are dealt whole instead, one
// after the other, and nothing is merged.
//
// Few rows (a chunk of at most 128 / g positions, a decode sequence): both chains take the same rows,
// chain 0 every other tile and chain 1 the rest.  In a unit that lies in one CTA (a chunk of 600 positions of
// 32 heads over 8 is 152 of them, dealt whole; the short sequences of a ragged batch that is cut) the chains'
// sums meet in shared memory; the pieces of a cut one hold both chains' sums, and the merge joins them too.
//
// Weights.  On bf16 pools with capped scores (and no bias) x lies in [-cap, cap], so the softmax needs
// no maximum: 2^(x - cap / 2) fits fp32 and bf16 for caps up to 55 (80 in log2 units), and a score
// needs no second look.  Otherwise a row's reference moves when a score passes it by more
// than SLACK, and the row's outputs are rescaled in TMEM.  The weights enter the value
// product as bf16 (f16 with e4m3 and int4 pools, where they stay under 2^15); their sum is taken before
// the rounding: a relative error of at most 2^-8 in each, independent, which an output rounded to
// bf16 hides.  A row that reads a few keys has no such average: against the fixed reference its outputs are
// divided by the sum of the rounded weights of the tiles it does not read whole (one key read gives its
// value back exactly, as the moving maximum's weight of 1 does), and lse keeps the unrounded sum.
#pragma once
#include <type_traits>

#include "kvc_decode_tc.cuh"
#include "kvc_mod.cuh"
#include "kvc_mod_line.cuh"

namespace kvc {

constexpr int kMtKeys = 64;                        // keys per tile
constexpr int kMtBlocks = kMtKeys / kBS;
constexpr int kMtJoin = 2;                         // the meeting of two chains, in tiles
constexpr int kMtCut = 16;                         // what cutting units costs a CTA, in tiles (run_tc)
constexpr int kMtBrief = 16;                       // a CTA's share of the line up to which kMtCappedBrief serves
constexpr float kMtCapLimit = 80.f;                // cap in log2 units up to which no maximum is needed

struct ModTcParams {
    ModParams m;          // m.d.ppu: positions per query tile (a decode sequence's one)
    int32_t units;        // units per head
    int32_t whole;        // 1: no partials, units are dealt whole
    int32_t split;        // 1: a unit is one query tile's positions, and both chains take its rows (below)
    int32_t total;        // positions the row holds (prefill)
    int32_t *prefix;      // few-row calls: [units + 1] place of each unit on a head's line, for the merge
    int4 *cuts;           // other calls: [G] {head, unit, pieces (0: none), slot} of the unit that CTA c starts
                          // and a later CTA ends, for the merge
    float *part_o;        // float4 [2 G][D / 4][256] (a warp's rows side by side), few-row calls [2 G][256][D / 4]
    float2 *part_ml;      // [2 G][256]
};

// How the weights are taken.  Plain: neither cap nor bias.  Capped: capped scores without a bias.  Brief: the same with
// one code for all tiles, half as much to fetch when a call starts and up to 5 % slower per tile; us brief / not, 32 heads
// over 8: 64 queries at 0 10.1 / 10.3, 256 at 0 10.5 / 11.9, 5 over 20 005 33.4 / 34.6, 1500 at 0 53.8 / 53.1, 2048 over
// 18 432 613 / 583.
enum TcMode { kMtGeneral, kMtPlain, kMtCapped, kMtCappedBrief };

template <int D, int KIND>
struct ModTcCfg {
    static constexpr bool QUANT = KIND != KV_BF16;
    static constexpr int THREADS = QUANT ? 512 : 384;
    static constexpr int BANDS = D / 64;
    static constexpr int QBAND = 128 * 128;            // one 128-byte column band of 128 query rows
    static constexpr int QTILE = BANDS * QBAND;
    static constexpr int KBAND = kMtKeys * 128;        // one band of 64 key or value rows
    static constexpr int STAGE = BANDS * KBAND;
    // A row's reference moves when a score passes it by more (log2 units).  f16 weights stay under 2^16; bf16's and
    // the sums have fp32's range.  (8 instead, 2048 positions over 18 432, scores of deviation 2: with a bias of slope
    // 2^-8 bf16 617 us against 533, e4m3 713 against 657; capped int4 794 against 787.  Where the bias itself climbs past
    // the slack every few tiles, slopes 2^(-8 i / H), 687 against 681 and 782 against 781.)
    static constexpr float SLACK = QUANT ? 15.f : 40.f;
    static constexpr int R = QUANT ? 3 : 4;            // ring depths (with QUANT: codes, keys and values alike)
    static constexpr int BLOCK = QUANT ? DecodeCfg<D, KIND>::STAGE : 0;   // a block's codes, keys then values
    static constexpr int RAW = kMtBlocks * BLOCK;
    static constexpr int Q = 0;                        // [2] query tiles
    static constexpr int K = 2 * QTILE;                // [R] key tiles
    static constexpr int V = K + R * STAGE;            // [R] value tiles
    static constexpr int C = V + R * STAGE;            // [R] tiles of codes
    static constexpr int PREFIX = C + R * RAW;         // int32 [kMtUnits + 1]
    static constexpr int BARS = PREFIX + ((kMtUnits + 1) * 4 + 15) / 16 * 16;
    static constexpr int NBARS = 7 * R + 14;
    static constexpr int MEET_PART = 128 * 128;        // where chains meet: 128 rows x 32 fp32 columns, twice
    static constexpr int MISC = BARS + NBARS * 8;      // scan sums [16], abort, TMEM base, block masks [16]
    static constexpr int MEET_SUMS = (MISC + 160 + 15) / 16 * 16;   // (m, l, divisor) of chain 1's 128 rows
    static constexpr int END = MEET_SUMS + 128 * 16;
    static constexpr int MEET = QTILE >= 2 * MEET_PART ? Q + QTILE : END;   // chain 1's query tile if it is large enough
    static constexpr int SMEM = 1024 + (MEET == END ? END + 2 * MEET_PART : END);
    static_assert(SMEM <= 232448, "shared memory of a CTA");
};

// The eight nibbles of a word (stored q + 8), widened to f16 in the order 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ uint4 widen_nibbles(uint32_t w)
{
    return make_uint4(nibbles_to_f16x2(w), nibbles_hi_to_f16x2(w), nibbles_to_f16x2(w >> 8), nibbles_hi_to_f16x2(w >> 8));
}

// Column of a widened eight that holds channel e.
template <int KIND>
__host__ __device__ constexpr int widened_column(int e)
{
    return KIND != KV_INT4 ? e : (e < 4 ? 2 * e : 2 * (e - 4) + 1);
}

// One warp: half of the 64 key (VALUES = false) or value rows of a tile of codes, widened into a tile of 16-bit rows
// (the 128-byte-swizzled bands that TMA writes for bf16 pools).  keep(row): false zeroes the row.  A lane takes the
// same 16-byte chunk of every 4th (e4m3) or 8th (int4) row, so that its addresses are a few bases with the swizzle
// folded in by exclusive or, plus constants.
template <int D, int KIND, bool VALUES, typename Keep>
__device__ __forceinline__ void widen_half(uint32_t codes, uint32_t wide, int half, int lane, Keep keep)
{
    using C = ModTcCfg<D, KIND>;
    constexpr bool INT4 = KIND == KV_INT4;
    static_assert(D == 128, "rows of 8 (e4m3) or 4 (int4) chunks of codes");
    constexpr int N = INT4 ? 4 : 8, ROWS = 32 / N, ITEMS = kMtKeys / 2 / ROWS;   // chunks of a row, rows at a time
    constexpr int OUT = INT4 ? 4 : 2;                                        // chunks of 8 widened channels from one
    const int lr = lane / N, ch = lane % N;
    // codes: row ROWS b + lr; int4 rows lie two to a 128-byte line (see swz, swz64)
    const uint32_t src = codes + (INT4 ? (lr >> 1) * 128 + (((((lr & 1) << 2) + ch) ^ (lr >> 1)) << 4) : lr * 128 + ((ch ^ lr) << 4)) +
                         (VALUES ? C::BLOCK / 2 : 0) + half * 2 * C::BLOCK;
    const int c8 = OUT * ch;   // the first eight channels of the chunk
    const uint32_t dst = wide + half * (kMtKeys / 2 * 128) + (c8 >> 3) * C::KBAND + lr * 128 + (((c8 & 7) ^ lr) << 4);
    constexpr int PB = kBS / ROWS;   // rows at a time per block of 16
    constexpr int LOADS = ITEMS < 8 ? ITEMS : 8;   // chunks in flight: one load at a time costs its latency
#pragma unroll
    for (int b0 = 0; b0 < ITEMS; b0 += LOADS) {
        uint4 x[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int b = b0 + i;
            x[i] = lds128((src ^ ((b & 1) ? 64u : 0u)) + (b / PB) * C::BLOCK + (b % PB) * 512);
        }
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int b = b0 + i;
            const uint32_t to = (dst ^ (!INT4 && (b & 1) ? 64u : 0u)) + b * ROWS * 128;
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            const bool ok = keep(half * (kMtKeys / 2) + b * ROWS + lr);
#pragma unroll
            for (int o = 0; o < OUT; ++o) {
                uint4 y;
                if constexpr (INT4) {
                    y = widen_nibbles(w[o]);
                } else {
                    uint32_t h[4];
                    e4m3x4_to_f16x2x2(w[2 * o], h[0], h[1]);
                    e4m3x4_to_f16x2x2(w[2 * o + 1], h[2], h[3]);
                    y = make_uint4(h[0], h[1], h[2], h[3]);
                }
                if (!ok) y = make_uint4(0u, 0u, 0u, 0u);
                sts128(to ^ (o << 4), y);
            }
        }
    }
}

// Scale 16 columns of this thread's TMEM lane (whole warp).
__device__ __forceinline__ void tmem_scale16(uint32_t taddr, float f)
{
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// A vote of the 128 threads of a query tile, or of both tiles' 256 (named barrier `id`).
__device__ __forceinline__ bool tile_all(bool v, uint32_t id, uint32_t threads)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r)
                 : "r"(v ? 1u : 0u), "r"(id), "r"(threads)
                 : "memory");
    return r != 0;
}

// Two fp32 values per instruction.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 f32x2_of(float lo, float hi)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float lo2(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v)); }
__device__ __forceinline__ float hi2(f32x2 v) { return __uint_as_float(static_cast<uint32_t>(v >> 32)); }
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b)   // NaN stays NaN
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ float fast_rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// Four capped scores in log2 units, plus (top - cap): x = top - 2 cap / (1 + 2^u), u = s * in, out = -2 cap.
// They share one reciprocal: 1 / a_i = (product of the others) / (product of all).  u is held under 30, where
// x already equals cap in fp32, so that the product stays finite.
__device__ __forceinline__ void capped4(f32x2 s01, f32x2 s23, f32x2 in, f32x2 out, f32x2 top, f32x2 &x01, f32x2 &x23)
{
    const f32x2 one = f32x2_of(1.f, 1.f), u01 = mul2(s01, in), u23 = mul2(s23, in);
    const f32x2 a = add2(f32x2_of(fast_exp2(min_nan(lo2(u01), 30.f)), fast_exp2(min_nan(hi2(u01), 30.f))), one);
    const f32x2 b = add2(f32x2_of(fast_exp2(min_nan(lo2(u23), 30.f)), fast_exp2(min_nan(hi2(u23), 30.f))), one);
    const f32x2 ab = mul2(a, b);   // (a0 a2, a1 a3)
    const float rc = fast_rcp(lo2(ab) * hi2(ab));
    const f32x2 ri = f32x2_of(rc * hi2(ab), rc * lo2(ab));   // (1 / a0 a2, 1 / a1 a3)
    x01 = fma2(mul2(ri, b), out, top);
    x23 = fma2(mul2(ri, a), out, top);
}

// Chunk position c (decode: sequence c): its position, the positions its row holds, what it reads.
struct RowView {
    int pos, total;
    Range r;
};

__device__ __forceinline__ RowView row_view(const ModTcParams &p, int c)
{
    const DecodeParams &d = p.m.d;
    RowView v;
    if (d.lens) {
        v.total = __ldg(d.lens + c);
        if (v.total < 0 || static_cast<int64_t>(v.total) > static_cast<int64_t>(d.max_blocks) * kBS) v.total = 0;
        v.pos = v.total - 1;
    } else {
        v.total = p.total;
        v.pos = d.len_base + c;
    }
    v.r = query_range(p.m, v.pos, v.total, p.m.doc_start ? __ldg(p.m.doc_start + c) : 0);
    if (v.total == 0) v.r = Range{0, 0, 0, 0};
    return v;
}

__device__ __forceinline__ int unit_positions_of(const ModTcParams &p)
{
    return p.split ? p.m.d.ppu : 2 * p.m.d.ppu;
}

// What a unit reads; the same in every thread of a warp.
struct UnitView {
    int pos0, n_pos;       // chunk positions [pos0, pos0 + n_pos)
    int a0, a1, e0, e1;    // the union of its rows' runs: [a0, a1) and [e0, e1)
    BlockRuns br;
    int tiles;             // key tiles (at least 1: a unit that reads nothing still writes its zeros)
};

// Whole warp (the reductions), u: unit of a head.
__device__ __forceinline__ UnitView unit_view(const ModTcParams &p, int u, int lane)
{
    const DecodeParams &d = p.m.d;
    const int ppu = unit_positions_of(p);
    UnitView v;
    v.pos0 = u * ppu;
    v.n_pos = min(ppu, d.n_pos - v.pos0);
    int a0 = 0x7FFFFFFF, a1 = 0, e0 = 0x7FFFFFFF, e1 = 0;
    // without documents lo, hi and e grow with the position: the first and the last row bound the runs
    const int step = p.m.doc_start ? 1 : max(1, v.n_pos - 1);
    for (int i = lane * step; i < v.n_pos; i += 32 * step) {
        const Range r = row_view(p, v.pos0 + i).r;
        if (r.hi > r.lo) {
            a0 = min(a0, r.lo);
            a1 = max(a1, r.hi);
        }
        if (r.e > r.d) {
            e0 = min(e0, r.d);
            e1 = max(e1, r.e);
        }
    }
    v.a1 = __reduce_max_sync(kFull, a1);
    v.a0 = v.a1 > 0 ? __reduce_min_sync(kFull, a0) : 0;
    v.e1 = __reduce_max_sync(kFull, e1);
    v.e0 = v.e1 > 0 ? __reduce_min_sync(kFull, e0) : 0;
    v.br = block_runs(v.e0, v.e1, v.a0, v.a1);
    v.tiles = max(1, (v.br.n + kMtBlocks - 1) / kMtBlocks);
    return v;
}

// The same count of tiles without documents, one thread.
__device__ __forceinline__ int unit_tiles(const ModTcParams &p, int u)
{
    const int ppu = unit_positions_of(p), c = u * ppu;
    const Range f = row_view(p, c).r, l = row_view(p, min(c + ppu, p.m.d.n_pos) - 1).r;
    const bool fe = f.e > f.d, le = l.e > l.d;
    const BlockRuns br = block_runs(le ? (fe ? min(f.d, l.d) : l.d) : 0, le ? l.e : 0, f.lo, l.hi);
    return max(1, (br.n + kMtBlocks - 1) / kMtBlocks);
}

// The view of a segment's unit; a whole unit's segment gets its tiles from it.
__device__ __forceinline__ UnitView unit_of(const ModTcParams &p, Segment &s, int lane)
{
    const UnitView v = unit_view(p, s.unit, lane);
    if (p.whole) s.tiles = s.k1 = v.tiles;
    return v;
}

// tmap: the pool's map of 16-row boxes (bf16), else the map of whole blocks.
template <int D, int KIND, TcMode MODE>
__global__ void __launch_bounds__(ModTcCfg<D, KIND>::THREADS, 1) mod_tc_kernel(const __grid_constant__ CUtensorMap tmap,
                                                                const ModTcParams tp)
{
    using C = ModTcCfg<D, KIND>;
    constexpr int R = C::R;
    constexpr bool CAPPED = MODE == kMtCapped || MODE == kMtCappedBrief, FIXED = CAPPED && !C::QUANT;   // FIXED: against the fixed reference
    static_assert(!C::QUANT || MODE != kMtCappedBrief, "bf16 pools");
    const ModParams &mp = tp.m;
    const DecodeParams &p = mp.d;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = p.g, ppt = p.ppu;   // positions per query tile
    const uint32_t sbase = smem_u32(smem);
    int32_t *prefix = reinterpret_cast<int32_t *>(smem + C::PREFIX);
    int32_t *misc = reinterpret_cast<int32_t *>(smem + C::MISC);
    volatile int32_t *abort_sh = misc + 32;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 33);
    volatile uint32_t *mask_sh = reinterpret_cast<volatile uint32_t *>(misc + 16);   // loaded blocks of tile kt, place kt mod 16
    auto bar = [&](int i) { return sbase + C::BARS + 8u * static_cast<uint32_t>(i); };
    // barriers: per ring slot, then per query tile
    auto kfull = [&](int s) { return bar(s); };
    auto kfree = [&](int s) { return bar(R + s); };
    auto vfull = [&](int s) { return bar(2 * R + s); };    // bf16: the copy; vready follows it
    auto vfree = [&](int s) { return bar(3 * R + s); };
    auto vready = [&](int s) { return bar(4 * R + s); };
    auto cfull = [&](int s) { return bar(5 * R + s); };    // codes
    auto cfree = [&](int s) { return bar(6 * R + s); };
    auto qfull = [&](int x) { return bar(7 * R + x); };
    auto sfull = [&](int x, int b) { return bar(7 * R + 2 + 2 * x + b); };   // per query tile and score buffer
    auto pfull = [&](int x, int b) { return bar(7 * R + 6 + 2 * x + b); };
    auto pvdone = [&](int x, int b) { return bar(7 * R + 10 + 2 * x + b); };

    if (tid == 0) {
        for (int s = 0; s < R; ++s) {
            mbar_init(kfull(s), C::QUANT ? 2 : 1);   // the copy, or the warps that widen
            mbar_init(kfree(s), tp.split ? 1 : 2);   // the chains that take the tile
            mbar_init(vfull(s), 1);
            mbar_init(vfree(s), tp.split ? 1 : 2);
            mbar_init(vready(s), C::QUANT ? 2 : 1);
            mbar_init(cfull(s), 1);
            mbar_init(cfree(s), 4);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(qfull(s), 128);
            for (int b = 0; b < 2; ++b) {
                mbar_init(sfull(s, b), 1);
                mbar_init(pfull(s, b), 128);
                mbar_init(pvdone(s, b), 1);
            }
        }
        fence_barrier_init();
        prefetch_tensormap(&tmap);
        *abort_sh = 0;
    }
    if (warp == 0) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    if (!tp.whole) allow_dependent_launch();   // for this call's own merge, which waits for this grid (kvc_mod.cuh)
    grid_dependency_wait();

    // ---- what each unit takes of the line, and the running sum
    if (tp.whole) {   // no line
    } else if (mp.doc_start) {
        for (int u = warp; u < tp.units; u += C::THREADS / 32) {
            const UnitView v = unit_view(tp, u, lane);
            if (lane == 0) prefix[u + 1] = v.tiles + kMtStart;
        }
    } else {
        for (int u = tid; u < tp.units; u += C::THREADS) {
            prefix[u + 1] = unit_tiles(tp, u) + kMtStart;
        }
    }
    if (p.lens && blockIdx.x == 0)
        for (int u = tid; u < tp.units; u += C::THREADS) {
            const int n = __ldg(p.lens + u);
            if (n < 0 || static_cast<int64_t>(n) > static_cast<int64_t>(p.max_blocks) * kBS) atomicOr(p.err, KVC_EBIT_RANGE);
        }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (!tp.whole) {
        const int per = (tp.units + C::THREADS - 1) / C::THREADS, b = tid * per, e = min(tp.units, b + per);
        int sum = 0;
        for (int u = b; u < e; ++u) sum += prefix[u + 1];
        int inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(kFull, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) misc[warp] = inc;
        __syncthreads();
        int before = inc - sum;
        for (int w = 0; w < warp; ++w) before += misc[w];
        for (int u = b; u < e; ++u) {
            before += prefix[u + 1];
            prefix[u + 1] = before;
            if (blockIdx.x == 0 && tp.split) tp.prefix[u + 1] = before;
        }
        if (tid == 0) {
            prefix[0] = 0;
            if (blockIdx.x == 0 && tp.split) tp.prefix[0] = 0;
        }
        __syncthreads();
    }
    Walk walk(prefix, tp.units, p.H_KV, blockIdx.x, gridDim.x, tp.whole != 0);

    // TMEM columns: query tile x has its score buffers at 128 x and 128 x + 64, its outputs at 256 + 128 x
    bool timed_out = false;
    // Whole warp; false: the wait expired (2 s) here or elsewhere in the CTA, which gives up.
    auto wait = [&](uint32_t b, uint32_t parity) {
        if (__all_sync(kFull, mbar_try_wait(b, parity))) return true;
        const uint64_t since = globaltimer_ns();
        for (uint32_t i = 1;; ++i) {
            if (__all_sync(kFull, mbar_try_wait(b, parity))) return true;
            if ((i & 15u) == 0u && __any_sync(kFull, *abort_sh != 0 || globaltimer_ns() - since > 2000000000ull)) break;
        }
        *abort_sh = 1;
        timed_out = true;
        return false;
    };

    if (warp >= 8) {
        if constexpr (C::QUANT) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        if (warp <= 9 || warp >= 12) {
            // -------------------------------------------------------- keys (8; 12, 13) and values (9; 14, 15)
            const bool values = C::QUANT ? warp >= 14 : warp == 9;
            const int64_t row_layer = static_cast<int64_t>(p.layer) * p.N;
            const int bl = lane & (kMtBlocks - 1), band = lane / kMtBlocks;   // this lane's block of a tile (and band)
            uint32_t kt = 0;   // tiles so far
            bool go = true;
            // which of a tile's value rows some row of the unit reads
            auto is_clean = [&](const UnitView &v, int k, uint32_t mask) {
                const int first = k * kMtBlocks;
                const bool one_run = first + kMtBlocks <= v.br.n && (first + kMtBlocks <= v.br.n0 || first >= v.br.n0);
                const int t0 = v.br.at(first) * kBS;
                return one_run && mask == (1u << kMtBlocks) - 1u && !mp.doc_start &&
                       ((t0 >= v.a0 && t0 + kMtKeys <= v.a1) || (t0 >= v.e0 && t0 + kMtKeys <= v.e1));
            };
            // which of tile k's value rows some row of the unit reads: bit row (whole warp)
            auto used_rows = [&](const UnitView &v, int k, uint32_t mask) -> uint64_t {
                const int first = k * kMtBlocks;
                uint32_t m[2] = {0u, 0u};
                auto add = [&](int lo, int hi) {   // positions [lo, hi)
#pragma unroll
                    for (int b = 0; b < kMtBlocks; ++b) {
                        if (first + b >= v.br.n || !(mask >> b & 1u)) continue;
                        const int t = v.br.at(first + b) * kBS;
                        auto below = [&](int end) -> uint32_t { return end <= t ? 0u : (end >= t + kBS ? 0xFFFFu : (1u << (end - t)) - 1u); };
                        m[b >> 1] |= (below(hi) & ~below(lo)) << (16 * (b & 1));
                    }
                };
                if (!mp.doc_start) {   // rows at consecutive positions read consecutive runs: their union has no holes
                    add(v.a0, v.a1);
                    add(v.e0, v.e1);
                } else {
                    for (int i = lane; i < v.n_pos; i += 32) {
                        const Range r = row_view(tp, v.pos0 + i).r;
                        add(r.lo, r.hi);
                        add(r.d, r.e);
                    }
                    m[0] = __reduce_or_sync(kFull, m[0]);
                    m[1] = __reduce_or_sync(kFull, m[1]);
                }
                return m[0] | static_cast<uint64_t>(m[1]) << 32;
            };
            auto is_read = [&](const UnitView &v, int t) {   // some row of the unit reads a position of block [t, t + 16)
                for (int i = 0; i < v.n_pos; ++i) {
                    const Range r = row_view(tp, v.pos0 + i).r;
                    if ((t < r.hi && t + kBS > r.lo && r.hi > r.lo) || (t < r.e && t + kBS > r.d && r.e > r.d)) return true;
                }
                return false;
            };
            auto table = [&](const Segment &s) { return p.bt + (p.lens ? static_cast<int64_t>(s.unit) * p.bt_stride : 0); };
            // table entry of this lane's block of the segment's tile k (-1: none)
            auto entry = [&](const Segment &s, const UnitView &v, int k) -> int32_t {
                const int vb = k * kMtBlocks + bl;
                return k < s.k1 && vb < v.br.n ? __ldg(table(s) + v.br.at(vb)) : -1;
            };
            auto valid = [&](int32_t e) { return e >= 0 && static_cast<int64_t>(e) < p.N; };
            if constexpr (!C::QUANT) {
                const bool box = lane < kMtBlocks * C::BANDS;
                int prev_slot = -1, prev_unit = -1, prev_tile = 0;
                uint32_t prev_mask = 0, prev_parity = 0;
                UnitView v{}, pv{};
                // values: once the previous tile has landed, zero the rows that nothing reads, then pass it on
                auto finish = [&]() -> bool {
                    if (prev_slot < 0) return true;
                    if (!wait(vfull(prev_slot), prev_parity)) return false;
                    if (!is_clean(pv, prev_tile, prev_mask)) {
                        const uint32_t st = sbase + C::V + prev_slot * C::STAGE;
                        const uint64_t used = used_rows(pv, prev_tile, prev_mask);
                        for (int k = lane; k < kMtKeys; k += 32)
                            if (!(used >> k & 1u))
#pragma unroll
                                for (int c = 0; c < 8 * C::BANDS; ++c)
                                    sts128_zero(st + (c >> 3) * C::KBAND + sw128(k, c & 7));
                        fence_proxy_async_smem();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(vready(prev_slot));
                    prev_slot = -1;
                    return true;
                };
                for (Segment s = walk.next(); go && s.ok; s = walk.next()) {
                    v = unit_of(tp, s, lane);
                    int32_t e_next = entry(s, v, s.k0);
                    for (int k = s.k0; k < s.k1; ++k, ++kt) {
                        const int slot = kt % R;
                        const int32_t e = e_next;
                        e_next = entry(s, v, k + 1);
                        if (kt >= R) {
                            const uint32_t fb = values ? vfree(slot) : kfree(slot), fp = (kt / R - 1) & 1;
                            // while the slot is in use, pass the previous value tile on first
                            if (values && !__any_sync(kFull, lane == 0 && mbar_test_wait(fb, fp))) go = finish();
                            go = go && wait(fb, fp);
                            if (!go) break;
                        }
                        const int vb = k * kMtBlocks + bl;
                        const bool have = vb < v.br.n, ok = have && valid(e);
                        if (!values && band == 0 && have && !ok && is_read(v, v.br.at(vb) * kBS)) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
                        const uint32_t mask = __ballot_sync(kFull, ok && lane < kMtBlocks);
                        if (!values && lane == 0) mask_sh[kt & 15] = mask;   // published by the arrive below
                        const uint32_t full = values ? vfull(slot) : kfull(slot);
                        if (p.stall_loads) {   // the test hook withholds every load
                        } else if (mask == 0u) {
                            if (lane == 0) mbar_arrive(full);
                        } else if (lane == 0) {
                            mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(mask)) * C::BANDS * (kBS * 128u));
                        }
                        __syncwarp();
                        if (box && ok && !p.stall_loads) {
                            const int32_t y = static_cast<int32_t>(((row_layer + e) * p.H_KV + s.head) * (2 * kBS)) + (values ? kBS : 0);
                            tma_load_2d(sbase + (values ? C::V : C::K) + slot * C::STAGE + band * C::KBAND + bl * (kBS * 128), &tmap,
                                        full, band * 64, y);
                        }
                        if (values) {
                            go = finish();
                            if (!go) break;
                            prev_slot = slot;
                            prev_parity = (kt / R) & 1;
                            prev_mask = mask;
                            prev_tile = k;
                            if (prev_unit != s.unit) {
                                pv = v;
                                prev_unit = s.unit;
                            }
                        }
                    }
                }
                if (values && go) go = finish();
                // before the CTA ends: every copy issued has landed (immediate unless a wait expired)
                if (!p.stall_loads)
                    for (uint32_t t = kt >= R ? kt - R : 0; t < kt; ++t)
                        (void)mbar_wait_bounded(values ? vfull(t % R) : kfull(t % R), (t / R) & 1, 100000000ull);
            } else {
                if (warp == 8) {   // the codes
                    for (Segment s = walk.next(); go && s.ok; s = walk.next()) {
                        const UnitView v = unit_of(tp, s, lane);
                        int32_t e_next = entry(s, v, s.k0);
                        for (int k = s.k0; k < s.k1; ++k, ++kt) {
                            const int slot = kt % R;
                            const int32_t e = e_next;
                            e_next = entry(s, v, k + 1);
                            if (kt >= R && !wait(cfree(slot), (kt / R - 1) & 1)) {
                                go = false;
                                break;
                            }
                            const int vb = k * kMtBlocks + bl;
                            const bool have = vb < v.br.n, ok = have && valid(e);
                            if (band == 0 && have && !ok && is_read(v, v.br.at(vb) * kBS)) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
                            const uint32_t mask = __ballot_sync(kFull, ok && lane < kMtBlocks);
                            if (lane == 0) mask_sh[kt & 15] = mask;   // published by the arrive below
                            if (p.stall_loads) {   // the test hook withholds every load
                            } else if (lane == 0) {
                                if (mask == 0u) mbar_arrive(cfull(slot));
                                else mbar_arrive_expect_tx(cfull(slot), static_cast<uint32_t>(__popc(mask)) * C::BLOCK);
                            }
                            __syncwarp();
                            if (lane < kMtBlocks && ok && !p.stall_loads)
                                tma_load_2d(sbase + C::C + slot * C::RAW + bl * C::BLOCK, &tmap, cfull(slot), 0,
                                            static_cast<int32_t>(((row_layer + e) * p.H_KV + s.head) * DecodeCfg<D, KIND>::BOX_ROWS));
                        }
                    }
                    // before the CTA ends: every copy issued has landed (immediate unless a wait expired)
                    if (!p.stall_loads)
                        for (uint32_t t = kt >= R ? kt - R : 0; t < kt; ++t)
                            (void)mbar_wait_bounded(cfull(t % R), (t / R) & 1, 100000000ull);
                } else if (warp >= 12) {
                    const int half = warp & 1;
                    for (Segment s = walk.next(); go && s.ok; s = walk.next()) {
                        const UnitView v = unit_of(tp, s, lane);
                        for (int k = s.k0; k < s.k1; ++k, ++kt) {
                            const int slot = kt % R;
                            go = wait(cfull(slot), (kt / R) & 1);
                            if (kt >= R) go = go && wait(values ? vfree(slot) : kfree(slot), (kt / R - 1) & 1);
                            if (!go) break;
                            const uint32_t codes = sbase + C::C + slot * C::RAW;
                            if (!values) {
                                widen_half<D, KIND, false>(codes, sbase + C::K + slot * C::STAGE, half, lane, [](int) { return true; });
                            } else {
                                const uint32_t mask = mask_sh[kt & 15];
                                if (is_clean(v, k, mask))
                                    widen_half<D, KIND, true>(codes, sbase + C::V + slot * C::STAGE, half, lane, [](int) { return true; });
                                else {
                                    const uint64_t used = used_rows(v, k, mask);
                                    widen_half<D, KIND, true>(codes, sbase + C::V + slot * C::STAGE, half, lane,
                                                              [=](int row) { return (used >> row & 1u) != 0; });
                                }
                            }
                            fence_proxy_async_smem();   // written here, read by the MMA; the codes' slot is rewritten by TMA
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(values ? vready(slot) : kfull(slot));
                                mbar_arrive(cfree(slot));
                            }
                        }
                    }
                }
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------- MMA issuer of query tile x
            const int x = warp - 10;
            constexpr uint32_t idesc_qk = tc_idesc_f16(128, kMtKeys, !C::QUANT, false, false);
            constexpr uint32_t idesc_pv = tc_idesc_f16(128, D, !C::QUANT, false, true);
            const uint64_t desc_q = tc_smem_desc(sbase + C::Q + x * C::QTILE, 16, 1024, kSwizzle128B);
            const uint32_t tm_s = tmem + 128 * x, tm_o = tmem + 256 + 128 * x;
            uint32_t kt = 0, it = 0, seg = 0;   // key tiles, this chain's steps and its segments so far
            // scores against the CTA's key tile `tile`, into score buffer b
            auto scores = [&](uint32_t tile, uint32_t b) -> bool {
                const uint32_t slot = tile % R;
                if (!wait(kfull(slot), (tile / R) & 1)) return false;
                tc_fence_after();
                const uint64_t b0 = tc_smem_desc(sbase + C::K + slot * C::STAGE, 16, 1024, kSwizzle128B);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)   // 16 channels (32 bytes) per MMA, 4 per 128-byte band
                    tc_mma_f16_warp(tm_s + b * kMtKeys, tc_desc_advance(desc_q, (kk >> 2) * C::QBAND + (kk & 3) * 32),
                                    tc_desc_advance(b0, (kk >> 2) * C::KBAND + (kk & 3) * 32), idesc_qk, kk > 0 ? 1u : 0u);
                tc_commit_warp(sfull(x, b));
                tc_commit_warp(kfree(slot));
                return true;
            };
            bool go = true;
            for (Segment s = walk.next(); go && s.ok; s = walk.next()) {
                if (tp.whole) (void)unit_of(tp, s, lane);
                const uint32_t n = s.k1 - s.k0;
                // the second tile may hold no position: it only lets the key and value tiles go
                if (!tp.split && s.unit * 2 * ppt + x * ppt >= p.n_pos) {
                    for (uint32_t k = 0; go && k < n; ++k, ++kt) {
                        const int slot = kt % R;
                        const uint32_t par = (kt / R) & 1;
                        go = wait(kfull(slot), par);
                        if (go && lane == 0) mbar_arrive(kfree(slot));
                        go = go && wait(vready(slot), par);
                        if (go && lane == 0) mbar_arrive(vfree(slot));
                        __syncwarp();
                    }
                    continue;
                }
                if (!wait(qfull(x), seg & 1)) break;
                ++seg;
                tc_fence_after();
                // few rows: chain x takes the segment's tiles x, x + 2, ...
                const uint32_t steps = tp.split ? (n + 1 - x) / 2 : n, stride = tp.split ? 2 : 1, t0 = kt + (tp.split ? x : 0);
                if (steps > 0) go = scores(t0, it & 1);
                if (go && steps > 1) go = scores(t0 + stride, (it + 1) & 1);
                for (uint32_t i = 0; go && i < steps; ++i, ++it) {
                    const uint32_t tile = t0 + i * stride, slot = tile % R, b = it & 1, par = (it >> 1) & 1;
                    if (!wait(vready(slot), (tile / R) & 1) || !wait(pfull(x, b), par)) {
                        go = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t v0 = tc_smem_desc(sbase + C::V + slot * C::STAGE, C::KBAND, 1024, kSwizzle128B);
#pragma unroll
                    for (int kk = 0; kk < kMtKeys / 16; ++kk)   // 16 keys: 8 columns of P, 2048 bytes of value rows
                        tc_mma_f16_tmem_a_warp(tm_o, tm_s + b * kMtKeys + kk * 8, tc_desc_advance(v0, kk * 2048), idesc_pv,
                                               (i > 0 || kk > 0) ? 1u : 0u);
                    tc_commit_warp(vfree(slot));
                    tc_commit_warp(pvdone(x, b));
                    // the scores two steps on go over these weights, once the product has read them
                    if (i + 2 < steps) go = wait(pvdone(x, b), par) && scores(tile + 2 * stride, b);
                }
                kt += n;
            }
        }
    } else {
        // ------------------------------------------------------------ softmax of query tile x
        if constexpr (C::QUANT) asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t ts = tmem + 128 * x + lane_off, to = tmem + 256 + 128 * x + lane_off;
        const float ref = 0.5f * mp.cap_out;
        auto bar_both = [] { asm volatile("bar.sync 6, 256;" ::: "memory"); };   // both chains' threads
        uint32_t it = 0, kt = 0;   // this query tile's steps, key tiles so far
        int piece = 0;             // segments so far
        int4 cut = make_int4(0, 0, 0, 0);
        for (Segment s = walk.next(); s.ok; s = walk.next(), ++piece) {
            const uint32_t kt0 = kt;
            const UnitView v = unit_of(tp, s, lane);
            kt += s.k1 - s.k0;
            const int c0 = v.pos0 + (tp.split ? 0 : x * ppt);
            const bool mine = c0 < p.n_pos;
            const bool join = tp.split && s.all();   // the two chains' sums meet here, not in the merge
            // up to 64 rows in a few-row call: chain 1's sit in the tile's upper half, so that the warps that have
            // work to do are on different schedulers
            const int ro = tp.split && !join && x == 1 && min(ppt, p.n_pos - c0) * g <= 64 ? 64 : 0;
            const int rq = row - ro;            // row of the query tile
            const int c = c0 + max(rq, 0) / g;   // its chunk position
            const bool real = rq >= 0 && rq < ppt * g && c < p.n_pos;
            const size_t orow = static_cast<size_t>(c) * p.H_Q + s.head * g + max(rq, 0) % g;
            if (!mine) continue;   // the same for the whole CTA
            // ---- queries into shared memory (zero where there is none), every load in flight at once
            asm volatile("bar.sync %0, 128;" ::"r"(4 + x) : "memory");   // the last segment's rows have left it
            {
                constexpr int N = D / 8, STEP = 128 / N;   // 16-byte chunks of a row; rows between a thread's chunks
                const int dc = STEP / g, dh = STEP % g, ch = row % N;
                int r = row / N, cp = c0 + r / g, hh = r % g;
                uint4 q[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    q[i] = make_uint4(0u, 0u, 0u, 0u);
                    if (r < ppt * g && cp < p.n_pos)
                        q[i] = __ldg(reinterpret_cast<const uint4 *>(p.q + (static_cast<size_t>(cp) * p.H_Q + s.head * g + hh) * D) + ch);
                    r += STEP;
                    cp += dc;
                    hh += dh;
                    if (hh >= g) {
                        hh -= g;
                        ++cp;
                    }
                }
                if constexpr (C::QUANT) {   // times the key scales, rounded to f16, in the widened keys' order
                    float sk[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) sk[j] = __ldg(p.s_k + static_cast<size_t>(s.head) * D + 8 * ch + j);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
                        float f[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            f[widened_column<KIND>(j)] = ((j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1])) * sk[j];
                        q[i] = make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i)
                    sts128(sbase + C::Q + x * C::QTILE + (ch >> 3) * C::QBAND + sw128((row / N + STEP * i + ro) & 127, ch & 7), q[i]);
            }
            fence_proxy_async_smem();
            tc_fence_before();   // this thread's reads of the last segment's outputs
            mbar_arrive(qfull(x));
            Range r{0, 0, 0, 0};
            float slope = 0.f;
            int pos = 0;
            if (real) {
                const RowView rv = row_view(tp, c);
                r = rv.r;
                pos = rv.pos;
                if (mp.alibi) slope = __ldg(mp.alibi + s.head * g + rq % g) * 1.4426950408889634f;
            }
            // every real row of the warp reads [flo, fhi) and [fd, fe)
            const int flo = __reduce_max_sync(kFull, real ? r.lo : 0), fhi = __reduce_min_sync(kFull, real ? r.hi : 0x7FFFFFFF);
            const int fd = __reduce_max_sync(kFull, real ? r.d : 0), fe = __reduce_min_sync(kFull, real ? r.e : 0x7FFFFFFF);
            const bool any_real = __any_sync(kFull, real);
            float m = FIXED ? ref : -INFINITY, l = 0.f;
            float dl = 0.f;   // FIXED: what rounding the weights added to their sum, in the tiles not read whole
            bool go = true;
            // every real row of the warp is at this position or past it
            const int from = __reduce_min_sync(kFull, real ? pos : 0x7FFFFFFF);
            const int steps = tp.split ? (s.k1 - s.k0 + 1 - x) / 2 : s.k1 - s.k0;
            for (int i = 0; i < steps; ++i, ++it) {
                const int b = it & 1, tile = tp.split ? 2 * i + x : i;
                if (!wait(sfull(x, b), (it >> 1) & 1)) {
                    go = false;
                    break;
                }
                tc_fence_after();
                if (!any_real) {   // rows past the chunk: their weights stay in their own lanes and are never read
                    mbar_arrive(pfull(x, b));
                    continue;
                }
                const uint32_t tsb = ts + b * kMtKeys;
                uint32_t r0[32], r1[32];
                tmem_ld32(tsb, r0);
                tmem_ld32(tsb + 32, r1);
                const int first = (s.k0 + tile) * kMtBlocks;   // the tile's first virtual block
                const bool one_run = first + kMtBlocks <= v.br.n && (first + kMtBlocks <= v.br.n0 || first >= v.br.n0);
                const int t0 = v.br.at(first) * kBS;
                const uint32_t loaded = mask_sh[(kt0 + tile) & 15];
                const bool full = one_run && loaded == (1u << kMtBlocks) - 1u &&
                                  ((t0 >= flo && t0 + kMtKeys <= fhi) || (t0 >= fd && t0 + kMtKeys <= fe));
                // bit j of a 16-key block's mask: this row reads the block's key j
                auto block_mask = [&](int b) -> uint32_t {
                    const int vb = first + b;
                    if (vb >= v.br.n || !(loaded >> b & 1u)) return 0u;
                    const int t = v.br.at(vb) * kBS;
                    auto below = [&](int end) -> uint32_t {   // keys of the block before position `end`
                        return end <= t ? 0u : (end >= t + kBS ? 0xFFFFu : (1u << (end - t)) - 1u);
                    };
                    return (below(r.hi) & ~below(r.lo)) | (below(r.e) & ~below(r.d));
                };
                uint32_t seen0 = 0xFFFFFFFFu, seen1 = 0xFFFFFFFFu;
                if (!full) {
                    seen0 = block_mask(0) | (block_mask(1) << 16);
                    seen1 = block_mask(2) | (block_mask(3) << 16);
                }
                tmem_ld_wait(r0);
                tmem_ld_wait(r1);
                f32x2 ls[4] = {f32x2_of(0.f, 0.f), f32x2_of(0.f, 0.f), f32x2_of(0.f, 0.f), f32x2_of(0.f, 0.f)};
                if constexpr (CAPPED) {
                    const f32x2 in = f32x2_of(mp.cap_in, mp.cap_in);
                    const f32x2 out2 = f32x2_of(-2.f * mp.cap_out, -2.f * mp.cap_out);
                    // Quantised pools: weights against the reference so far, which moves when a score turns out to
                    // pass it by more than the slack; the weights are then taken again (in a row's first tile, and
                    // seldom after).  (The tile's maximum first, then the weights: 833 us against 710 at 2048
                    // positions over 18 432, e4m3.)
                    for (;;) {
                        const float mref = m == -INFINITY ? 0.f : m, top = mp.cap_out - mref;
                        const f32x2 top2 = f32x2_of(top, top);
                        float best0 = -INFINITY, best1 = -INFINITY;
                        auto weigh4 = [&](const uint32_t *s, float (&x)[4], float (&w)[4]) {
                            f32x2 x01, x23;   // x - the reference
                            capped4(f32x2_of(__uint_as_float(s[0]), __uint_as_float(s[1])),
                                    f32x2_of(__uint_as_float(s[2]), __uint_as_float(s[3])), in, out2, top2, x01, x23);
                            x[0] = lo2(x01);
                            x[1] = hi2(x01);
                            x[2] = lo2(x23);
                            x[3] = hi2(x23);
#pragma unroll
                            for (int k = 0; k < 4; ++k) w[k] = fast_exp2(x[k]);
                        };
                        auto pack = [](float a, float b) { return C::QUANT ? pack_f16(a, b) : pack_bf16(a, b); };
#pragma unroll
                        for (int k = 0; k < 4; ++k) ls[k] = f32x2_of(0.f, 0.f);
                        if constexpr (MODE == kMtCappedBrief) {
                            uint32_t pk[32];
                            if (!full) {   // a hidden key's score may be anything, and would reach its group's reciprocal
#pragma unroll
                                for (int c = 0; c < 32; ++c) {
                                    r0[c] = seen0 >> c & 1u ? r0[c] : 0u;
                                    r1[c] = seen1 >> c & 1u ? r1[c] : 0u;
                                }
                            }
#pragma unroll
                            for (int c = 0; c < 64; c += 4) {
                                float x[4], w[4];
                                weigh4(c < 32 ? r0 + c : r1 + (c - 32), x, w);
                                if (!full) {
                                    const uint32_t seen = (c < 32 ? seen0 : seen1) >> (c & 31);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) w[k] = seen >> k & 1u ? w[k] : 0.f;
                                }
                                ls[(c >> 2) & 1] = add2(ls[(c >> 2) & 1], f32x2_of(w[0], w[1]));
                                ls[2 + ((c >> 2) & 1)] = add2(ls[2 + ((c >> 2) & 1)], f32x2_of(w[2], w[3]));
                                pk[c / 2] = pack(w[0], w[1]);
                                pk[c / 2 + 1] = pack(w[2], w[3]);
                            }
                            if (!full) {
                                f32x2 rounded = f32x2_of(0.f, 0.f);
#pragma unroll
                                for (int c = 0; c < 32; ++c) rounded = add2(rounded, f32x2_of(bf16_lo(pk[c]), bf16_hi(pk[c])));
                                const f32x2 sum = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
                                dl += (lo2(rounded) + hi2(rounded)) - (lo2(sum) + hi2(sum));
                            }
                            tmem_st32(tsb, pk);   // over the first half of the step's scores
                            break;
                        }
                        // Code of their own for the tiles read whole: with the others' selects between them, a score
                        // and the weight before it were not interleaved (2048 positions over 18 432: 592 against 571 us).
                        if (full) {
                            uint32_t pk[32];
#pragma unroll
                            for (int c = 0; c < 64; c += 4) {
                                float x[4], w[4];
                                weigh4(c < 32 ? r0 + c : r1 + (c - 32), x, w);
                                if constexpr (C::QUANT) {
                                    best0 = max3f(best0, x[0], x[1]);
                                    best1 = max3f(best1, x[2], x[3]);
                                }
                                ls[(c >> 2) & 1] = add2(ls[(c >> 2) & 1], f32x2_of(w[0], w[1]));
                                ls[2 + ((c >> 2) & 1)] = add2(ls[2 + ((c >> 2) & 1)], f32x2_of(w[2], w[3]));
                                pk[c / 2] = pack(w[0], w[1]);
                                pk[c / 2 + 1] = pack(w[2], w[3]);
                            }
                            tmem_st32(tsb, pk);   // over the first half of the step's scores
                        } else {
                            // Thirty-two scores at a time, which keeps the code small: a few tiles come this way, and
                            // with straight code for all 64 a 600-position chunk over 1 800 took 45.7 us against 43.7.
#pragma unroll 1
                            for (int half = 0; half < 2; ++half) {
                                const uint32_t seen = half ? seen1 : seen0;
                                uint32_t pk[16];
                                // a hidden key's score may be anything, and would reach its group's reciprocal
#pragma unroll
                                for (int c = 0; c < 32; ++c) r0[c] = seen >> c & 1u ? r0[c] : 0u;
#pragma unroll
                                for (int c = 0; c < 32; c += 4) {
                                    float x[4], w[4];
                                    weigh4(r0 + c, x, w);
#pragma unroll
                                    for (int k = 0; k < 4; ++k) {
                                        w[k] = seen >> (c + k) & 1u ? w[k] : 0.f;
                                        if constexpr (C::QUANT) best0 = fmaxf(best0, seen >> (c + k) & 1u ? x[k] : -INFINITY);
                                    }
                                    ls[0] = add2(ls[0], f32x2_of(w[0], w[1]));
                                    ls[1] = add2(ls[1], f32x2_of(w[2], w[3]));
                                    pk[c / 2] = pack(w[0], w[1]);
                                    pk[c / 2 + 1] = pack(w[2], w[3]);
                                    if constexpr (!C::QUANT)
                                        dl += ((bf16_lo(pk[c / 2]) - w[0]) + (bf16_hi(pk[c / 2]) - w[1])) +
                                              ((bf16_lo(pk[c / 2 + 1]) - w[2]) + (bf16_hi(pk[c / 2 + 1]) - w[3]));
                                }
                                tmem_st16(tsb + 16 * half, pk);
#pragma unroll
                                for (int c = 0; c < 32; ++c) {   // the other half; after two turns they are back
                                    const uint32_t t = r0[c];
                                    r0[c] = r1[c];
                                    r1[c] = t;
                                }
                            }
                        }
                        if constexpr (!C::QUANT) break;
                        const float bm = fmaxf(best0, best1) + mref;
                        const bool move = bm > m + C::SLACK;   // false while nothing has been read
                        if (!__any_sync(kFull, move)) break;
                        float alpha = 1.f;
                        if (move) {
                            alpha = fast_exp2(m - bm);
                            m = bm;
                            l *= alpha;
                        }
                        // the warp rescales its rows of O together, once the previous product is in them
                        if (i > 0) {
                            go = wait(pvdone(x, b ^ 1), ((it - 1) >> 1) & 1);
                            if (!go) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int part = 0; part < D / 16; ++part) tmem_scale16(to + part * 16, alpha);
                        }
                    }
                    if (!go) break;
                } else if constexpr (MODE == kMtPlain) {
                    // Against the reference so far, and again where a score passes it by more than the slack (in a
                    // row's first tile, and seldom after): the maximum first took 520 us against 501.
                    for (;;) {
                        const float neg = m == -INFINITY ? 0.f : -m;
                        const f32x2 sc2 = f32x2_of(p.scale_log2, p.scale_log2), neg2 = f32x2_of(neg, neg);
                        float b0 = -INFINITY, b1 = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 4; ++k) ls[k] = f32x2_of(0.f, 0.f);
                        uint32_t pk[32];
                        if (!full) {
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                r0[c] = seen0 >> c & 1u ? r0[c] : 0xFF800000u;
                                r1[c] = seen1 >> c & 1u ? r1[c] : 0xFF800000u;
                            }
                        }
#pragma unroll
                        for (int c = 0; c < 64; c += 4) {
                            const uint32_t *sr = c < 32 ? r0 + c : r1 + (c - 32);
                            const float s0 = __uint_as_float(sr[0]), s1 = __uint_as_float(sr[1]), s2 = __uint_as_float(sr[2]), s3 = __uint_as_float(sr[3]);
                            b0 = max3f(b0, s0, s1);
                            b1 = max3f(b1, s2, s3);
                            const f32x2 e01 = fma2(f32x2_of(s0, s1), sc2, neg2), e23 = fma2(f32x2_of(s2, s3), sc2, neg2);
                            const float w0 = fast_exp2(lo2(e01)), w1 = fast_exp2(hi2(e01)), w2 = fast_exp2(lo2(e23)), w3 = fast_exp2(hi2(e23));
                            ls[(c >> 2) & 1] = add2(ls[(c >> 2) & 1], f32x2_of(w0, w1));
                            ls[2 + ((c >> 2) & 1)] = add2(ls[2 + ((c >> 2) & 1)], f32x2_of(w2, w3));
                            pk[c / 2] = C::QUANT ? pack_f16(w0, w1) : pack_bf16(w0, w1);
                            pk[c / 2 + 1] = C::QUANT ? pack_f16(w2, w3) : pack_bf16(w2, w3);
                        }
                        tmem_st32(tsb, pk);   // over the first half of the step's scores
                        const float bm = fmaxf(b0, b1) * p.scale_log2;
                        const bool move = bm > m + C::SLACK;   // false while nothing has been read
                        if (!__any_sync(kFull, move)) break;
                        float alpha = 1.f;
                        if (move) {
                            alpha = fast_exp2(m - bm);
                            m = bm;
                            l *= alpha;
                        }
                        // the warp rescales its rows of O together, once the previous product is in them
                        if (i > 0) {
                            go = wait(pvdone(x, b ^ 1), ((it - 1) >> 1) & 1);
                            if (!go) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int part = 0; part < D / 16; ++part) tmem_scale16(to + part * 16, alpha);
                        }
                    }
                    if (!go) break;
                } else {
                    uint32_t pk[32];
                    float sv[64];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        sv[c] = __uint_as_float(r0[c]);
                        sv[32 + c] = __uint_as_float(r1[c]);
                    }
                    if (mp.capped) {
                        if (!full) {   // a hidden key's score may be anything, and would reach its group's reciprocal
#pragma unroll
                            for (int c = 0; c < 32; ++c) {
                                sv[c] = seen0 >> c & 1u ? sv[c] : 0.f;
                                sv[32 + c] = seen1 >> c & 1u ? sv[32 + c] : 0.f;
                            }
                        }
                        const f32x2 in = f32x2_of(mp.cap_in, mp.cap_in);
                        const f32x2 out2 = f32x2_of(-2.f * mp.cap_out, -2.f * mp.cap_out), cap2 = f32x2_of(mp.cap_out, mp.cap_out);
#pragma unroll
                        for (int c = 0; c < 64; c += 4) {
                            f32x2 x01, x23;
                            capped4(f32x2_of(sv[c], sv[c + 1]), f32x2_of(sv[c + 2], sv[c + 3]), in, out2, cap2, x01, x23);
                            sv[c] = lo2(x01);
                            sv[c + 1] = hi2(x01);
                            sv[c + 2] = lo2(x23);
                            sv[c + 3] = hi2(x23);
                        }
                    }
                    const float mul = mp.capped ? 1.f : p.scale_log2;   // into log2 units
                    if (mp.alibi && one_run && from >= t0 + kMtKeys - 1) {
                        // keys before the row's position: the bias is slope (t - p), a line.  Eight chains of pairs, four
                        // additions each; with every key's distance on its own 2048 over 18 432, slopes 2^(-8 i / H), took
                        // 708 us against 681 (e4m3 826 against 781).
                        f32x2 line[8];
                        const float at = slope * static_cast<float>(t0 - pos);
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            line[c] = f32x2_of(fmaf(slope, static_cast<float>(2 * c), at), fmaf(slope, static_cast<float>(2 * c + 1), at));
                        const f32x2 on = f32x2_of(16.f * slope, 16.f * slope), mul2_ = f32x2_of(mul, mul);
#pragma unroll
                        for (int c = 0; c < 64; c += 2) {
                            const f32x2 y = fma2(f32x2_of(sv[c], sv[c + 1]), mul2_, line[(c / 2) & 7]);
                            line[(c / 2) & 7] = add2(line[(c / 2) & 7], on);
                            sv[c] = lo2(y);
                            sv[c + 1] = hi2(y);
                        }
                    } else if (C::QUANT || mp.alibi) {   // quantised pools: always with a bias here
#pragma unroll
                        for (int b2 = 0; b2 < kMtBlocks; ++b2) {
                            const int vb = min(first + b2, max(v.br.n - 1, 0));
                            const float away = static_cast<float>(pos - v.br.at(vb) * kBS);
#pragma unroll
                            for (int c = 0; c < kBS; ++c)
                                sv[kBS * b2 + c] = fmaf(sv[kBS * b2 + c], mul, -slope * fabsf(away - static_cast<float>(c)));
                        }
                    }
                    if (!full) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) {
                            sv[c] = seen0 >> c & 1u ? sv[c] : -INFINITY;
                            sv[32 + c] = seen1 >> c & 1u ? sv[32 + c] : -INFINITY;
                        }
                    }
                    float b0 = sv[0], b1 = sv[1], b2 = sv[2], b3 = sv[3];   // four chains of 3-input maxima
#pragma unroll
                    for (int c = 4; c < 60; c += 8) {
                        b0 = max3f(b0, sv[c], sv[c + 1]);
                        b1 = max3f(b1, sv[c + 2], sv[c + 3]);
                        b2 = max3f(b2, sv[c + 4], sv[c + 5]);
                        b3 = max3f(b3, sv[c + 6], sv[c + 7]);
                    }
                    b0 = max3f(b0, sv[60], sv[61]);
                    b1 = max3f(b1, sv[62], sv[63]);
                    const float bm = max3f(b0, b1, fmaxf(b2, b3));
                    const bool move = bm > m + C::SLACK;              // false while nothing has been read
                    float alpha = 1.f;
                    if (move) {
                        alpha = fast_exp2(m - bm);
                        m = bm;
                        l *= alpha;
                    }
                    // the warp rescales its rows of O together, once the previous product is in them
                    if (i > 0 && __any_sync(kFull, move && alpha != 1.f)) {
                        if (!wait(pvdone(x, b ^ 1), ((it - 1) >> 1) & 1)) {
                            go = false;
                            break;
                        }
                        tc_fence_after();
#pragma unroll 1
                        for (int part = 0; part < D / 16; ++part) tmem_scale16(to + part * 16, alpha);
                    }
                    const float neg = m == -INFINITY ? 0.f : -m;
                    const f32x2 neg2 = f32x2_of(neg, neg);
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        const f32x2 e = add2(f32x2_of(sv[c], sv[c + 1]), neg2);
                        const float w0 = fast_exp2(lo2(e)), w1 = fast_exp2(hi2(e));
                        ls[(c / 2) & 3] = add2(ls[(c / 2) & 3], f32x2_of(w0, w1));
                        pk[c / 2] = C::QUANT ? pack_f16(w0, w1) : pack_bf16(w0, w1);
                    }
                    tmem_st32(tsb, pk);   // over the first half of the step's scores
                }
                const f32x2 lt = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
                l += lo2(lt) + hi2(lt);
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(pfull(x, b));
            }
            if (go && steps > 0) go = wait(pvdone(x, (it - 1) & 1), ((it - 1) >> 1) & 1);   // the segment's last product
            // every thread of the query tile takes this vote once per segment, so the barriers below meet; of both
            // tiles where the chains share rows: the next segment may be one in which they meet
            if (!tile_all(go, tp.split ? 6 : 4 + x, tp.split ? 256 : 128)) {
                timed_out = true;
                break;
            }
            tc_fence_after();

            // ---- epilogue: the unit's rows, or a piece of them for the merge (rows [128 x, 128 x + 128) of a slot)
            const bool done = s.all() && !tp.split;
            if (!any_real && !join) continue;
            const int64_t slot = piece_slot(blockIdx.x, piece);
            if (tid == 0 && !done && !tp.whole && s.k0 == 0) {
                const int64_t end = static_cast<int64_t>(s.head) * walk.per_head + prefix[s.unit + 1];
                cut = make_int4(s.head, s.unit, cta_of(end - 1, walk.W, walk.G) - static_cast<int>(blockIdx.x) + 1, static_cast<int>(slot));
            }
            const int prow = x * 128 + rq;
            float inv = l == 0.f ? 0.f : 1.f / (l + dl), other = 0.f;
            if (join) {   // chain 1 hands over m, l and the sum that its outputs go with; chain 0 weighs both
                float4 *meet = reinterpret_cast<float4 *>(smem + C::MEET_SUMS);
                if (x == 1) meet[row] = make_float4(m, l, l + dl, 0.f);
                bar_both();
                if (x == 0) {
                    const float4 o = meet[row];
                    const float M = fmaxf(l != 0.f ? m : -INFINITY, o.y != 0.f ? o.x : -INFINITY);
                    const float e0 = l != 0.f ? fast_exp2(m - M) : 0.f, e1 = o.y != 0.f ? fast_exp2(o.x - M) : 0.f;
                    const float sum = e0 * (l + dl) + e1 * o.z;
                    l = e0 * l + e1 * o.y;
                    m = M;
                    const float r = l == 0.f ? 0.f : 1.f / sum;
                    inv = e0 * r;
                    other = e1 * r;
                }
            }
            const bool leaves = done || (join && x == 0);   // this thread's row leaves finished
            const float even = FIXED && l != 0.f ? l * inv : 1.f;   // a piece's outputs go with its l
            // finished rows go through the warp's quarter of the tile's query memory (its products are done;
            // 16-byte chunk c of row r at c ^ (r mod 8)), so that whole rows leave: a lane's row written
            // straight to global memory measured 2.8 us a unit against 1.3 us
            const uint32_t stage = sbase + C::Q + x * C::QTILE + (warp & 3) * (C::QTILE / 4);
            auto load_part = [&](int part, uint32_t (&o)[32]) {   // 32 channels of this row's sums
                tmem_ld32(to + part * 32, o);
                tmem_ld_wait(o);
                if constexpr (C::QUANT) {   // the channels' order, and the value scales
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) w[c] = o[(c & ~7) + widened_column<KIND>(c & 7)];
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const float4 sv = __ldg(reinterpret_cast<const float4 *>(p.s_v + static_cast<size_t>(s.head) * D + part * 32) + c);
                        o[4 * c] = __float_as_uint(__uint_as_float(w[4 * c]) * sv.x);
                        o[4 * c + 1] = __float_as_uint(__uint_as_float(w[4 * c + 1]) * sv.y);
                        o[4 * c + 2] = __float_as_uint(__uint_as_float(w[4 * c + 2]) * sv.z);
                        o[4 * c + 3] = __float_as_uint(__uint_as_float(w[4 * c + 3]) * sv.w);
                    }
                }
            };
            auto stage_part = [&](int part, const uint32_t (&o)[32], float by) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t w[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        w[u] = l == 0.f ? 0u : pack_bf16(__uint_as_float(o[8 * c + 2 * u]) * by,
                                                         __uint_as_float(o[8 * c + 2 * u + 1]) * by);
                    sts128(stage + lane * (D * 2) + (((part * 4 + c) ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
                }
            };
            if (join) {   // 32 channels at a time through two buffers: one barrier each
#pragma unroll 1
                for (int part = 0; part < D / 32; ++part) {
                    uint32_t o[32];
                    load_part(part, o);
                    const uint32_t at = sbase + C::MEET + (part & 1) * C::MEET_PART + row * 16;
                    if (x == 1) {
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            sts128(at + c * 2048, make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]));
                    }
                    bar_both();
                    if (x == 1) continue;
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint4 e = lds128(at + c * 2048);
                        const uint32_t ew[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {   // a chain that read nothing left nothing to add
                            const float a = inv != 0.f ? __uint_as_float(o[4 * c + k]) * inv : 0.f;
                            o[4 * c + k] = __float_as_uint(other != 0.f ? fmaf(__uint_as_float(ew[k]), other, a) : a);
                        }
                    }
                    stage_part(part, o, 1.f);
                }
                bar_both();   // chain 1's columns have been read: its next queries may go there
            } else {
#pragma unroll
                for (int part = 0; part < D / 32; ++part) {
                    uint32_t o[32];
                    load_part(part, o);
                    if (!real) continue;
                    if (done) {
                        stage_part(part, o, inv);
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(tp.part_o) +
                                      (tp.split ? (slot * 256 + prow) * (D / 4) + part * 8 : (slot * (D / 4) + part * 8) * 256 + prow);
                        const int step = tp.split ? 1 : 256;
#pragma unroll
                        for (int c = 0; c < 8; ++c)
                            dst[c * step] = make_float4(__uint_as_float(o[4 * c]) * even, __uint_as_float(o[4 * c + 1]) * even,
                                                       __uint_as_float(o[4 * c + 2]) * even, __uint_as_float(o[4 * c + 3]) * even);
                    }
                }
            }
            if (leaves) {
                __syncwarp();
                constexpr int N = D / 8, STEP = 32 / N;   // chunks of a row, rows a warp writes at once
                const int ch = lane % N;
                int r = (warp & 3) * 32 + lane / N, cp = c0 + r / g, hh = r % g;
                const int dc = STEP / g, dh = STEP % g;
#pragma unroll 4
                for (int i = 0; i < N; ++i) {
                    const int ri = lane / N + STEP * i;
                    if (r < ppt * g && cp < p.n_pos)
                        *reinterpret_cast<uint4 *>(mp.out + (static_cast<size_t>(cp) * p.H_Q + s.head * g + hh) * D + 8 * ch) =
                            lds128(stage + ri * (D * 2) + ((ch ^ (ri & 7)) << 4));
                    r += STEP;
                    cp += dc;
                    hh += dh;
                    if (hh >= g) {
                        hh -= g;
                        ++cp;
                    }
                }
            }
            if (real && leaves && p.lse) p.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
            if (real && !done && !join) tp.part_ml[slot * 256 + prow] = make_float2(m, l);
        }
        if (tid == 0 && !tp.whole && !tp.split) tp.cuts[blockIdx.x] = cut;
    }
    if (timed_out && lane == 0) atomicOr(p.err, KVC_EBIT_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds the pieces of units that CTA borders cut, in CTA order (in few-row calls: chain 0's and chain 1's of
// every CTA):  M = max m_s, L = sum 2^(m_s - M) l_s, out = sum 2^(m_s - M) o_s / L, lse = (M + log2 L) ln 2.
// Whole chunks (T = 1): grid (8, the attention kernel's CTAs), 256 threads = 32 rows x 8 groups of D / 8
// channels; a thread has its loads of a piece in flight at once.  Few-row calls (T = 8), whose rows have tens
// of pieces: grid (row groups, units, KV heads), 256 threads = 128 / D rows x D / 4 float4 columns x 8 groups of
// pieces.  A programmatic dependent of mod_tc_kernel (its CTAs are in place when that ends).  ctas: that
// kernel's grid.
template <int D, int T>
__global__ void __launch_bounds__(256) mod_tc_merge_kernel(const ModTcParams tp, const int ctas)
{
    constexpr int V = T > 1 ? 1 : D / 32;                // float4 columns per thread
    constexpr int COLS = D / 4 / V, RG = 256 / COLS / T;   // column groups, rows per CTA
    const ModParams &mp = tp.m;
    const DecodeParams &p = mp.d;
    const int g = p.g;
    const int rr = blockIdx.x * RG + threadIdx.x % RG, dg = threadIdx.x / RG % COLS, grp = threadIdx.x / (RG * COLS);
    const int tile = rr >> 7, r = rr & 127;
    const int hr = r % g, pr = tile * p.ppu + r / g;   // head of the group, position of the unit
    grid_dependency_wait();
    int unit, head, n, slot0;   // the unit's pieces: slot0 in its first CTA, then every later CTA's first slot
    if constexpr (T == 1) {
        const int4 cut = __ldcg(tp.cuts + blockIdx.y);
        head = cut.x;
        unit = cut.y;
        n = cut.z;
        slot0 = cut.w;
        if (n == 0) return;
    } else {
        unit = blockIdx.y;
        head = blockIdx.z;
        const int per_head = __ldcg(tp.prefix + tp.units), u0 = __ldcg(tp.prefix + unit), u1 = __ldcg(tp.prefix + unit + 1);
        const int64_t W = static_cast<int64_t>(p.H_KV) * per_head, G = min(static_cast<int64_t>(ctas), W);
        const int64_t at = static_cast<int64_t>(head) * per_head;
        const Pieces ps = pieces_of(at + u0, at + u1, W, G);
        if (ps.ctas == 1) return;   // finished by its CTA (the same for the whole block)
        n = ps.ctas * 2;
        slot0 = ps.slot0;
    }
    const int c = unit * unit_positions_of(tp) + pr;
    const bool real = r < p.ppu * g && c < p.n_pos;
    if (T == 1 && !real) return;
    // piece t: slot * 256 + row in it (few rows: chain t mod 2 of CTA t / 2)
    auto at = [&](int t) -> int {
        const int cta = T > 1 ? t >> 1 : t, chain = T > 1 ? t & 1 : tile;
        return (cta == 0 ? slot0 : (slot0 & ~1) + 2 * cta) * 256 + chain * 128 + r;
    };
    float M = -INFINITY, L = 0.f;
    float4 acc[V];
#pragma unroll
    for (int k = 0; k < V; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (real) {   // every group of pieces finds its own maximum; the groups meet below
#pragma unroll 8
        for (int t = grp; t < n; t += T) {
            const float2 ml = __ldcg(tp.part_ml + at(t));
            M = fmaxf(M, ml.y != 0.f ? ml.x : -INFINITY);
        }
        constexpr int U = T > 1 ? 8 : 2;
#pragma unroll U
        for (int t = grp; t < n; t += T) {
            const int i = at(t);
            const float2 ml = __ldcg(tp.part_ml + i);
            const float4 *src = reinterpret_cast<const float4 *>(tp.part_o) +
                                (T > 1 ? static_cast<size_t>(i) * (D / 4) + dg
                                       : (static_cast<size_t>(i >> 8) * (D / 4) + dg * V) * 256 + (i & 255));
            float4 o[V];
#pragma unroll
            for (int k = 0; k < V; ++k) o[k] = __ldcg(src + k * 256);
            const bool some = ml.y != 0.f;   // else the piece reads nothing for this row
            const float e = some ? fast_exp2(ml.x - M) : 0.f;
            L = fmaf(e, ml.y, L);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                acc[k].x = some ? fmaf(e, o[k].x, acc[k].x) : acc[k].x;
                acc[k].y = some ? fmaf(e, o[k].y, acc[k].y) : acc[k].y;
                acc[k].z = some ? fmaf(e, o[k].z, acc[k].z) : acc[k].z;
                acc[k].w = some ? fmaf(e, o[k].w, acc[k].w) : acc[k].w;
            }
        }
    }
    if constexpr (T > 1) {
        __shared__ float4 part[256];
        __shared__ float part_l[256], part_m[256];
        part[threadIdx.x] = acc[0];
        part_l[threadIdx.x] = L;
        part_m[threadIdx.x] = M;
        __syncthreads();
        if (grp > 0 || !real) return;
        float top = M;
#pragma unroll
        for (int k = 1; k < T; ++k) top = fmaxf(top, part_m[threadIdx.x + k * RG * COLS]);
        acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
        L = 0.f;
#pragma unroll
        for (int k = 0; k < T; ++k) {
            const int i = threadIdx.x + k * RG * COLS;
            const float lk = part_l[i];
            const float e = lk != 0.f ? fast_exp2(part_m[i] - top) : 0.f;   // a group without pieces: nothing
            const float4 o = part[i];
            L = fmaf(e, lk, L);
            acc[0].x = e != 0.f ? fmaf(e, o.x, acc[0].x) : acc[0].x;
            acc[0].y = e != 0.f ? fmaf(e, o.y, acc[0].y) : acc[0].y;
            acc[0].z = e != 0.f ? fmaf(e, o.z, acc[0].z) : acc[0].z;
            acc[0].w = e != 0.f ? fmaf(e, o.w, acc[0].w) : acc[0].w;
        }
        M = top;
    }
    const size_t orow = static_cast<size_t>(c) * p.H_Q + head * g + hr;
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint2 *dst = reinterpret_cast<uint2 *>(mp.out + orow * D + 4 * V * dg);
#pragma unroll
    for (int k = 0; k < V; ++k)
        dst[k] = L == 0.f ? make_uint2(0u, 0u)
                          : make_uint2(pack_bf16(acc[k].x * inv, acc[k].y * inv), pack_bf16(acc[k].z * inv, acc[k].w * inv));
    if (dg == 0 && p.lse) p.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

template <int D, int KIND, TcMode MODE>
DecodeKernel mod_tc_instance()
{
    struct Tag {};
    return configured<Tag>(reinterpret_cast<const void *>(&mod_tc_kernel<D, KIND, MODE>), ModTcCfg<D, KIND>::SMEM,
                           ModTcCfg<D, KIND>::THREADS, KIND == KV_BF16);
}

// The tensor-memory kernel for a head width, pool kind and mode.
DecodeKernel select_mod_tc_bf16(int D, TcMode mode);
DecodeKernel select_mod_tc_quant(bool int4, TcMode mode);
const void *select_mod_tc_merge(int D, bool few);

}  // namespace kvc
