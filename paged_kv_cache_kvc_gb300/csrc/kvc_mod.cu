// Entry points of attention with modified scores, their split sizing and the merge of splits.
#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "kvc_mod_tc.cuh"

namespace kvc {

// Log-sum-exp merge of a row's split partials: M = max m_s, L = sum 2^(m_s - M) l_s,
// out = sum 2^(m_s - M) o_s / L, lse = (M + log2 L) ln 2.  One CTA of 128 threads per
// output row: D / 4 float4 columns x 128 / (D / 4) groups of splits.  A row whose first split
// left l < 0 was finished by the attention kernel.  A programmatic dependent of that kernel.
template <int D>
__global__ void __launch_bounds__(128) mod_merge_kernel(const ModParams mp)
{
    constexpr int ND4 = D / 4, G = 128 / ND4;
    __shared__ float red[4], red2[4];
    __shared__ float4 part[128];
    const DecodeParams &p = mp.d;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, d4 = tid % ND4, grp = tid / ND4;
    const size_t bq = static_cast<size_t>(blockIdx.y) * p.H_Q + blockIdx.x;
    const int S = p.max_splits;
    const float2 *ml = p.part_ml + bq * S;
    const float4 *po = reinterpret_cast<const float4 *>(p.part_o + bq * S * D) + d4;
    grid_dependency_wait();
    if (ml[0].y < 0.f) return;   // uniform
    float m = -INFINITY;
    for (int s = tid; s < S; s += 128) m = fmaxf(m, ml[s].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (lane == 0) red[warp] = m;
    __syncthreads();
    const float M = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    const float Mref = M == -INFINITY ? 0.f : M;
    float l = 0.f;
    for (int s = tid; s < S; s += 128) l += fast_exp2(ml[s].x - Mref) * ml[s].y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
    if (lane == 0) red2[warp] = l;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = grp; s < S; s += G) {
        const float2 v = ml[s];
        if (v.y == 0.f) continue;   // a split that read nothing for this row wrote no partial row
        const float e = fast_exp2(v.x - Mref);
        const float4 o = po[static_cast<size_t>(s) * ND4];
        acc.x = fmaf(e, o.x, acc.x);
        acc.y = fmaf(e, o.y, acc.y);
        acc.z = fmaf(e, o.z, acc.z);
        acc.w = fmaf(e, o.w, acc.w);
    }
    part[tid] = acc;
    __syncthreads();
    const float L = (red2[0] + red2[1]) + (red2[2] + red2[3]);
    if (grp == 0) {
#pragma unroll
        for (int g2 = 1; g2 < G; ++g2) {
            const float4 v = part[g2 * ND4 + d4];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint2 *>(mp.out + bq * D + 4 * d4) =
            make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    }
    if (tid == 0 && p.lse) p.lse[bq] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
}

static cudaError_t launch_dependent(const void *fn, dim3 grid, dim3 block, int smem, cudaStream_t stream, void **args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, fn, args);
}

static bool aligned(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

// Query positions per unit of the split kernel: a decode sequence, or as many chunk positions as
// fill 32 query columns.
static int unit_positions(int g, bool tile) { return tile ? std::max(1, 32 / g) : 1; }

// The most blocks that a unit of `ppu` positions visits.
static int most_blocks(const kvc_score_mod *mod, int ppu, int max_blocks)
{
    if (!mod || mod->window <= 0) return max_blocks;
    if (mod->doc_start && mod->sink > 0) return max_blocks;   // sinks of several documents: their whole span
    const int64_t lead = std::max<int64_t>(mod->sink, mod->prefix);
    const int64_t n = (lead + kBS - 1) / kBS + (static_cast<int64_t>(mod->window) + ppu + 2 * kBS - 2) / kBS + 1;
    return static_cast<int>(std::min<int64_t>(n, max_blocks));
}

// The workspace: kCounters arrival counters at a fixed place whatever the call (zero between calls,
// so calls of other shapes may follow), then the call's split partials: fp32 sums
// [rows][H_Q][splits][D], then (max, sum) [rows][H_Q][splits].
constexpr int64_t kCounters = 16384;
constexpr size_t kCounterBytes = kCounters * sizeof(uint32_t);
static size_t partial_bytes(int64_t rows, int H_Q, int D)
{
    return static_cast<size_t>(rows) * H_Q * (D * sizeof(float) + sizeof(float2));
}

constexpr int kMinSplit = 16;     // blocks, choose_split's floor
constexpr int kInlineRows = 64;   // partial rows of a unit that its last split CTA merges itself

static kvc_status run_split(kvc_pool *pool, ModParams &mp, const DecodeKernel &k, int visit, void *ws, size_t ws_bytes,
                            cudaStream_t stream)
{
    if (!k.fn) return KVC_ERR_UNSUPPORTED;
    if (k.ctas_per_sm <= 0) return KVC_ERR_CUDA;
    DecodeParams &p = mp.d;
    choose_split(pool, p.B * p.H_KV, visit, k.ctas_per_sm, &p.chunk, &p.max_splits, n_tiles(p.ppu * p.g));
    if (!ws) {   // no room for partials: one split a unit
        p.chunk = visit;
        p.max_splits = 1;
    }
    if (p.max_splits > 65535) return KVC_ERR_UNSUPPORTED;
    p.counters = nullptr;
    p.part_o = nullptr;
    p.part_ml = nullptr;
    if (p.max_splits > 1) {
        const int64_t rows = static_cast<int64_t>(p.n_pos) * p.max_splits;
        if (ws_bytes < kCounterBytes + partial_bytes(rows, p.H_Q, pool->D)) return KVC_ERR_ARG;
        p.part_o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + kCounterBytes);
        p.part_ml = reinterpret_cast<float2 *>(p.part_o + static_cast<size_t>(rows) * p.H_Q * pool->D);
        if (p.ppu * p.g * p.max_splits <= kInlineRows && static_cast<int64_t>(p.B) * p.H_KV <= kCounters)
            p.counters = static_cast<uint32_t *>(ws);
    }
    void *args[] = {&pool->tmap, &mp};
    cudaError_t e = launch_dependent(k.fn, dim3(p.max_splits, p.H_KV, p.B), dim3(kThreads), k.smem, stream, args);
    if (e != cudaSuccess) return cuda_status(e);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    if (p.max_splits > 1 && !p.counters) {
        void *margs[] = {&mp};
        const void *mfn = pool->D == 64 ? reinterpret_cast<const void *>(&mod_merge_kernel<64>)
                                        : reinterpret_cast<const void *>(&mod_merge_kernel<128>);
        e = launch_dependent(mfn, dim3(p.H_Q, p.n_pos), dim3(128), 0, stream, margs);
        if (e != cudaSuccess) return cuda_status(e);
        g_launches.fetch_add(1, std::memory_order_relaxed);
    }
    return KVC_OK;
}

// The tensor-memory kernel's part of the workspace behind the counters: the units' running tile counts,
// then two pieces of a unit's 256 rows per CTA.
constexpr size_t kPrefixBytes = ((kMtUnits + 1) * sizeof(int32_t) + 255) & ~size_t(255);   // or one int4 per CTA
static size_t tc_bytes(int64_t ctas, int D)
{
    return kPrefixBytes + static_cast<size_t>(ctas) * 2 * 256 * (D * sizeof(float) + sizeof(float2));
}

// KVC_TC=0 selects the split kernel (as for the plain calls).
static bool use_tc(const kvc_pool *pool)
{
    const char *e = std::getenv("KVC_TC");
    return !(e && e[0] == '0') && (pool->dtype != KVC_BF16 || pool->tmap16_ok);   // the other map is checked for every call
}

// Decode groups of query heads from which the tensor-memory kernel serves a step.  Measured, capped, 32 heads, us against
// the split kernel's, bf16, e4m3, int4: 8 x 32 768 positions 45 / 44, 43 / 45, 50 / 53 (as good as level); 1 x 32 768:
// 34 / 37, 37 / 37, 38 / 42; 64 x 1 000: 20 / 37, 23 / 36, 25 / 40; ragged, bf16: 64 of 117 .. 30 000 63 / 120, 5 x 32 768
// beside 59 x 16 46 / 120, but 1 x 32 768 beside 79 x 500 371 / 119 (dealt whole, run_tc).  Smaller groups: 8 heads,
// 8 x 8 192 x 4 KV heads 42 / 32; 16 heads (bf16, whose weights the split kernel feeds as 16 bits), 8 x 8 192 x 2: 27 / 19.
constexpr int kTcGroup = 17;

// A chunk (or a decode batch of large head groups) on the tensor-memory kernel, as many units at a time as one
// launch takes.
static kvc_status run_tc(kvc_pool *pool, const ModParams &mp0, int visit, void *ws, size_t ws_bytes, cudaStream_t stream)
{
    ModTcParams tp{};
    tp.m = mp0;
    DecodeParams &p = tp.m.d;
    const bool decode = p.lens != nullptr;
    p.ppu = decode ? 1 : 128 / p.g;
    tp.total = p.len_base + p.n_pos;
    // Whole units of two query tiles ("dealt"), whole units of one that both chains share ("joined"), or cut units, by
    // the busiest CTA's time in tiles of 1.1 us.  A unit costs its tiles (joined: half of them, and kMtJoin) and
    // kMtStart; cutting costs the partials' way through memory and the merge, together about kMtCut.  The lengths of
    // documents and of decode sequences are not known here: documents are taken as a quarter of the row, sequences as
    // full, which is where the rule goes wrong.  Measured, capped, 32 heads over 8, us dealt / joined / cut: 64 queries at 0
    // 10 / 10 / 14, 300 at 300 20 / 16 / 24, 600 at 1 200 42 / 35 / 40, 1500 at 0 61 / 66 / 53, 100 at 2 000 48 / 37 / 27,
    // 2 000 in documents of 333 (e4m3, bias) 59 / 74 / 72, in one document 165 / 189 / 143 (dealt); decode, 32 heads over 1,
    // joined / cut: 64 x 1 000 20 / 31, 8 x 32 768 376 / 45, 64 of 117 .. 30 000 344 / 62, 1 x 32 768 beside 79 x 500
    // 372 / 35 (joined).
    int64_t longest = (visit + kMtBlocks - 1) / kMtBlocks, average = longest;
    if (mp0.doc_start) longest = average = longest / 4 + 1;
    else if (!decode && visit == p.max_blocks) average = std::max<int64_t>(1, longest - p.n_pos / 2 / kMtKeys);   // causal
    const int64_t sms = pool->num_sms, tall = (p.n_pos + 2 * p.ppu - 1) / (2 * p.ppu), low = (p.n_pos + p.ppu - 1) / p.ppu;
    auto rounds = [&](int64_t units) { return (p.H_KV * units + sms - 1) / sms; };
    const int64_t line = p.H_KV * (decode ? low : tall) * (average + kMtStart) / sms;   // a CTA's share of the line
    const int64_t joined = rounds(low) * (longest / 2 + kMtStart + kMtJoin);
    const int64_t dealt = decode ? joined : rounds(tall) * (longest + kMtStart);
    tp.whole = !ws || std::min(dealt, joined) <= line + kMtCut;
    tp.split = tp.whole ? joined <= dealt : decode || p.n_pos <= p.ppu;
    const bool fixed = tp.m.capped && !tp.m.alibi && (pool->dtype != KVC_BF16 || tp.m.cap_out <= kMtCapLimit);
    const TcMode mode = !tp.m.capped && !tp.m.alibi ? kMtPlain : !fixed ? kMtGeneral : pool->dtype == KVC_BF16 && line <= kMtBrief ? kMtCappedBrief : kMtCapped;
    const DecodeKernel k = pool->dtype == KVC_BF16 ? select_mod_tc_bf16(pool->D, mode)
                                                   : select_mod_tc_quant(pool->dtype == KVC_INT4, mode);
    if (!k.fn) return KVC_ERR_UNSUPPORTED;
    if (k.ctas_per_sm <= 0) return KVC_ERR_CUDA;
    const int unit = tp.split ? p.ppu : 2 * p.ppu;   // positions per unit
    const int units = tp.whole ? kMtUnits : units_per_launch((static_cast<int64_t>(p.max_blocks) + kMtBlocks - 1) / kMtBlocks);
    const int per_launch = units * unit, n_q = p.n_pos, start = p.len_base;
    for (int at = 0; at < n_q; at += per_launch) {
        p.n_pos = std::min(per_launch, n_q - at);
        p.len_base = start + at;
        p.q = mp0.d.q + static_cast<size_t>(at) * p.H_Q * pool->D;
        tp.m.out = mp0.out + static_cast<size_t>(at) * p.H_Q * pool->D;
        p.lse = mp0.d.lse ? mp0.d.lse + static_cast<size_t>(at) * p.H_Q : nullptr;
        tp.m.doc_start = mp0.doc_start ? mp0.doc_start + at : nullptr;
        if (decode) {
            p.lens = mp0.d.lens + at;
            p.bt = mp0.d.bt + static_cast<size_t>(at) * p.bt_stride;
        }
        tp.units = (p.n_pos + unit - 1) / unit;
        // no more CTAs than units dealt whole, or places on the line
        const int64_t most = static_cast<int64_t>(p.H_KV) * tp.units * (tp.whole ? 1 : (p.max_blocks + kMtBlocks - 1) / kMtBlocks + kMtStart);
        const int ctas = static_cast<int>(std::min<int64_t>(std::min(pool->num_sms, 512), most));
        if (!tp.whole) {
            if (ws_bytes < kCounterBytes + tc_bytes(ctas, pool->D)) return KVC_ERR_ARG;
            uint8_t *base = static_cast<uint8_t *>(ws) + kCounterBytes;
            tp.prefix = reinterpret_cast<int32_t *>(base);
            tp.cuts = reinterpret_cast<int4 *>(base);
            tp.part_o = reinterpret_cast<float *>(base + kPrefixBytes);
            tp.part_ml = reinterpret_cast<float2 *>(tp.part_o + static_cast<size_t>(ctas) * 2 * 256 * pool->D);
        }
        void *args[] = {k.tmap16 ? &pool->tmap16 : &pool->tmap, &tp};
        cudaError_t e = launch_dependent(k.fn, dim3(static_cast<unsigned>(ctas)), dim3(k.threads), k.smem, stream, args);
        if (e != cudaSuccess) return cuda_status(e);
        g_launches.fetch_add(1, std::memory_order_relaxed);
        if (!tp.whole) {
            const int rows = std::min(p.ppu, p.n_pos) * p.g, per = 128 / pool->D;
            const dim3 grid = tp.split ? dim3((rows + per - 1) / per, tp.units, p.H_KV) : dim3(8, ctas);
            void *margs[] = {&tp, const_cast<int *>(&ctas)};
            e = launch_dependent(select_mod_tc_merge(pool->D, tp.split != 0), grid, dim3(256), 0, stream, margs);
            if (e != cudaSuccess) return cuda_status(e);
            g_launches.fetch_add(1, std::memory_order_relaxed);
        }
    }
    return KVC_OK;
}

static kvc_status mod_checks(kvc_pool *pool, int32_t layer, const void *q, int32_t rows, int32_t H_Q, const int32_t *bt,
                             int32_t max_blocks, const kvc_score_mod *mod, void *out, float *lse, float scale, void *ws)
{
    if (!pool || !q || !bt || !out) return KVC_ERR_ARG;
    if (layer < 0 || layer >= pool->L) return KVC_ERR_ARG;
    if (H_Q <= 0 || H_Q % pool->H_KV != 0) return KVC_ERR_ARG;
    if (max_blocks <= 0 || max_blocks > (1 << 26)) return KVC_ERR_ARG;
    // scores are compared before they are scaled: a scale that is not positive would turn their order
    if (!std::isfinite(scale) || scale <= 0.f) return KVC_ERR_ARG;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(bt, 4) || !aligned(ws, 256)) return KVC_ERR_ARG;
    // out may be q: a row is written by the unit that has read it, or by the merge after every unit.  Shifted, a unit
    // would write rows that another has yet to read.
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
    const uintptr_t bytes = static_cast<uintptr_t>(rows) * H_Q * pool->D * 2;
    if (q0 != o0 && q0 < o0 + bytes && o0 < q0 + bytes) return KVC_ERR_ARG;
    if (mod) {
        if (!std::isfinite(mod->softcap) || mod->softcap < 0.f || mod->window < 0 || mod->sink < 0 || mod->prefix < 0)
            return KVC_ERR_ARG;
        if (mod->softcap > 0.f && !std::isfinite(2.f * scale * 1.4426950408889634f / mod->softcap)) return KVC_ERR_ARG;
        // the cap's error is absolute, 2^-23 of it: past this it would show in the weights, however small the scores
        if (mod->softcap > 4096.f) return KVC_ERR_UNSUPPORTED;
        if (!aligned(mod->alibi, 4) || !aligned(mod->doc_start, 4)) return KVC_ERR_ARG;
        if (mod->doc_start && mod->prefix > 0) return KVC_ERR_UNSUPPORTED;
    }
    if (H_Q / pool->H_KV > 32) return KVC_ERR_UNSUPPORTED;
    if (pool->bs != kBS || !pool->tmap_ok) return KVC_ERR_UNSUPPORTED;
    return check_device(pool);
}

static void fill(ModParams &mp, const kvc_pool *pool, int32_t layer, const void *q, int32_t H_Q, const int32_t *bt,
                 int32_t max_blocks, const kvc_score_mod *mod, void *out, float *lse, float scale)
{
    DecodeParams &p = mp.d;
    p.q = static_cast<const uint16_t *>(q);
    p.bt = bt;
    p.max_blocks = max_blocks;
    p.H_Q = H_Q;
    p.H_KV = pool->H_KV;
    p.g = H_Q / pool->H_KV;
    p.layer = layer;
    p.N = pool->N;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.s_k = pool->scales ? pool->scales + static_cast<size_t>(layer) * 2 * pool->H_KV * pool->D : nullptr;
    p.s_v = p.s_k ? p.s_k + static_cast<size_t>(pool->H_KV) * pool->D : nullptr;
    p.lse = lse;
    p.err = pool->err;
    p.pool = pool->base;
    p.stall_loads = std::getenv("KVC_TEST_STALL") ? 1 : 0;
    mp.out = static_cast<uint16_t *>(out);
    if (mod) {
        mp.alibi = mod->alibi;
        mp.doc_start = mod->doc_start;
        mp.window = mod->window;
        mp.sink = mod->sink;
        mp.prefix = mod->prefix;
        mp.capped = mod->softcap > 0.f;
        if (mp.capped) {
            mp.cap_in = 2.f * p.scale_log2 / mod->softcap;
            mp.cap_out = mod->softcap * 1.4426950408889634f;
        }
    }
}

static DecodeKernel select(const kvc_pool *pool, int cols, bool tile)
{
    if (pool->dtype == KVC_FP8_E4M3) return select_mod_fp8(cols, tile);
    if (pool->dtype == KVC_INT4) return select_mod_int4(cols, tile);
    return select_mod_bf16(pool->D, cols, tile);
}

}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_mod_workspace_bytes(const kvc_pool *pool, int32_t rows, int32_t num_q_heads,
                                              int32_t max_blocks, uint64_t *bytes)
{
    if (!pool || !bytes || rows < 0 || rows > 65535 || num_q_heads <= 0 || num_q_heads % pool->H_KV != 0 ||
        max_blocks <= 0 || max_blocks > (1 << 26))
        return KVC_ERR_ARG;
    if (num_q_heads / pool->H_KV > 32) return KVC_ERR_UNSUPPORTED;
    // The most partial rows that a call of up to `rows` rows plans.  choose_split gives a unit at most
    // 1.7 CTAs a resident slot over the units (at most 8 slots an SM), or what 288-block splits need,
    // and no split under kMinSplit blocks; a unit holds ppu rows, so units x splits x ppu stays under
    // the first bound whatever the rows are.
    const int ppu = unit_positions(num_q_heads / pool->H_KV, true);
    const int64_t by_len = (max_blocks + kMinSplit - 1) / kMinSplit;
    const int64_t by_slots = ppu * (14ll * pool->num_sms / pool->H_KV + 1) + 2ll * rows;
    const int64_t by_cap = rows * ((max_blocks + 283ll) / 284 + 1);
    const int64_t n = std::min(rows * by_len, std::max(by_slots, by_cap));
    *bytes = kCounterBytes + std::max(partial_bytes(n, num_q_heads, pool->D), tc_bytes(pool->num_sms, pool->D));
    return KVC_OK;
}

extern "C" kvc_status kvc_decode_attn_mod(kvc_pool *pool, int32_t layer, const void *q, int32_t num_q_heads,
                                          const int32_t *block_tables, int32_t max_blocks, const int32_t *seq_lens,
                                          int32_t B, const kvc_score_mod *mod, void *out, float *lse, float scale,
                                          void *workspace, uint64_t workspace_bytes, kvc_stream_t stream)
{
    if (B < 0 || B > 65535) return KVC_ERR_ARG;
    if (B == 0) return pool ? KVC_OK : KVC_ERR_ARG;
    if (!seq_lens || !aligned(seq_lens, 4)) return KVC_ERR_ARG;
    if (mod && mod->doc_start) return KVC_ERR_ARG;
    kvc_status st = mod_checks(pool, layer, q, B, num_q_heads, block_tables, max_blocks, mod, out, lse, scale, workspace);
    if (st != KVC_OK) return st;
    ModParams mp{};
    fill(mp, pool, layer, q, num_q_heads, block_tables, max_blocks, mod, out, lse, scale);
    mp.d.lens = seq_lens;
    mp.d.bt_stride = max_blocks;
    mp.d.B = B;
    mp.d.ppu = 1;
    mp.d.n_pos = B;
    // Large head groups: one tensor-memory step serves the whole group
    if (workspace && use_tc(pool) && mp.d.g >= kTcGroup)
        return run_tc(pool, mp, most_blocks(mod, 1, max_blocks), workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
    return run_split(pool, mp, select(pool, mp.d.g, false), most_blocks(mod, 1, max_blocks), workspace, workspace_bytes,
                     static_cast<cudaStream_t>(stream));
}

extern "C" kvc_status kvc_prefill_attn_mod(kvc_pool *pool, int32_t layer, const void *q, int32_t n_q,
                                           int32_t num_q_heads, const int32_t *block_table_row, int32_t max_blocks,
                                           int32_t q_start, const kvc_score_mod *mod, void *out, float *lse,
                                           float scale, void *workspace, uint64_t workspace_bytes, kvc_stream_t stream)
{
    if (n_q < 0 || n_q > 65535 || q_start < 0) return KVC_ERR_ARG;
    if (n_q == 0) return pool ? KVC_OK : KVC_ERR_ARG;
    kvc_status st = mod_checks(pool, layer, q, n_q, num_q_heads, block_table_row, max_blocks, mod, out, lse, scale, workspace);
    if (st != KVC_OK) return st;
    if (static_cast<int64_t>(q_start) + n_q > static_cast<int64_t>(max_blocks) * kBS) return KVC_ERR_RANGE;
    ModParams mp{};
    const int blocks = static_cast<int>((static_cast<int64_t>(q_start) + n_q + kBS - 1) / kBS);
    fill(mp, pool, layer, q, num_q_heads, block_table_row, blocks, mod, out, lse, scale);
    DecodeParams &p = mp.d;
    p.len_base = q_start;
    p.n_pos = n_q;
    if (use_tc(pool))
        return run_tc(pool, mp, most_blocks(mod, 256 / p.g, blocks), workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
    p.ppu = unit_positions(p.g, true);
    p.B = (n_q + p.ppu - 1) / p.ppu;
    return run_split(pool, mp, select(pool, p.ppu * p.g, true), most_blocks(mod, p.ppu, blocks), workspace, workspace_bytes,
                     static_cast<cudaStream_t>(stream));
}
