// Rotary write: per token, optional RMS norm of each query and key head, the
// position rotation of queries and keys, and the store of keys and values into
// the paged pool, in one pass over the fused projection's output.
//
// Mathematics, per head row x of d_h channels at position t:
//   y_i = x_i                                    (no norm weight)
//   y_i = x_i / sqrt(mean_j x_j^2 + eps) * w_i   (RMS norm)
//   angle a_i = t f_i, pair (i, j) = (i, i + R/2) or (2i, 2i + 1), i < R/2:
//   z_i = y_i cos a_i - y_j sin a_i,  z_j = y_j cos a_i + y_i sin a_i
// and channels at or past R pass through.  All of it in fp32 from the bf16
// inputs, rounded once: queries to bf16, keys to the pool's element type
// (values as kvc_append stores them).
//
// Angles.  t f_i grows to 1e5 radians and more, where one fp32 product is off
// by whole hundredths, so the angle is kept in turns as unevaluated sums: f/2pi
// is split into two floats, t into a multiple of 4096 and the rest (both exact
// in fp32), the products keep their fma remainders, and whole turns drop out
// exactly at each step.  The angle is good to 1e-6 radians up to t = 2^24
// (bf16 outputs round at 4e-3) without fp64, whose units are few on this part.
#include "kvc_decode.cuh"

namespace kvc {

struct RopeParams {
    uint8_t *base;
    int64_t N;
    int32_t bs, H_KV, H_Q, layer, bits;
    const int32_t *bt;
    int32_t max_blocks, B;
    const int32_t *start;      // [B] first position written
    const int32_t *cu;         // [B+1] row offsets, or nullptr: row b is sequence b's one token
    int64_t rows;              // rows of q, k, v, q_out
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    uint16_t *q_out;           // [rows][H_Q][D]
    const float *inv_freq;
    int32_t R, interleaved;
    const uint16_t *q_norm, *k_norm;
    float eps;
    const float *scales;       // this layer's [2][H_KV][D], or nullptr (bf16)
    uint32_t *err;
};

// cos and sin of t * f (radians), t a position
__device__ __forceinline__ float2 rotation(int32_t t, float f)
{
    constexpr float kInv2Pi = 0.15915494309189535f;                                       // 1 / 2pi to fp32
    constexpr float kInv2PiLo = static_cast<float>(0.15915494309189533577 - static_cast<double>(kInv2Pi));
    const float th = f * kInv2Pi;
    const float tl = fmaf(f, kInv2PiLo, fmaf(f, kInv2Pi, -th));
    const float p1 = static_cast<float>(t & ~4095), p0 = static_cast<float>(t & 4095);   // t = p1 + p0, exact
    float a = p1 * th, b = p0 * th;
    const float lo = fmaf(p1, tl, fmaf(p0, tl, fmaf(p1, th, -a) + fmaf(p0, th, -b)));
    a -= rintf(a);
    b -= rintf(b);
    float r = a + b;
    r -= rintf(r);
    r += lo - rintf(lo);
    float2 cs;
    sincospif(2.f * r, &cs.y, &cs.x);
    return cs;
}

__device__ __forceinline__ void unpack8(const uint4 &x, float (&f)[8])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

// Eight channels of a key or value row into the pool at element index e; vals in fp32.
__device__ __forceinline__ void store_pool8(const RopeParams &p, int64_t e, const float (&y)[8], const float *sc)
{
    if (p.bits == 16) {
        *reinterpret_cast<uint4 *>(p.base + e * 2) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    } else if (p.bits == 4) {
        uint32_t o = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) o |= int4_code(y[i], __ldg(sc + i)) << (4 * i);
        *reinterpret_cast<uint32_t *>(p.base + e / 2) = o;
    } else {
        uint32_t o[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = __nv_cvt_float_to_fp8(__fdiv_rn(y[i], __ldg(sc + i)), __NV_SATFINITE, __NV_E4M3);
            o[i >> 2] |= c << (8 * (i & 3));
        }
        *reinterpret_cast<uint2 *>(p.base + e) = make_uint2(o[0], o[1]);
    }
}

constexpr int kRopeThreads = 256;

// The sequence holding row r: the last b with cu[b] <= r, or -1 (r is past cu[B], or cu[0] > r).
// Whole warp; 32 probes per step.
__device__ __forceinline__ int find_sequence(const int32_t *cu, int B, int64_t r, int lane)
{
    if (r >= static_cast<int64_t>(__ldg(cu + B))) return -1;
    int lo = 0, n = B;   // candidates lo .. lo + n - 1
    while (true) {
        const int step = (n + 31) / 32;
        const int i = lo + lane * step;
        const bool le = lane * step < n && static_cast<int64_t>(__ldg(cu + i)) <= r;
        const int hits = __popc(__ballot_sync(kFull, le));   // cu is non-decreasing: a prefix of the probes
        if (hits == 0) return -1;
        lo += (hits - 1) * step;
        n = min(step, n - (hits - 1) * step);
        if (step == 1) return lo;
    }
}

// grid (tokens / TPC); 256 threads = TPC tokens x groups of D / 8 lanes, one lane per 16-byte
// chunk of a head row, so a lane keeps its chunk (and its 8 angles) and walks the token's heads.
template <int D, int TPC>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeParams p)
{
    constexpr int CPR = D / 8;                            // chunks (lanes) per head row
    constexpr int GPT = kRopeThreads / CPR / TPC;         // lane groups per token
    __shared__ float2 cs[TPC][D / 2];
    __shared__ int64_t dst_block[TPC];                    // (layer * N + block) of the token, or -1: not stored
    __shared__ int32_t dst_slot[TPC], pos_sh[TPC];
    __shared__ bool live[TPC];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * TPC;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp < TPC) {   // warp w resolves token w
        const int64_t r = row0 + warp;
        int b = -1;
        int64_t first = 0;
        if (r < p.rows) {
            if (p.cu) {
                b = find_sequence(p.cu, p.B, r, lane);
                if (b >= 0) first = __ldg(p.cu + b);
            } else {
                b = static_cast<int>(r);
                first = r;
            }
        }
        if (lane == 0) {
            live[warp] = b >= 0;
            int64_t blk = -1;
            if (b >= 0) {
                const int32_t s = __ldg(p.start + b);
                const int64_t t = static_cast<int64_t>(s) + (r - first);
                pos_sh[warp] = static_cast<int32_t>(min(t, static_cast<int64_t>(0x7FFFFFFF)));
                if (s < 0 || t / p.bs >= p.max_blocks) {
                    atomicOr(p.err, KVC_EBIT_RANGE);
                } else {
                    const int32_t phys = __ldg(p.bt + static_cast<int64_t>(b) * p.max_blocks + t / p.bs);
                    if (phys < 0 || static_cast<int64_t>(phys) >= p.N) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
                    else blk = static_cast<int64_t>(p.layer) * p.N + phys;
                    dst_slot[warp] = static_cast<int32_t>(t % p.bs);
                }
            }
            dst_block[warp] = blk;
        }
    }
    __syncthreads();
    const int half = p.R >> 1;
    for (int i = tid; i < TPC * half; i += kRopeThreads) {
        const int tk = i / half, j = i - tk * half;
        if (live[tk]) cs[tk][j] = rotation(pos_sh[tk], __ldg(p.inv_freq + j));
    }
    __syncthreads();

    const int c = tid % CPR, grp = tid / CPR;
    const int tk = grp / GPT, gi = grp % GPT;
    const int heads = p.H_Q + 2 * p.H_KV;
    const bool on = live[tk];
    const int64_t r = row0 + tk;
    const int64_t blk = on ? dst_block[tk] : -1;
    const int slot = on && blk >= 0 ? dst_slot[tk] : 0;
    const bool turns = 8 * c < p.R;
    // partner chunk of the half-split pairing and this lane's side of the pair
    const int hc = half >> 3;
    const bool second = !p.interleaved && turns && c >= hc;
    const int pc = p.interleaved || !turns ? c : (second ? c - hc : c + hc);
    const int src_lane = (lane & ~(CPR - 1)) | pc;
    float co[8], si[8];   // the cosine and signed sine each channel takes
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        co[j] = 1.f;
        si[j] = 0.f;
        if (on && turns) {
            const int i = p.interleaved ? 4 * c + (j >> 1) : 8 * (second ? c - hc : c) + j;
            const float2 v = cs[tk][i];
            const bool minus = p.interleaved ? !(j & 1) : !second;
            co[j] = v.x;
            si[j] = minus ? -v.y : v.y;
        }
    }
    // heads in order q, k, v; every lane runs every iteration (the shuffles are warp-wide)
    for (int h = gi; h - gi < heads; h += GPT) {
        const bool act = on && h < heads;
        const int kind = h < p.H_Q ? 0 : (h < p.H_Q + p.H_KV ? 1 : 2);
        const int hh = kind == 0 ? h : (kind == 1 ? h - p.H_Q : h - p.H_Q - p.H_KV);
        uint4 raw = make_uint4(0u, 0u, 0u, 0u);
        if (act) {
            const uint16_t *src = kind == 0 ? p.q + r * p.q_stride : (kind == 1 ? p.k + r * p.k_stride : p.v + r * p.v_stride);
            raw = *reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(hh) * D + 8 * c);
        }
        float y[8];
        unpack8(raw, y);
        const uint16_t *w = kind == 0 ? p.q_norm : (kind == 1 ? p.k_norm : nullptr);
        float ss = 0.f;
        if (p.q_norm || p.k_norm) {   // uniform: either norm runs the reduction for every lane
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
#pragma unroll
            for (int o = CPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
        }
        if (act && w) {
            const float inv = rsqrtf(ss * (1.f / D) + p.eps);
            float wf[8];
            unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + c), wf);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = y[j] * inv * wf[j];
        }
        float z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float other = __shfl_sync(kFull, y[j], src_lane);   // the partner chunk's channel (half-split)
            const float mate = p.interleaved ? y[j ^ 1] : other;
            z[j] = kind == 2 || !turns ? y[j] : fmaf(y[j], co[j], mate * si[j]);
        }
        if (!act) continue;
        if (kind == 0) {
            *reinterpret_cast<uint4 *>(p.q_out + (r * p.H_Q + hh) * D + 8 * c) =
                make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]), pack_bf16(z[6], z[7]));
        } else if (blk >= 0) {
            const int kv = kind - 1;
            const int64_t e = (((blk * p.H_KV + hh) * 2 + kv) * p.bs + slot) * D + 8 * c;
            if (kv == 1 && p.bits == 16) *reinterpret_cast<uint4 *>(p.base + e * 2) = raw;   // values: bits unchanged
            else store_pool8(p, e, z, p.scales + (static_cast<int64_t>(kv) * p.H_KV + hh) * D + 8 * c);
        }
    }
}

template <int D, int TPC>
static cudaError_t launch_rope_tpc(const RopeParams &p, cudaStream_t stream)
{
    // A programmatic dependent: its launch overlaps the tail of the kernel before it, which it
    // waits for before its first access.  It never lets its own dependents start early: the
    // chunk's kernel of kvc_mixed_step starts without waiting for the kernel before the step,
    // which may be this one.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.rows + TPC - 1) / TPC));
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rope_kernel<D, TPC>, p);
}

static bool aligned(const void *ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) & (a - 1)) == 0; }

// Whether the bytes of two row sets (rows x stride elements, the last row `width` long) meet.
static bool overlap(const void *a, int64_t sa, int64_t wa, const void *b, int64_t sb, int64_t wb, int64_t rows)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    const uintptr_t a1 = a0 + static_cast<uintptr_t>((rows - 1) * sa + wa) * 2;
    const uintptr_t b1 = b0 + static_cast<uintptr_t>((rows - 1) * sb + wb) * 2;
    return a0 < b1 && b0 < a1;
}

static kvc_status rope_write(kvc_pool *pool, int32_t layer, const int32_t *bt, int32_t max_blocks,
                             const int32_t *start, const int32_t *cu, int32_t B, int64_t rows, const void *q,
                             int64_t q_stride, int32_t H_Q, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const kvc_rope *rope, void *q_out, cudaStream_t stream)
{
    if (!pool || !rope || B < 0 || rows < 0 || rows > 0x7FFFFFFF || H_Q < 0 || H_Q > 65536) return KVC_ERR_ARG;
    const int D = pool->D;
    if (rope->rotary_dim < 0 || rope->rotary_dim > D || (rope->rotary_dim > 0 && !rope->inv_freq) ||
        !aligned(rope->inv_freq, 4) || !aligned(rope->q_norm, 16) || !aligned(rope->k_norm, 16) ||
        (rope->interleaved != 0 && rope->interleaved != 1))
        return KVC_ERR_ARG;
    if (rope->rotary_dim % 16 != 0) return KVC_ERR_UNSUPPORTED;
    if ((rope->q_norm || rope->k_norm) && !(std::isfinite(rope->norm_eps) && rope->norm_eps >= 0.f)) return KVC_ERR_ARG;
    if (B == 0 || rows == 0) return KVC_OK;
    if (layer < 0 || layer >= pool->L || max_blocks <= 0) return KVC_ERR_ARG;
    if (!bt || !start || !k || !v || !aligned(k, 16) || !aligned(v, 16) || !aligned(bt, 4) || !aligned(start, 4))
        return KVC_ERR_ARG;
    const int64_t qw = static_cast<int64_t>(H_Q) * D, kw = static_cast<int64_t>(pool->H_KV) * D;
    if (k_stride < kw || v_stride < kw || k_stride % 8 != 0 || v_stride % 8 != 0) return KVC_ERR_ARG;
    if (H_Q > 0) {
        if (!q || !q_out || !aligned(q, 16) || !aligned(q_out, 16) || q_stride < qw || q_stride % 8 != 0)
            return KVC_ERR_ARG;
        // q_out may be q itself (each row is read whole by the warp that writes it), nothing else
        if (!(q_out == q && q_stride == qw) && overlap(q, q_stride, qw, q_out, qw, qw, rows)) return KVC_ERR_ARG;
        if (overlap(k, k_stride, kw, q_out, qw, qw, rows) || overlap(v, v_stride, kw, q_out, qw, qw, rows))
            return KVC_ERR_ARG;
    }
    kvc_status st = check_device(pool);
    if (st != KVC_OK) return st;
    RopeParams p{};
    p.base = pool->base;
    p.N = pool->N;
    p.bs = pool->bs;
    p.H_KV = pool->H_KV;
    p.H_Q = H_Q;
    p.layer = layer;
    p.bits = pool->bits;
    p.bt = bt;
    p.max_blocks = max_blocks;
    p.B = B;
    p.start = start;
    p.cu = cu;
    p.rows = rows;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = static_cast<uint16_t *>(q_out);
    p.inv_freq = rope->inv_freq;
    p.R = rope->rotary_dim;
    p.interleaved = rope->interleaved;
    p.q_norm = static_cast<const uint16_t *>(rope->q_norm);
    p.k_norm = static_cast<const uint16_t *>(rope->k_norm);
    p.eps = rope->norm_eps;
    p.scales = pool->scales ? pool->scales + static_cast<size_t>(layer) * 2 * pool->H_KV * D : nullptr;
    p.err = pool->err;
    // four tokens a CTA once that still gives every SM several CTAs, else one
    const bool wide = rows >= 16ll * pool->num_sms;
    cudaError_t e;
    if (D == 64) e = wide ? launch_rope_tpc<64, 4>(p, stream) : launch_rope_tpc<64, 1>(p, stream);
    else e = wide ? launch_rope_tpc<128, 4>(p, stream) : launch_rope_tpc<128, 1>(p, stream);
    if (e != cudaSuccess) return cuda_status(e);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return KVC_OK;
}

}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_rope_append(kvc_pool *pool, int32_t layer, const int32_t *block_tables, int32_t max_blocks,
                                      const int32_t *seq_lens, int32_t B, const void *q, int64_t q_stride,
                                      int32_t num_q_heads, const void *k_new, int64_t k_stride, const void *v_new,
                                      int64_t v_stride, const kvc_rope *rope, void *q_out, kvc_stream_t stream)
{
    return rope_write(pool, layer, block_tables, max_blocks, seq_lens, nullptr, B, B, q, q_stride, num_q_heads, k_new,
                      k_stride, v_new, v_stride, rope, q_out, static_cast<cudaStream_t>(stream));
}

extern "C" kvc_status kvc_rope_write_tokens(kvc_pool *pool, int32_t layer, const int32_t *block_tables,
                                            int32_t max_blocks, const int32_t *start_pos, const int32_t *cu_tokens,
                                            int32_t B, int64_t n_rows, const void *q, int64_t q_stride,
                                            int32_t num_q_heads, const void *k, int64_t k_stride, const void *v,
                                            int64_t v_stride, const kvc_rope *rope, void *q_out, kvc_stream_t stream)
{
    if (B > 0 && (!cu_tokens || !aligned(cu_tokens, 4))) return KVC_ERR_ARG;
    return rope_write(pool, layer, block_tables, max_blocks, start_pos, cu_tokens, B, n_rows, q, q_stride, num_q_heads,
                      k, k_stride, v, v_stride, rope, q_out, static_cast<cudaStream_t>(stream));
}
