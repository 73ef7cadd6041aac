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
#include <algorithm>
#include <type_traits>

#include "kvc_configured.cuh"

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
    // rows by slot (kvc_rope_write_slots): bt, start and cu are unused
    const int32_t *slots;      // [rows]
    const int32_t *positions;  // [num_axes][axis_stride]
    int64_t axis_stride;
    int32_t num_axes;
    const uint8_t *axis_of;    // [R / 2] or nullptr
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

// Eight channels of a key or value row into the pool at d (the elements' bytes), in fp32.
__device__ __forceinline__ void store_pool8(uint8_t *d, int bits, const float (&y)[8], const float *sc)
{
    if (bits == 16) {
        *reinterpret_cast<uint4 *>(d) =
            make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
    } else if (bits == 4) {
        uint32_t o = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) o |= int4_code(y[i], __ldg(sc + i)) << (4 * i);
        *reinterpret_cast<uint32_t *>(d) = o;
    } else {
        uint32_t o[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t c = __nv_cvt_float_to_fp8(__fdiv_rn(y[i], __ldg(sc + i)), __NV_SATFINITE, __NV_E4M3);
            o[i >> 2] |= c << (8 * (i & 3));
        }
        *reinterpret_cast<uint2 *>(d) = make_uint2(o[0], o[1]);
    }
}

constexpr int kRopeThreads = 256;              // the threads that move rows; one warp more looks ahead
constexpr int kRopeCta = kRopeThreads + 32;

// The sequence holding row r: the last b with cu[b] <= r, or -1 (r is past cu[B], or cu[0] > r).
__device__ __forceinline__ int find_sequence(const int32_t *cu, int B, int64_t r)
{
    if (r >= static_cast<int64_t>(__ldg(cu + B)) || r < static_cast<int64_t>(__ldg(cu))) return -1;
    int lo = 0, hi = B;   // cu[lo] <= r < cu[hi]
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (static_cast<int64_t>(__ldg(cu + mid)) <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

// What the CTA knows of a batch of TPC tokens.
template <int D, int TPC>
struct alignas(16) RopeBatch {
    // (own factor, mate's factor) of each channel of a query and a key row: the cosine and the signed sine
    // with the norm's weights folded in,  z_i = r (x_i (w_i cos a) - x_j (w_j sin a))
    float2 f[TPC][2][D];
    int64_t block[TPC];   // layer * N + block, or -1: not stored
    int32_t slot[TPC], pos[TPC];
    bool live[TPC];
};

// One thread: the given place of row r, the batch's token w.
template <int D, int TPC>
__device__ __forceinline__ void resolve_slot(const RopeParams &p, RopeBatch<D, TPC> &s, int w, int64_t r)
{
    const int32_t slot = r < p.rows ? __ldg(p.slots + r) : -1;
    s.live[w] = slot != -1;
    int64_t blk = -1;
    if (slot != -1) {
        if (slot < 0 || slot / p.bs >= p.N) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
        else blk = static_cast<int64_t>(p.layer) * p.N + slot / p.bs;
        s.slot[w] = slot % p.bs;
    }
    s.block[w] = blk;
}

// One thread: sequence, position and place of row r, the batch's token w.
template <int D, int TPC>
__device__ __forceinline__ void resolve_token(const RopeParams &p, RopeBatch<D, TPC> &s, int w, int64_t r)
{
    int b = -1;
    int64_t first = 0;
    if (r < p.rows) {
        if (p.cu) {
            b = find_sequence(p.cu, p.B, r);
            if (b >= 0) first = __ldg(p.cu + b);
        } else {
            b = static_cast<int>(r);
            first = r;
        }
    }
    s.live[w] = b >= 0;
    int64_t blk = -1;
    if (b >= 0) {
        const int32_t st = __ldg(p.start + b);
        const int64_t t = static_cast<int64_t>(st) + (r - first);
        s.pos[w] = static_cast<int32_t>(min(t, static_cast<int64_t>(0x7FFFFFFF)));
        if (st < 0 || t / p.bs >= p.max_blocks) {
            atomicOr(p.err, KVC_EBIT_RANGE);
        } else {
            const int32_t phys = __ldg(p.bt + static_cast<int64_t>(b) * p.max_blocks + t / p.bs);
            if (phys < 0 || static_cast<int64_t>(phys) >= p.N) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
            else blk = static_cast<int64_t>(p.layer) * p.N + phys;
            s.slot[w] = static_cast<int32_t>(t % p.bs);
        }
    }
    s.block[w] = blk;
}

// Threads tid of n: the factors of the batch's tokens, a pair (i, j) at a time.  SLOTS: r0 is the batch's first row,
// whose positions the pairs take from their axes.
template <int D, int TPC, bool SLOTS>
__device__ __forceinline__ void build_factors(const RopeParams &p, RopeBatch<D, TPC> &s, int tid, int n, int64_t r0)
{
    const int half = p.R >> 1;
    const int per = D / 2;   // pairs of a row: half that turn, the rest pass through
    for (int x = tid; x < TPC * per; x += n) {
        const int tk = x / per, i = x - tk * per;
        if (!s.live[tk]) continue;
        const bool turn = i < half;
        const int a = turn ? (p.interleaved ? 2 * i : i) : p.R + 2 * (i - half);
        const int b = turn ? (p.interleaved ? 2 * i + 1 : i + half) : a + 1;
        int32_t t = 0;
        if constexpr (SLOTS) {
            int axis = turn && p.axis_of ? __ldg(p.axis_of + i) : 0;
            if (axis >= p.num_axes) {
                atomicOr(p.err, KVC_EBIT_RANGE);
                axis = 0;
            }
            if (turn) t = __ldg(p.positions + axis * p.axis_stride + r0 + tk);
        } else {
            t = s.pos[tk];
        }
        const float2 cs = turn ? rotation(t, __ldg(p.inv_freq + i)) : make_float2(1.f, 0.f);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint16_t *w = k ? p.k_norm : p.q_norm;
            const float wa = w ? __uint_as_float(static_cast<uint32_t>(__ldg(w + a)) << 16) : 1.f;
            const float wb = w ? __uint_as_float(static_cast<uint32_t>(__ldg(w + b)) << 16) : 1.f;
            // a channel that passes through has no mate: not even a weight that is not finite reaches it
            s.f[tk][k][a] = make_float2(wa * cs.x, turn ? -wb * cs.y : 0.f);
            s.f[tk][k][b] = make_float2(wb * cs.x, turn ? wa * cs.y : 0.f);
        }
    }
}

// Persistent CTAs; each walks batches of TPC tokens.  256 threads = TPC tokens x GPT groups of D / 8 lanes, one
// lane per 16-byte chunk of a head row: a lane keeps its chunk and its eight channels' factors and walks the
// token's heads, U rows at a time with the next ones' loads in flight.  A ninth warp finds the next batch's
// sequences, positions and blocks (a chain of four dependent loads) and its factors meanwhile.
// Bound by HBM and by issue slots alike: 16 384 tokens of 32 + 2 x 8 heads of 128, normalised, bf16 (403 MB) take
// 74 us, 5.4 TB/s, 80 % of the copy rate; e4m3 pools 95 us and int4 98 (the exact divisions by the scales).  A CTA
// per four tokens without the ninth warp took 97 us (each CTA began with the chain of loads), the same with one row
// in flight 111 us; per-row address arithmetic and one loop over all kinds of head 95 us.
// SLOTS: rows whose places and positions are given (16 384 tokens with three axes: 74 us too, the axes' positions
// come out of L1); else sequences' runs of tokens.
template <int D, int GPT, int U, bool SLOTS>
__global__ void __launch_bounds__(kRopeCta, 3) rope_kernel(const RopeParams p)
{
    constexpr int CPR = D / 8;                            // chunks (lanes) per head row
    constexpr int TPC = kRopeThreads / CPR / GPT;         // tokens per batch
    __shared__ RopeBatch<D, TPC> sh[2];
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t batches = (p.rows + TPC - 1) / TPC;
    const int c = tid % CPR, grp = tid / CPR;
    const int tk = min(grp / GPT, TPC - 1), gi = grp % GPT;
    const bool mover = tid < kRopeThreads;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    // Rows of one kind (0: q, 1: k, 2: v) of a token: this group takes heads gi, gi + GPT, ...
    auto source = [&](int kind, int64_t r) {
        return (kind == 0 ? p.q + r * p.q_stride : kind == 1 ? p.k + r * p.k_stride : p.v + r * p.v_stride) + gi * D + 8 * c;
    };
    auto load = [&](uint4 (&x)[U], const uint16_t *src, int left) {   // left: heads from this one on
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[u] = u * GPT < left ? *reinterpret_cast<const uint4 *>(src + u * GPT * D) : make_uint4(0u, 0u, 0u, 0u);
    };
    int64_t batch = blockIdx.x;
    uint4 cur[U];
    const int kind0 = p.H_Q > 0 ? 0 : 1;   // the first kind of a token
    auto first_rows = [&](int64_t r) {
        load(cur, source(kind0, r), r < p.rows ? (kind0 == 0 ? p.H_Q : p.H_KV) - gi : 0);
    };
    if (mover) first_rows(batch * TPC + tk);
    static_assert(TPC <= 32, "one warp resolves a batch");
    auto resolve = [&](RopeBatch<D, TPC> &n, int w, int64_t r) {
        if constexpr (SLOTS) resolve_slot(p, n, w, r);
        else resolve_token(p, n, w, r);
    };
    if (tid < TPC) resolve(sh[0], tid, batch * TPC + tid);
    __syncthreads();
    build_factors<D, TPC, SLOTS>(p, sh[0], tid, kRopeCta, batch * TPC);
    const bool turns = 8 * c < p.R;
    // partner chunk of the half-split pairing
    const int hc = p.R >> 4;
    const int pc = p.interleaved || !turns ? c : (c >= hc ? c - hc : c + hc);
    const int src_lane = (lane & ~(CPR - 1)) | pc;
    const int64_t head_bytes = static_cast<int64_t>(2) * p.bs * D * p.bits / 8;   // a block's keys and values of a head

    for (int it = 0; batch < batches; batch += gridDim.x, ++it) {
        __syncthreads();   // this batch's facts are there; the buffer of the batch before is free
        const RopeBatch<D, TPC> &s = sh[it & 1];
        const int64_t after = batch + gridDim.x;
        if (!mover) {
            if (after < batches) {
                RopeBatch<D, TPC> &n = sh[(it + 1) & 1];
                if (lane < TPC) resolve(n, lane, after * TPC + lane);
                __syncwarp();
                build_factors<D, TPC, SLOTS>(p, n, lane, 32, after * TPC);
            }
            continue;
        }
        const int64_t r = batch * TPC + tk;
        const bool on = s.live[tk];
        const int64_t blk = on ? s.block[tk] : -1;
        // this lane's bytes of head gi's key slot
        uint8_t *pool = p.base + (blk >= 0 ? (blk * p.H_KV + gi) * head_bytes + (static_cast<int64_t>(s.slot[tk]) * D + 8 * c) * p.bits / 8 : 0);
        auto rows = [&](auto kind_c) {
            constexpr int KIND = decltype(kind_c)::value;
            const int n = KIND == 0 ? p.H_Q : p.H_KV;
            const bool act = KIND == 0 ? on : blk >= 0;
            const bool norm = KIND == 0 ? p.q_norm != nullptr : (KIND == 1 && p.k_norm != nullptr);
            const uint16_t *src = source(KIND, r);
            uint16_t *q_dst = p.q_out + (r * p.H_Q + gi) * D + 8 * c;
            uint8_t *dst = pool + (KIND == 2 ? static_cast<int64_t>(p.bs) * D * p.bits / 8 : 0);
            const float *sc = p.scales ? p.scales + ((KIND == 2 ? p.H_KV : 0) + gi) * static_cast<int64_t>(D) + 8 * c : nullptr;
            float2 f[8];
            if constexpr (KIND < 2) {
                const float4 *fs = reinterpret_cast<const float4 *>(&s.f[tk][KIND][8 * c]);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 v = fs[j];
                    f[2 * j] = make_float2(v.x, v.y);
                    f[2 * j + 1] = make_float2(v.z, v.w);
                }
            }
            // every lane runs every iteration (the shuffles are warp-wide)
            for (int h0 = 0; h0 < n; h0 += U * GPT) {
                uint4 next[U];
                src += U * GPT * D;
                if (h0 + U * GPT < n) load(next, src, r < p.rows ? n - gi - h0 - U * GPT : 0);
                else if constexpr (KIND < 2) load(next, source(KIND + 1, r), r < p.rows ? p.H_KV - gi : 0);
                else {
                    const int64_t r2 = r + static_cast<int64_t>(gridDim.x) * TPC;   // the next batch's first rows
                    load(next, source(kind0, r2), r2 < p.rows ? (kind0 == 0 ? p.H_Q : p.H_KV) - gi : 0);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const uint4 raw = cur[u];
                    float y[8];
                    if (KIND < 2 || p.bits != 16) unpack8(raw, y);
                    if constexpr (KIND < 2) {
                        uint4 mr;   // the mates: the partner chunk (half-split), or the pair's other channels
                        if (p.interleaved) {
                            mr = make_uint4(__byte_perm(raw.x, 0, 0x1032), __byte_perm(raw.y, 0, 0x1032),
                                            __byte_perm(raw.z, 0, 0x1032), __byte_perm(raw.w, 0, 0x1032));
                        } else {
                            mr.x = __shfl_sync(kFull, raw.x, src_lane);
                            mr.y = __shfl_sync(kFull, raw.y, src_lane);
                            mr.z = __shfl_sync(kFull, raw.z, src_lane);
                            mr.w = __shfl_sync(kFull, raw.w, src_lane);
                        }
                        if (!turns) mr = make_uint4(0u, 0u, 0u, 0u);   // whatever stands there, it adds nothing
                        float inv = 1.f;
                        if (norm) {
                            float ss = 0.f;
#pragma unroll
                            for (int j = 0; j < 8; ++j) ss = fmaf(y[j], y[j], ss);
#pragma unroll
                            for (int o = CPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
                            inv = rsqrtf(ss * (1.f / D) + p.eps);
                        }
                        float m[8];
                        unpack8(mr, m);
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = fmaf(m[j], f[j].y, y[j] * f[j].x);
                        if (norm)
#pragma unroll
                            for (int j = 0; j < 8; ++j) y[j] *= inv;
                    }
                    if (act && gi + h0 + u * GPT < n) {
                        if constexpr (KIND == 0)
                            *reinterpret_cast<uint4 *>(q_dst + u * GPT * D) = make_uint4(
                                pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
                        else if (KIND == 2 && p.bits == 16)
                            *reinterpret_cast<uint4 *>(dst + u * GPT * head_bytes) = raw;   // values: bits unchanged
                        else
                            store_pool8(dst + u * GPT * head_bytes, p.bits, y, sc + u * GPT * D);
                    }
                }
                q_dst += U * GPT * D;
                dst += U * GPT * head_bytes;
                if (sc) sc += U * GPT * D;
#pragma unroll
                for (int u = 0; u < U; ++u) cur[u] = next[u];
            }
        };
        if (p.H_Q > 0) rows(std::integral_constant<int, 0>{});
        rows(std::integral_constant<int, 1>{});
        rows(std::integral_constant<int, 2>{});
    }
}

template <int D, int GPT, int U, bool SLOTS>
static kvc_status launch_rope_as(const RopeParams &p, int sms, cudaStream_t stream)
{
    constexpr int TPC = kRopeThreads / (D / 8) / GPT;
    struct Tag {};
    const DecodeKernel k = configured<Tag>(reinterpret_cast<const void *>(&rope_kernel<D, GPT, U, SLOTS>), 0, kRopeCta, false);
    if (k.ctas_per_sm <= 0) return KVC_ERR_CUDA;
    // A programmatic dependent: its launch overlaps the tail of the kernel before it, which it
    // waits for before its first access.  It never lets its own dependents start early: the
    // chunk's kernel of kvc_mixed_step starts without waiting for the kernel before the step,
    // which may be this one.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>((p.rows + TPC - 1) / TPC, static_cast<int64_t>(sms) * k.ctas_per_sm)));
    cfg.blockDim = dim3(kRopeCta);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, rope_kernel<D, GPT, U, SLOTS>, p);
    if (e != cudaSuccess) return cuda_status(e);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return KVC_OK;
}

template <int D, int GPT, int U>
static kvc_status launch_rope(const RopeParams &p, int sms, cudaStream_t stream)
{
    return p.slots ? launch_rope_as<D, GPT, U, true>(p, sms, stream) : launch_rope_as<D, GPT, U, false>(p, sms, stream);
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

// Where the rows go: runs of sequences' tokens through a block table, or slots with positions of their own.
struct RopePlaces {
    const int32_t *bt = nullptr;
    int32_t max_blocks = 0;
    const int32_t *start = nullptr, *cu = nullptr;
    int32_t B = 0;
    bool by_slot = false;
    const int32_t *slots = nullptr, *positions = nullptr;
    int64_t axis_stride = 0;
    int32_t num_axes = 0;
    const uint8_t *axis_of = nullptr;
};

static kvc_status rope_write(kvc_pool *pool, int32_t layer, const RopePlaces &at, int64_t rows, const void *q,
                             int64_t q_stride, int32_t H_Q, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, const kvc_rope *rope, void *q_out, cudaStream_t stream)
{
    if (!pool || !rope || at.B < 0 || rows < 0 || rows > 0x7FFFFFFF || H_Q < 0 || H_Q > 65536) return KVC_ERR_ARG;
    const int D = pool->D;
    if (rope->rotary_dim < 0 || rope->rotary_dim > D || (rope->rotary_dim > 0 && !rope->inv_freq) ||
        !aligned(rope->inv_freq, 4) || !aligned(rope->q_norm, 16) || !aligned(rope->k_norm, 16) ||
        (rope->interleaved != 0 && rope->interleaved != 1))
        return KVC_ERR_ARG;
    if (rope->rotary_dim % 16 != 0) return KVC_ERR_UNSUPPORTED;
    if ((rope->q_norm || rope->k_norm) && !(std::isfinite(rope->norm_eps) && rope->norm_eps >= 0.f)) return KVC_ERR_ARG;
    if (at.by_slot && (at.num_axes < 1 || at.num_axes > 8 || at.axis_stride < 0)) return KVC_ERR_ARG;
    if ((!at.by_slot && at.B == 0) || rows == 0) return KVC_OK;
    if (layer < 0 || layer >= pool->L) return KVC_ERR_ARG;
    if (at.by_slot) {
        if (!at.slots || !at.positions || !aligned(at.slots, 4) || !aligned(at.positions, 4)) return KVC_ERR_ARG;
    } else if (at.max_blocks <= 0 || !at.bt || !at.start || !aligned(at.bt, 4) || !aligned(at.start, 4)) {
        return KVC_ERR_ARG;
    }
    if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return KVC_ERR_ARG;
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
    p.bt = at.bt;
    p.max_blocks = at.max_blocks;
    p.B = at.B;
    p.start = at.start;
    p.cu = at.cu;
    p.slots = at.slots;
    p.positions = at.positions;
    p.axis_stride = at.axis_stride;
    p.num_axes = at.num_axes;
    p.axis_of = at.axis_of;
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
    // Lane groups per token and rows in flight per lane: a token per CTA while there are few (latency), more
    // tokens per CTA as they grow (each batch costs a barrier and a look-up).  Measured, 32 + 2 x 8 heads of 128,
    // normalised: 64 tokens 4.3 us (16 groups, 1 row) against 5.0 (8, 1) and 6.4 (4, 2); 600 tokens 8.1, 6.1 and
    // 6.6; 4 000 tokens 32.5, 23.8 and 19.9; 16 384 tokens 121, 93 and 72.  Three rows in flight spill.
    const int sms = pool->num_sms;
    const int size = rows <= 2ll * sms ? 0 : (rows <= 8ll * sms ? 1 : 2);
    if (D == 64)
        return size == 0 ? launch_rope<64, 32, 1>(p, sms, stream)
                         : (size == 1 ? launch_rope<64, 8, 1>(p, sms, stream) : launch_rope<64, 2, 2>(p, sms, stream));
    return size == 0 ? launch_rope<128, 16, 1>(p, sms, stream)
                     : (size == 1 ? launch_rope<128, 8, 1>(p, sms, stream) : launch_rope<128, 4, 2>(p, sms, stream));
}

}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_rope_append(kvc_pool *pool, int32_t layer, const int32_t *block_tables, int32_t max_blocks,
                                      const int32_t *seq_lens, int32_t B, const void *q, int64_t q_stride,
                                      int32_t num_q_heads, const void *k_new, int64_t k_stride, const void *v_new,
                                      int64_t v_stride, const kvc_rope *rope, void *q_out, kvc_stream_t stream)
{
    RopePlaces at;
    at.bt = block_tables;
    at.max_blocks = max_blocks;
    at.start = seq_lens;
    at.B = B;
    return rope_write(pool, layer, at, B, q, q_stride, num_q_heads, k_new, k_stride, v_new, v_stride, rope, q_out,
                      static_cast<cudaStream_t>(stream));
}

extern "C" kvc_status kvc_rope_write_tokens(kvc_pool *pool, int32_t layer, const int32_t *block_tables,
                                            int32_t max_blocks, const int32_t *start_pos, const int32_t *cu_tokens,
                                            int32_t B, int64_t n_rows, const void *q, int64_t q_stride,
                                            int32_t num_q_heads, const void *k, int64_t k_stride, const void *v,
                                            int64_t v_stride, const kvc_rope *rope, void *q_out, kvc_stream_t stream)
{
    if (B > 0 && (!cu_tokens || !aligned(cu_tokens, 4))) return KVC_ERR_ARG;
    RopePlaces at;
    at.bt = block_tables;
    at.max_blocks = max_blocks;
    at.start = start_pos;
    at.cu = cu_tokens;
    at.B = B;
    return rope_write(pool, layer, at, n_rows, q, q_stride, num_q_heads, k, k_stride, v, v_stride, rope, q_out,
                      static_cast<cudaStream_t>(stream));
}

extern "C" kvc_status kvc_rope_write_slots(kvc_pool *pool, int32_t layer, const int32_t *slots,
                                           const int32_t *positions, int64_t axis_stride, int32_t num_axes,
                                           const uint8_t *axis_of, int64_t n_rows, const void *q, int64_t q_stride,
                                           int32_t num_q_heads, const void *k, int64_t k_stride, const void *v,
                                           int64_t v_stride, const kvc_rope *rope, void *q_out, kvc_stream_t stream)
{
    RopePlaces at;
    at.by_slot = true;
    at.slots = slots;
    at.positions = positions;
    at.axis_stride = axis_stride;
    at.num_axes = num_axes;
    at.axis_of = axis_of;
    return rope_write(pool, layer, at, n_rows, q, q_stride, num_q_heads, k, k_stride, v, v_stride, rope, q_out,
                      static_cast<cudaStream_t>(stream));
}
