// Block tables and slot maps of a step, built on the GPU from the lengths that sequences have and shall have.
//
// Mathematics.  have = ceil(len / bs), want = ceil(new / bs); per sequence rel = max(have - want, 0),
// grow = max(want - have, 0), tok = max(new - len, 0).  With inclusive sums G, T over the sequences and
// avail = free + sum rel, sequence b's growth is over the limit when G_b > avail or T_b > n_rows.  The sums never
// fall, so from the first sequence over the limit every later one is over it too: "first come, first served" needs
// no serial walk, and what is granted in all is the largest G and T that are not over.  Block i of the granted ones
// comes from stack[avail - 1 - i]; row r belongs to the sequence with cu_b <= r < cu_{b+1}.
//
// One cluster does a step in one launch.  Each CTA owns a run of sequences; the CTAs exchange their sums through
// distributed shared memory, and two cluster barriers order what passes through global memory: blocks pushed before
// blocks popped, tables written before slots are looked up.  Sums are 32 bits and stop at 2^31 - 1 (adding numbers
// that are not negative, such sums stay associative), which is over every limit.
//
// Latency bounds it: a decoding batch reads and writes a few kilobytes.  8 sequences, one more token each, take 3.8 us
// back to back (one CTA; 6.7 with the cluster's barriers and a thread's four rows looked up one after another).  512
// sequences with 65 536 new rows take 13: 8 in the cluster (three barriers, two passes over the tables), then the
// maps in a kernel over the whole GPU (written by the cluster's eight SMs they took 12 alone: 60 instructions a row).
#include <algorithm>

#include "kvc_cluster.cuh"
#include "kvc_configured.cuh"

namespace kvc {

constexpr int kPlanCluster = 8;
constexpr int kPlanMost = 32768;      // sequences: a CTA keeps five words for each of its own, and all row offsets

struct PlanParams {
    int32_t *bt;
    int32_t max_blocks;
    const int32_t *lens, *want;
    int32_t B, bs;
    int64_t N;
    int32_t *stack;
    int32_t capacity;
    const int32_t *count;
    int32_t *lens_out, *count_out, *cu, *slots, *positions, *seqs;
    int32_t n_rows;
    bool rows_here;   // the cluster writes the maps too
    uint32_t *err;
};

__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return min(a + b, 0x7FFFFFFFu); }

// Blocks returned, blocks asked for, rows asked for.
struct PlanSum {
    uint32_t rel, grow, tok;
};

__device__ __forceinline__ PlanSum operator+(const PlanSum &a, const PlanSum &b)
{
    return {add_sat(a.rel, b.rel), add_sat(a.grow, b.grow), add_sat(a.tok, b.tok)};
}

// The i with off[i] <= x < off[i + 1], given off[0] <= x < off[n]; ties go to the last i with off[i] <= x.
__device__ __forceinline__ int find_run(const uint32_t *off, int n, uint32_t x)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ bool maps_aligned(const PlanParams &p)   // to 16 bytes; null pointers are
{
    return ((reinterpret_cast<uintptr_t>(p.slots) | reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.seqs)) & 15) == 0;
}

// Rows r0 .. r0 + 3 of the maps.  cu: row offsets of n sequences from `first` on (and one more), which hold the rows below
// `total`; rows from there on are padding.  wide: the maps are 16-byte aligned.
__device__ __forceinline__ void write_rows(const PlanParams &p, int64_t r0, uint32_t total, const uint32_t *cu, int first, int n, bool wide)
{
    // the four rows' sequences first, then what each has to look up: two loads after one another, not eight
    int s[4], pos[4], seq[4];
    int b = -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint32_t r = static_cast<uint32_t>(r0) + u;
        seq[u] = -1;
        if (r < total) {
            if (b < 0) b = find_run(cu, n, r);
            while (r >= cu[b + 1]) ++b;
            seq[u] = first + b;
        }
    }
    int32_t has[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) has[u] = seq[u] >= 0 ? __ldcg(p.lens_out + seq[u]) : 0;
    int32_t blk[4], place[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        pos[u] = place[u] = blk[u] = -1;
        if (seq[u] >= 0) {   // the last of the sequence's new tokens is at has - 1
            pos[u] = has[u] - static_cast<int32_t>(cu[seq[u] - first + 1] - (static_cast<uint32_t>(r0) + u));
            const int32_t j = pos[u] / p.bs;
            place[u] = pos[u] - j * p.bs;
            blk[u] = __ldcg(p.bt + static_cast<int64_t>(seq[u]) * p.max_blocks + j);
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const bool bad = seq[u] >= 0 && (blk[u] < 0 || blk[u] >= p.N);
        if (bad) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
        s[u] = seq[u] < 0 || bad ? -1 : blk[u] * p.bs + place[u];
    }
    if (wide && r0 + 4 <= p.n_rows) {
        *reinterpret_cast<int4 *>(p.slots + r0) = make_int4(s[0], s[1], s[2], s[3]);
        if (p.positions) *reinterpret_cast<int4 *>(p.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        if (p.seqs) *reinterpret_cast<int4 *>(p.seqs + r0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
    } else {
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (r0 + u < p.n_rows) {
                p.slots[r0 + u] = s[u];
                if (p.positions) p.positions[r0 + u] = pos[u];
                if (p.seqs) p.seqs[r0 + u] = seq[u];
            }
    }
}

// One CTA of 256 threads for a decoding batch (CLUSTER false), else a cluster of larger ones.
template <int kPlanThreads, bool CLUSTER>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p)
{
    constexpr int kPlanWarps = kPlanThreads / 32;
    auto sync_all = [] {
        if constexpr (CLUSTER) cluster_sync();
        else __syncthreads();
    };
    auto peek = [](const uint32_t &x, int c) {   // CTA c's copy of a shared variable
        if constexpr (CLUSTER) return cluster_ld(cluster_addr(static_cast<uint32_t>(__cvta_generic_to_shared(&x)), c));
        else return x;
    };
    // this CTA's sequences: lengths, and exclusive sums of what they return and take (one more: the total);
    // afterwards the row offsets of all sequences
    extern __shared__ uint32_t plan_smem[];
    __shared__ PlanSum warp_sum[kPlanWarps], total;   // total: this CTA's
    __shared__ uint2 granted;                         // the largest sums (blocks, rows) of this CTA that are not over
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int C = CLUSTER ? kPlanCluster : 1;
    const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
    const int per = (p.B + C - 1) / C;
    const int b0 = min(p.B, rank * per), nb = min(p.B, b0 + per) - b0;
    uint32_t *s_len = plan_smem, *s_new = s_len + per, *s_rel = s_new + per, *s_grow = s_rel + per + 1,
             *s_tok = s_grow + per + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");

    const int raw_count = *p.count;
    const int64_t most = static_cast<int64_t>(p.max_blocks) * p.bs;
    auto blocks_of = [&](uint32_t n) { return (n + static_cast<uint32_t>(p.bs) - 1u) / static_cast<uint32_t>(p.bs); };

    // ---- what each sequence asks for, and exclusive sums inside the CTA
    PlanSum carry{0u, 0u, 0u};
    for (int base = 0; base < nb; base += kPlanThreads) {
        const int i = base + tid;
        PlanSum x{0u, 0u, 0u};
        if (i < nb) {
            const int len = p.lens[b0 + i];
            int fresh = p.want[b0 + i];
            if (len < 0 || len > most || fresh < 0 || fresh > most) {
                atomicOr(p.err, KVC_EBIT_RANGE);
                fresh = len;   // stays as it is
            }
            s_len[i] = static_cast<uint32_t>(len);
            s_new[i] = static_cast<uint32_t>(fresh);
            if (fresh > len) {
                x.tok = static_cast<uint32_t>(fresh - len);
                x.grow = blocks_of(fresh) - blocks_of(len);
            } else if (fresh < len) {
                x.rel = blocks_of(len) - blocks_of(fresh);
            }
        }
        PlanSum inc = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const PlanSum y{__shfl_up_sync(kFull, inc.rel, o), __shfl_up_sync(kFull, inc.grow, o),
                            __shfl_up_sync(kFull, inc.tok, o)};
            if (lane >= o) inc = inc + y;
        }
        if (lane == 31) warp_sum[warp] = inc;
        __syncthreads();
        PlanSum before = carry, all = carry;
        const int used = min(kPlanWarps, (nb - base + 31) / 32);
        for (int w = 0; w < used; ++w) {
            if (w < warp) before = before + warp_sum[w];
            all = all + warp_sum[w];
        }
        // the sum up to the lane before: saturated sums cannot be taken back, so it is passed on
        PlanSum up{__shfl_up_sync(kFull, inc.rel, 1), __shfl_up_sync(kFull, inc.grow, 1), __shfl_up_sync(kFull, inc.tok, 1)};
        if (lane == 0) up = PlanSum{0u, 0u, 0u};
        const PlanSum ex = before + up;
        if (i < nb) {
            s_rel[i] = ex.rel;
            s_grow[i] = ex.grow;
            s_tok[i] = ex.tok;
        }
        carry = all;
        __syncthreads();
    }
    if (tid == 0) {
        s_rel[nb] = carry.rel;
        s_grow[nb] = carry.grow;
        s_tok[nb] = carry.tok;
        total = carry;
        granted = make_uint2(0u, 0u);
    }
    sync_all();

    // ---- sums of the CTAs before this one, and in all
    PlanSum first{0u, 0u, 0u}, whole{0u, 0u, 0u}, of[C];
#pragma unroll
    for (int c = 0; c < C; ++c) of[c] = PlanSum{peek(total.rel, c), peek(total.grow, c), peek(total.tok, c)};
#pragma unroll
    for (int c = 0; c < C; ++c) {
        if (c < rank) first = first + of[c];
        whole = whole + of[c];
    }
    const uint32_t count = static_cast<uint32_t>(min(max(raw_count, 0), p.capacity));
    if (rank == 0 && tid == 0 && (raw_count != static_cast<int>(count) || add_sat(count, whole.rel) > static_cast<uint32_t>(p.capacity)))
        atomicOr(p.err, KVC_EBIT_RANGE);
    const uint32_t avail = min(add_sat(count, whole.rel), static_cast<uint32_t>(p.capacity));
    const uint32_t rows = static_cast<uint32_t>(p.n_rows);
    auto over = [&](int i) {   // whether the sums up to and including this CTA's sequence i - 1 are over the limit
        return add_sat(first.grow, s_grow[i]) > avail || add_sat(first.tok, s_tok[i]) > rows;
    };
    for (int i = tid; i <= nb; i += kPlanThreads)
        if (!over(i) && (i == nb || over(i + 1)))   // at most one i of the CTA
            granted = make_uint2(add_sat(first.grow, s_grow[i]), add_sat(first.tok, s_tok[i]));

    // ---- push what sequences return
    for (uint32_t x0 = 4u * tid; x0 < s_rel[nb]; x0 += 4u * kPlanThreads) {   // four neighbours a thread, one search
        const uint32_t n = min(4u, s_rel[nb] - x0);
        int i = find_run(s_rel, nb, x0);
        int32_t blk[4];
#pragma unroll
        for (uint32_t u = 0; u < 4u; ++u) {
            while (u < n && x0 + u >= s_rel[i + 1]) ++i;
            blk[u] = 0;
            if (u < n) blk[u] = p.bt[static_cast<int64_t>(b0 + i) * p.max_blocks + blocks_of(s_new[i]) + (x0 + u - s_rel[i])];
        }
#pragma unroll
        for (uint32_t u = 0; u < 4u; ++u) {
            if (u >= n) break;
            if (blk[u] < 0 || blk[u] >= p.N) atomicOr(p.err, KVC_EBIT_BAD_BLOCK);
            const uint32_t at = add_sat(add_sat(count, first.rel), x0 + u);
            if (at < static_cast<uint32_t>(p.capacity)) p.stack[at] = blk[u];
        }
    }
    sync_all();

    // ---- lengths, row offsets, and blocks for those that grow
    uint32_t blocks_in_all = 0u, rows_in_all = 0u;
    uint2 got[C];
#pragma unroll
    for (int c = 0; c < C; ++c) got[c] = make_uint2(peek(granted.x, c), peek(granted.y, c));
#pragma unroll
    for (int c = 0; c < C; ++c) {
        blocks_in_all = max(blocks_in_all, got[c].x);
        rows_in_all = max(rows_in_all, got[c].y);
    }
    for (int i = tid; i < nb; i += kPlanThreads) {
        const bool refused = over(i + 1);
        const int b = b0 + i;
        p.lens_out[b] = static_cast<int32_t>(refused && static_cast<int32_t>(s_new[i]) > static_cast<int32_t>(s_len[i]) ? s_len[i] : s_new[i]);
        p.cu[b + 1] = static_cast<int32_t>(refused ? rows_in_all : add_sat(first.tok, s_tok[i + 1]));
    }
    if (rank == 0 && tid == 0) {
        p.cu[0] = 0;
        *p.count_out = static_cast<int32_t>(avail - blocks_in_all);   // every CTA has read the count by now
    }
    const uint32_t mine = blocks_in_all > first.grow ? min(s_grow[nb], blocks_in_all - first.grow) : 0u;
    for (uint32_t x0 = 4u * tid; x0 < mine; x0 += 4u * kPlanThreads) {
        const uint32_t n = min(4u, mine - x0);
        int32_t blk[4];
#pragma unroll
        for (uint32_t u = 0; u < 4u; ++u) blk[u] = u < n ? __ldcg(p.stack + (avail - 1u - first.grow - x0 - u)) : 0;
        int i = find_run(s_grow, nb, x0);
#pragma unroll
        for (uint32_t u = 0; u < 4u; ++u) {
            if (u >= n) break;
            while (x0 + u >= s_grow[i + 1]) ++i;
            p.bt[static_cast<int64_t>(b0 + i) * p.max_blocks + blocks_of(s_len[i]) + (x0 + u - s_grow[i])] = blk[u];
        }
    }
    sync_all();

    if (!p.rows_here) return;   // no CTA reads another's shared memory after the barrier above

    // ---- rows, four at a time
    uint32_t *cu = plan_smem;
    for (int i = tid; i <= p.B; i += kPlanThreads) cu[i] = static_cast<uint32_t>(__ldcg(p.cu + i));
    __syncthreads();
    const bool wide = maps_aligned(p);
    for (int64_t r0 = 4ll * (rank * kPlanThreads + tid); r0 < p.n_rows; r0 += 4ll * C * kPlanThreads) {
        write_rows(p, r0, rows_in_all, cu, 0, p.B, wide);
    }
}

constexpr int kRowsThreads = 256;
constexpr int kRowsCta = 4 * kRowsThreads;

// The maps of many rows, over the whole GPU after the cluster's kernel: a CTA finds the sequences of its 1024 rows, a
// warp narrowing the offsets by 32 at a time, and keeps their offsets in shared memory.
__global__ void __launch_bounds__(kRowsThreads) plan_rows_kernel(const PlanParams p)
{
    __shared__ uint32_t cu[kRowsCta + 1];
    __shared__ int ends[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRowsCta;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const uint32_t total = static_cast<uint32_t>(__ldcg(p.cu + p.B));
    int b0 = 0, n = 0;
    const uint32_t *offsets = cu;
    if (r0 < total) {   // the same for the whole CTA
        if (warp < 2) {
            const uint32_t r = warp == 0 ? static_cast<uint32_t>(r0) : min(static_cast<uint32_t>(r0) + kRowsCta - 1u, total - 1u);
            int lo = 0, hi = p.B;   // cu[lo] <= r < cu[hi]
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) / 32, at = lo + lane * step;
                const uint32_t m = __ballot_sync(kFull, at < hi && static_cast<uint32_t>(__ldcg(p.cu + min(at, hi))) <= r);
                lo += (31 - __clz(m)) * step;   // lane 0's offset is not above r
                hi = min(hi, lo + step);
            }
            if (lane == 0) ends[warp] = lo;
        }
        __syncthreads();
        b0 = ends[0];
        n = ends[1] - b0 + 1;
        if (n <= kRowsCta) {
            for (int i = tid; i <= n; i += kRowsThreads) cu[i] = static_cast<uint32_t>(__ldcg(p.cu + b0 + i));
            __syncthreads();
        } else {   // many sequences without rows among them
            offsets = reinterpret_cast<const uint32_t *>(p.cu) + b0;
        }
    }
    if (r0 + 4 * tid < p.n_rows) write_rows(p, r0 + 4 * tid, total, offsets, b0, n, maps_aligned(p));
}

template <int THREADS, bool CLUSTER>
static kvc_status launch_plan(const PlanParams &p, cudaStream_t stream)
{
    constexpr int C = CLUSTER ? kPlanCluster : 1;
    constexpr int kPer = CLUSTER ? kPlanMost / C : 512;   // sequences of a CTA at most
    constexpr int kSmem = 4 * (5 * kPer + 3 > kPer * C + 1 ? 5 * kPer + 3 : kPer * C + 1);
    struct Tag {};
    const DecodeKernel k = configured<Tag>(reinterpret_cast<const void *>(&plan_kernel<THREADS, CLUSTER>), kSmem, THREADS, false);
    if (k.ctas_per_sm <= 0) return KVC_ERR_CUDA;
    const int per = (p.B + C - 1) / C;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = static_cast<size_t>(4) * std::max(5 * per + 3, p.B + 1);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, plan_kernel<THREADS, CLUSTER>, p);
    if (e != cudaSuccess) return cuda_status(e);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return KVC_OK;
}

// Rows that the cluster's eight SMs write themselves; more go to a kernel of their own.
constexpr int kRowsHere = 8192;

static kvc_status launch_rows(const PlanParams &p, cudaStream_t stream)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((p.n_rows + kRowsCta - 1) / kRowsCta));
    cfg.blockDim = dim3(kRowsThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, plan_rows_kernel, p);
    if (e != cudaSuccess) return cuda_status(e);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    return KVC_OK;
}

static bool aligned4(const void *ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 3) == 0; }

}  // namespace kvc

using namespace kvc;

extern "C" kvc_status kvc_plan_step(kvc_pool *pool, int32_t *block_tables, int32_t max_blocks, const int32_t *seq_lens,
                                    const int32_t *new_lens, int32_t B, int32_t *free_list, int64_t free_capacity,
                                    const int32_t *free_count, int32_t *lens_out, int32_t *count_out,
                                    int32_t *cu_tokens, int32_t *slots, int32_t *positions, int32_t *seq_ids,
                                    int64_t n_rows, kvc_stream_t stream)
{
    if (!pool || B < 0 || n_rows < 0 || n_rows > 0x7FFFFFF0 || max_blocks < 0) return KVC_ERR_ARG;
    if (B > 0 && (max_blocks == 0 || !block_tables || !seq_lens || !new_lens || !lens_out)) return KVC_ERR_ARG;
    if (!free_list || !free_count || !count_out || !cu_tokens || (n_rows > 0 && !slots)) return KVC_ERR_ARG;
    if (free_capacity < pool->N || free_capacity > 0x7FFFFFF0) return KVC_ERR_ARG;
    const void *all[] = {block_tables, seq_lens, new_lens, free_list, free_count, lens_out, count_out, cu_tokens, slots, positions, seq_ids};
    for (const void *a : all)
        if (!aligned4(a)) return KVC_ERR_ARG;
    if (B > kPlanMost) return KVC_ERR_UNSUPPORTED;
    const kvc_status st = check_device(pool);
    if (st != KVC_OK) return st;
    PlanParams p{};
    p.bt = block_tables;
    p.max_blocks = max_blocks;
    p.lens = seq_lens;
    p.want = new_lens;
    p.B = B;
    p.bs = pool->bs;
    p.N = pool->N;
    p.stack = free_list;
    p.capacity = static_cast<int32_t>(free_capacity);
    p.count = free_count;
    p.lens_out = lens_out;
    p.count_out = count_out;
    p.cu = cu_tokens;
    p.slots = slots;
    p.positions = positions;
    p.seqs = seq_ids;
    p.n_rows = static_cast<int32_t>(n_rows);
    p.err = pool->err;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool one = B <= 512 && n_rows <= 1024;   // 1024 rows are one pass of 256 threads
    p.rows_here = n_rows <= kRowsHere;
    const kvc_status planned = one ? launch_plan<256, false>(p, s) : launch_plan<512, true>(p, s);
    return planned != KVC_OK || p.rows_here ? planned : launch_rows(p, s);
}
