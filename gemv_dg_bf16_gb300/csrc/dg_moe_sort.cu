// dg_moe_sort.cu -- (token, slot) pairs sorted by expert (dg_moe_sort), rows taken there
// (dg_moe_gather) and back with their weights (dg_moe_combine), and the gradient of the way back
// (dg_moe_combine_grad).
//
// Sort: a stable counting sort in one launch of one cluster, without atomics whose order would matter.  Each CTA
// owns a run of tokens and takes them in blocks of up to 1024.  A token has an expert at most once, so a
// block is a bit matrix in shared memory, tokens by experts: every live slot sets its bit, in any order, and the
// rank of a slot among its expert's in the block is the number of bits in front of its own -- a sum over whole
// words, kept for each (32 tokens, expert), and one popc.  The experts' totals go over the cluster through
// distributed shared memory, and a scan over the experts gives the starts.  (Ranks by __match_any_sync and counters a
// warp and expert took 4.1 us for 64 tokens of 6 slots and 64 us for 32768 of 8: it steps through
// the distinct values of a warp.)
//
// Measured: 64 tokens of 6 slots 2.4 us, 512 of 8 5.7, 8192 of 8 12.7, 32768 of 8 48: one cluster's blocks one after the other.
//
// Rows move in 16-byte pieces, any type; a token's row is read once and written to its up to 32
// places.  On the way back a thread has the loads of eight slots in flight, and adds in slot
// order in binary32.  Bytes bind them: rows of 4096 bf16, 8 slots: 32768 tokens there 355.6 us and back 354.5 (6.8 TB/s),
// 8192 back 90.1 and the gradient 171.9 (6.6 TB/s); 64 tokens are a launch and two loads in a row, 2.2 us.
#include "dg_internal.h"
#include "dg_tc_common.cuh"

namespace dg {
namespace {

constexpr int kMaxCtas = 8;              // portable cluster
constexpr int kMaxThreads = 1024;
constexpr int kSlotsPerCta = 2048;
constexpr int kIds = 4;                  // loads of ids in flight a thread

struct SortArgs {
    const int32_t* ids;
    int32_t *offsets, *pos, *slots;
    int M, topk, E;
    int run, block;                      // tokens of a CTA, and of one of its blocks (a multiple of 32)
    uint64_t recip;                      // 2^32 / topk, rounded up
};

__device__ __forceinline__ int ld_peer(const int* local, uint32_t rank)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(tc::map_to_rank(tc::su32(local), rank)) : "memory");
    return v;
}

// The expert of slot i, or -1 where its id is outside [0, E) or an earlier slot of its token has it.
__device__ __forceinline__ int expert_of(const SortArgs& a, int i)
{
    const int e = a.ids[i];
    const int first = i / a.topk * a.topk;
    bool live = e >= 0 && e < a.E;
#pragma unroll 8
    for (int j = first; j < i; ++j) live &= a.ids[j] != e;
    return live ? e : -1;
}

__global__ void __launch_bounds__(kMaxThreads, 1) moe_sort_kernel(SortArgs a)
{
    extern __shared__ int sh[];
    __shared__ int again;                                  // some token of a block has an expert twice
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, words = a.block / 32;
    const int rank = static_cast<int>(tc::cluster_rank()), ctas = gridDim.x;
    uint32_t* bits = reinterpret_cast<uint32_t*>(sh);      // [words][E]
    int* front = sh + words * a.E;                         // [words][E]: bits of the words in front
    int* total = front + words * a.E;                      // [E]: this CTA's slots of each expert
    int* start = total + a.E;                              // [E]: row of the next of them
    int* part = start + a.E;                               // [warps]: sums of the scan over experts
    const int t0 = min(a.M, rank * a.run), t1 = min(a.M, t0 + a.run), blocks = (t1 - t0 + a.block - 1) / a.block;
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) total[e] = 0;
    if (threadIdx.x == 0) again = 0;
    // x / topk of x < 32768: the reciprocal is rounded up, and off by less than 1 / 32768
    const auto token_of = [&](int x) { return static_cast<int>((static_cast<uint64_t>(x) * a.recip) >> 32); };
    pdl_launch_dependents();
    pdl_wait();
    // Block b's matrix, its sums in front and the experts' totals with it; which of this thread's slots are
    // live, a bit each (at most 1024 * 32 slots over 1024 threads).
    auto build = [&](int b, bool count) {
        const int lo = (t0 + b * a.block) * a.topk, hi = min(t1, t0 + (b + 1) * a.block) * a.topk;
        if (b > 0 || !count) __syncthreads();      // the block in front is read
        for (int i = threadIdx.x; i < words * a.E; i += blockDim.x) bits[i] = 0;
        __syncthreads();
        // Slots whose token has their expert twice find its bit set, whichever comes first: then every thread
        // asks for its slots in turn which are live.  (The bits are the same either way.)
        uint32_t live = 0;
        for (int i0 = lo + static_cast<int>(threadIdx.x), n0 = 0; i0 < hi; i0 += kIds * blockDim.x, n0 += kIds) {
            int e[kIds];
#pragma unroll
            for (int u = 0; u < kIds; ++u) e[u] = i0 + u * static_cast<int>(blockDim.x) < hi ? a.ids[i0 + u * blockDim.x] : -1;
#pragma unroll
            for (int u = 0; u < kIds; ++u) {
                if (e[u] < 0 || e[u] >= a.E) continue;
                const int t = token_of(i0 + u * static_cast<int>(blockDim.x) - lo);
                const uint32_t bit = 1u << (t & 31);
                if (atomicOr(bits + (t >> 5) * a.E + e[u], bit) & bit) again = 1;
                live |= 1u << (n0 + u);
            }
        }
        __syncthreads();
        if (again) {
            live = 0;
            for (int i = lo + static_cast<int>(threadIdx.x), n = 0; i < hi; i += blockDim.x, ++n)
                if (expert_of(a, i) >= 0) live |= 1u << n;
        }
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
            int sum = 0;
#pragma unroll 4
            for (int w = 0; w < words; ++w) {
                front[w * a.E + e] = sum;
                sum += __popc(bits[w * a.E + e]);
            }
            if (count) total[e] += sum;
        }
        return live;
    };
    uint32_t live = 0;
    for (int b = 0; b < blocks; ++b) live = build(b, true);
    if (ctas > 1)
        tc::cluster_sync_all();
    else
        __syncthreads();
    // Experts in runs of `per` a thread: slots of lower experts, and of this one in the CTAs in front.
    const int per = (a.E + blockDim.x - 1) / blockDim.x;
    const int e0 = min(a.E, static_cast<int>(threadIdx.x) * per), e1 = min(a.E, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e)
        for (int r = 0; r < ctas; ++r) sum += ctas > 1 ? ld_peer(total + e, r) : total[e];
    int scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(kFull, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) part[warp] = scan;
    __syncthreads();
    int row = scan - sum, all = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) row += part[w];
        all += part[w];
    }
    for (int e = e0; e < e1; ++e) {
        if (rank == 0) a.offsets[e] = row;
        for (int r = 0; r < ctas; ++r) {
            if (r == rank) start[e] = row;
            row += ctas > 1 ? ld_peer(total + e, r) : total[e];
        }
    }
    if (rank == 0 && threadIdx.x == 0) a.offsets[a.E] = all;
    if (ctas > 1)
        tc::cluster_sync_all();                            // (no CTA leaves while others read its totals)
    else
        __syncthreads();
    for (int b = 0; b < blocks; ++b) {
        if (blocks > 1) {
            live = build(b, false);
            __syncthreads();
        }
        const int lo = (t0 + b * a.block) * a.topk, hi = min(t1, t0 + (b + 1) * a.block) * a.topk;
        for (int i = lo + static_cast<int>(threadIdx.x), n = 0; i < hi; i += blockDim.x, ++n) {
            int p = -1;
            if ((live >> n) & 1u) {
                const int e = a.ids[i], t = token_of(i - lo), w = (t >> 5) * a.E + e;
                p = start[e] + front[w] + __popc(bits[w] & ((1u << (t & 31)) - 1u));
                a.slots[p] = i;
            }
            a.pos[i] = p;
        }
        if (b + 1 == blocks) break;
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += blockDim.x)
            start[e] += front[(words - 1) * a.E + e] + __popc(bits[(words - 1) * a.E + e]);
    }
    for (long long p = all + static_cast<long long>(rank) * blockDim.x + threadIdx.x; p < static_cast<long long>(a.M) * a.topk;
         p += static_cast<long long>(ctas) * blockDim.x)
        a.slots[p] = -1;
}

// ------------------------------------------------------------------------ rows

constexpr int kRowThreads = 256;
constexpr int kInFlight = 8;

struct RowArgs {
    const uint4* x;                      // gather: x [M], combine: z [P], gradient: z [P]
    const uint4* dy;                     // gradient: [M]
    uint4* out;                          // gather: xs [P], combine: y [M], gradient: dz [P]
    const int32_t* pos;                  // [M, topk]
    const float* w;                      // [M, topk] or NULL
    float* dw;                           // gradient: [M, topk]
    int M, topk, P, nv;                  // nv: 16-byte pieces of a row
    int slices;                          // pieces of kRowThreads along a row
};

__global__ void __launch_bounds__(kRowThreads) moe_gather_kernel(RowArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int t = static_cast<int>(blockIdx.x / a.slices), v = static_cast<int>(blockIdx.x % a.slices) * kRowThreads + threadIdx.x;
    if (v >= a.nv) return;
    const uint4 row = ld_stream_after(a.x + static_cast<size_t>(t) * a.nv + v);
    const int32_t* pos = a.pos + static_cast<size_t>(t) * a.topk;
    for (int k = 0; k < a.topk; ++k) {
        const int p = pos[k];
        if (p >= 0 && p < a.P) a.out[static_cast<size_t>(p) * a.nv + v] = row;
    }
}

__device__ __forceinline__ void unpack8(uint4 r, float (&f)[8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_lo(w[j]);
        f[2 * j + 1] = bf16_hi(w[j]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        memcpy(&w[j], &p, sizeof w[j]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__global__ void __launch_bounds__(kRowThreads) moe_combine_kernel(RowArgs a)
{
    pdl_launch_dependents();
    pdl_wait();
    const int t = static_cast<int>(blockIdx.x / a.slices), v = static_cast<int>(blockIdx.x % a.slices) * kRowThreads + threadIdx.x;
    if (v >= a.nv) return;
    const int32_t* pos = a.pos + static_cast<size_t>(t) * a.topk;
    const float* wt = a.w ? a.w + static_cast<size_t>(t) * a.topk : nullptr;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
#pragma unroll 1
    for (int k0 = 0; k0 < a.topk; k0 += kInFlight) {
        uint4 z[kInFlight];
        float w[kInFlight];
        bool live[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            const int k = k0 + u, p = k < a.topk ? pos[k] : -1;
            live[u] = p >= 0 && p < a.P;
            w[u] = live[u] && wt ? wt[k] : 1.0f;
            if (live[u]) z[u] = ld_stream_after(a.x + static_cast<size_t>(p) * a.nv + v);
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            if (!live[u]) continue;
            float f[8];
            unpack8(z[u], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[j] = __fmaf_rn(w[u], f[j], acc[j]);
        }
    }
    a.out[static_cast<size_t>(t) * a.nv + v] = pack8(acc);
}

// One token a CTA.  dw's sums: a thread's columns in ascending order, lanes by a butterfly, warps
// in order: a fixed order for a row length.
__global__ void __launch_bounds__(kRowThreads) moe_combine_grad_kernel(RowArgs a)
{
    __shared__ float part[kRowThreads / 32][32];
    pdl_launch_dependents();
    pdl_wait();
    const int t = static_cast<int>(blockIdx.x), warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    const int32_t* pos = a.pos + static_cast<size_t>(t) * a.topk;
    const float* wt = a.w + static_cast<size_t>(t) * a.topk;
#pragma unroll 1
    for (int k0 = 0; k0 < a.topk; k0 += kInFlight) {
        float dot[kInFlight], w[kInFlight];
        int p[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
            dot[u] = 0.0f;
            p[u] = k0 + u < a.topk ? pos[k0 + u] : -1;
            if (p[u] >= a.P) p[u] = -1;
            w[u] = p[u] >= 0 ? wt[k0 + u] : 0.0f;
        }
#pragma unroll 1
        for (int v = threadIdx.x; v < a.nv; v += blockDim.x) {
            uint4 z[kInFlight];
            const uint4 g = ld_stream_after(a.dy + static_cast<size_t>(t) * a.nv + v);
#pragma unroll
            for (int u = 0; u < kInFlight; ++u)
                if (p[u] >= 0) z[u] = ld_stream_after(a.x + static_cast<size_t>(p[u]) * a.nv + v);
            float dy[8];
            unpack8(g, dy);
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                if (p[u] < 0) continue;
                float f[8], d[8];
                unpack8(z[u], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    dot[u] = __fmaf_rn(dy[j], f[j], dot[u]);
                    d[j] = __fmul_rn(w[u], dy[j]);
                }
                a.out[static_cast<size_t>(p[u]) * a.nv + v] = pack8(d);
            }
        }
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot[u] += __shfl_xor_sync(kFull, dot[u], o);
            if (lane == 0) part[warp][k0 + u] = dot[u];
        }
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.topk; k += blockDim.x) {
        float s = 0.0f;
        for (int i = 0; i < warps; ++i) s += part[i][k];
        a.dw[static_cast<size_t>(t) * a.topk + k] = s;
    }
}

dg_status launch_rows(const void* fn, const RowArgs& a, long long grid, int threads, cudaStream_t stream)
{
    if (grid > 0x7fffffffll) return DG_ERR_UNSUPPORTED_SHAPE;
    RowArgs b = a;
    void* args[] = {&b};
    if (launch_kernel(fn, static_cast<unsigned>(grid), static_cast<unsigned>(threads), 0, stream, args, Early::kNothing) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace

dg_status launch_moe_sort(const int32_t* ids, int32_t* offsets, int32_t* pos, int32_t* slots, int M, int topk, int E,
                          cudaStream_t stream)
{
    // A block's matrix and its sums take at most 128 KB; a CTA for every 2048 slots, up to a cluster.
    SortArgs a{};
    a.ids = ids;
    a.offsets = offsets;
    a.pos = pos;
    a.slots = slots;
    a.M = M;
    a.topk = topk;
    a.E = E;
    const long long n = static_cast<long long>(M) * topk;
    int ctas = 1;
    while (ctas < kMaxCtas && n > static_cast<long long>(kSlotsPerCta) * ctas) ctas *= 2;
    a.recip = ((uint64_t{1} << 32) + topk - 1) / topk;
    a.run = (M - 1) / ctas + 1;
    a.block = 1024;
    while (a.block > 32 && (static_cast<long long>(a.block) * E > 512 * 1024 || a.block / 2 >= a.run)) a.block /= 2;
    const long long most = static_cast<long long>(a.run < a.block ? a.run : a.block) * topk;
    int threads = 128;
    while (threads < kMaxThreads && (threads < most || threads < E)) threads *= 2;
    const size_t smem = (static_cast<size_t>(a.block / 32) * E * 2 + 2 * static_cast<size_t>(E) + threads / 32) * 4;
    const void* fn = reinterpret_cast<const void*>(&moe_sort_kernel);
    if (occupancy(fn, threads, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    void* args[] = {&a};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ctas);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    if (launch_ordered(cfg, attr, 1, fn, args, Early::kNothing) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

dg_status launch_moe_gather(const void* x, const int32_t* pos, void* xs, int M, int topk, int P, int64_t row_bytes, cudaStream_t stream)
{
    RowArgs a{};
    a.x = static_cast<const uint4*>(x);
    a.out = static_cast<uint4*>(xs);
    a.pos = pos;
    a.M = M;
    a.topk = topk;
    a.P = P;
    a.nv = static_cast<int>(row_bytes / 16);
    a.slices = (a.nv - 1) / kRowThreads + 1;
    return launch_rows(reinterpret_cast<const void*>(&moe_gather_kernel), a, static_cast<long long>(M) * a.slices, kRowThreads, stream);
}

dg_status launch_moe_combine(const void* z, const int32_t* pos, const float* w, void* y, int M, int topk, int P, int N, cudaStream_t stream)
{
    RowArgs a{};
    a.x = static_cast<const uint4*>(z);
    a.out = static_cast<uint4*>(y);
    a.pos = pos;
    a.w = w;
    a.M = M;
    a.topk = topk;
    a.P = P;
    a.nv = N / 8;
    a.slices = (a.nv - 1) / kRowThreads + 1;
    return launch_rows(reinterpret_cast<const void*>(&moe_combine_kernel), a, static_cast<long long>(M) * a.slices, kRowThreads, stream);
}

dg_status launch_moe_combine_grad(const void* dy, const void* z, const int32_t* pos, const float* w, void* dz, float* dw, int M, int topk,
                                  int P, int N, cudaStream_t stream)
{
    RowArgs a{};
    a.x = static_cast<const uint4*>(z);
    a.dy = static_cast<const uint4*>(dy);
    a.out = static_cast<uint4*>(dz);
    a.pos = pos;
    a.w = w;
    a.dw = dw;
    a.M = M;
    a.topk = topk;
    a.P = P;
    a.nv = N / 8;
    const int threads = a.nv >= kRowThreads ? kRowThreads : (a.nv + 31) / 32 * 32;
    return launch_rows(reinterpret_cast<const void*>(&moe_combine_grad_kernel), a, M, threads, stream);
}

}  // namespace dg
