// dg_moe_sort.cu -- (token, slot) pairs sorted by expert (dg_moe_sort), rows taken there
// (dg_moe_gather) and back with their weights (dg_moe_combine), and the gradient of the way back
// (dg_moe_combine_grad).
//
// Sort: a stable counting sort in one launch of one cluster.  Every warp of every CTA owns a
// contiguous run of the pairs.  It ranks them by expert as it goes -- __match_any_sync finds the
// lanes with the same expert, one counter per (warp, expert) in shared memory holds how many
// came before -- and leaves each rank in pos.  Then the counters become starts: over the warps of
// a CTA, over the cluster's CTAs (read through distributed shared memory) and over the experts.
// A second pass over its own pairs adds each one's start to its rank.  No atomics between warps:
// the order is that of the pairs, run to run.
//
// Rows move in 16-byte pieces, any type; a token's row is read once and written to its up to 32
// places.  On the way back a thread has the loads of eight slots in flight, and adds in slot
// order in binary32.
#include "dg_internal.h"
#include "dg_common.cuh"

namespace dg {
namespace {

constexpr int kMaxCtas = 8;              // portable cluster
constexpr int kMaxWarps = 32;
constexpr int kMaxExperts = 1024;

struct SortArgs {
    const int32_t* ids;
    int32_t *offsets, *pos, *slots;
    int n, topk, E;                      // n = M * topk pairs
    int run;                             // pairs per warp, a multiple of 32
};

__device__ __forceinline__ uint32_t ctarank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ int ld_peer(const int* local, uint32_t rank)
{
    uint32_t at;
    int v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(local))), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void cluster_sync()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The expert of pair i, or -1 where its id is outside [0, E) or an earlier slot of its token has it.
__device__ __forceinline__ int expert_of(const SortArgs& a, int i)
{
    const int e = a.ids[i];
    if (e < 0 || e >= a.E) return -1;
    const int first = i / a.topk * a.topk;
    bool again = false;
    for (int j = first; j < i; ++j) again |= a.ids[j] == e;
    return again ? -1 : e;
}

__global__ void __launch_bounds__(kMaxWarps * 32, 1) moe_sort_kernel(SortArgs a)
{
    extern __shared__ int sh[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(ctarank()), ctas = gridDim.x;
    int* count = sh;                               // [warps][E]: pairs so far, then starts
    int* total = sh + warps * a.E;                 // [E]: this CTA's pairs of each expert
    int* part = total + a.E;                       // [warps]: sums of the scan over experts
    pdl_launch_dependents();
    pdl_wait();
    for (int i = threadIdx.x; i < warps * a.E; i += blockDim.x) count[i] = 0;
    __syncthreads();
    const long long begin = (static_cast<long long>(rank) * warps + warp) * a.run;
    const int lo = static_cast<int>(min(begin, static_cast<long long>(a.n))), hi = static_cast<int>(min(begin + a.run, static_cast<long long>(a.n)));
    int* mine = count + warp * a.E;
#pragma unroll 1
    for (int i0 = lo; i0 < hi; i0 += 32) {
        const int i = i0 + lane;
        const int e = i < hi ? expert_of(a, i) : -1;
        const unsigned same = __match_any_sync(kFull, e);
        const int before = e >= 0 ? mine[e] : 0;
        __syncwarp();
        if (e >= 0 && lane == 31 - __clz(same)) mine[e] = before + __popc(same);
        __syncwarp();
        if (i < hi) a.pos[i] = e >= 0 ? before + __popc(same & ((1u << lane) - 1)) : -1;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
        int sum = 0;
        for (int w = 0; w < warps; ++w) {
            const int c = count[w * a.E + e];
            count[w * a.E + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    if (ctas > 1)
        cluster_sync();
    else
        __syncthreads();
    // Experts in runs of `per` a thread: pairs in front of this CTA's, and of all CTAs.
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
    int start = scan - sum, all = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) start += part[w];
        all += part[w];
    }
    for (int e = e0; e < e1; ++e) {
        int front = start;
        for (int r = 0; r < ctas; ++r) {
            const int c = ctas > 1 ? ld_peer(total + e, r) : total[e];
            if (r < rank) front += c;
            start += c;
        }
        if (rank == 0) a.offsets[e] = front;
        for (int w = 0; w < warps; ++w) count[w * a.E + e] += front;
    }
    if (rank == 0 && threadIdx.x == 0) a.offsets[a.E] = all;
    if (ctas > 1)
        cluster_sync();                            // (no CTA leaves while others read its totals)
    else
        __syncthreads();
#pragma unroll 1
    for (int i = lo + lane; i < hi; i += 32) {
        const int r = a.pos[i];
        if (r < 0) continue;
        const int p = r + mine[a.ids[i]];
        a.pos[i] = p;
        a.slots[p] = i;
    }
    for (long long p = all + static_cast<long long>(rank) * blockDim.x + threadIdx.x; p < a.n; p += static_cast<long long>(ctas) * blockDim.x)
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
    const long long n = static_cast<long long>(M) * topk;
    const int warps = n <= 1024 ? 8 : kMaxWarps;
    int ctas = 1;
    while (ctas < kMaxCtas && n > 4096ll * ctas) ctas *= 2;
    SortArgs a{};
    a.ids = ids;
    a.offsets = offsets;
    a.pos = pos;
    a.slots = slots;
    a.n = static_cast<int>(n);
    a.topk = topk;
    a.E = E;
    const long long owners = static_cast<long long>(ctas) * warps;
    a.run = static_cast<int>(((n + owners - 1) / owners + 31) / 32 * 32);
    const void* fn = reinterpret_cast<const void*>(&moe_sort_kernel);
    const size_t smem = (static_cast<size_t>(warps) * E + E + warps) * 4;
    if (occupancy(fn, warps * 32, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    void* args[] = {&a};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(static_cast<unsigned>(warps * 32));
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
