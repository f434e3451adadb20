// dg_i8_linear.cu -- the linear on 8-bit integer weights and activations with a scale for each
// weight row and each token (dg_gemv_i8_rowscale).
//
// sm_103a has no integer tcgen05.mma, and its warp-level integer MMA and dp4a run at 250
// multiply-adds a clock and SM (f16: mma.sync 1020, tcgen05 4096; measured), so the codes are multiplied as
// binary16 numbers, exactly (dg_i8.cuh).  The activations are quantised to binary16 codes
// ahead (i8_quant_kernel); the weights stay bytes until they are in the SM.
//
// Swap-AB: a CTA owns a tile of 128 weight rows (the MMA's M), a group of up to MP tokens (its
// N) and a range of 128-element blocks of K.
//   warp 0      streams the weights: 128 x 128 bytes a stage by TMA (128-byte swizzle)
//   warp 1      allocates tensor memory; one elected lane issues tcgen05.mma, 8 of K = 16 a block
//   warps 2-5   convert: a lane takes one weight row's 128 bytes from shared memory, turns
//               them into binary16 and stores them in tensor memory, where the MMA reads A
//               (two buffers of 64 columns)
//   warps 6-9   epilogue: every 1024 elements the accumulator (two of them) is taken out of tensor
//               memory, as integers, and added up; then scaled and stored, or folded
//   warp 10     streams the activations: two MP x 64 boxes of binary16 a stage
// The CTAs of a K split form a cluster: each parks its integers in shared memory, and each folds a
// share of the tokens over all ranks.
// Every wait is bounded: on timeout the kernel flags DG_DEVERR_WAIT_TIMEOUT and winds down.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "dg_i8.cuh"
#include "dg_internal.h"
#include "dg_tc_common.cuh"

namespace dg {
namespace {

constexpr int kTileRows = 128;                     // MMA M
constexpr int kBlock = 128;                        // K elements a stage: one swizzled row of bytes
constexpr int kWBox = kTileRows * kBlock;          // 16 KB
constexpr int kThreads = 352;
constexpr int kMaxRanks = 8;
constexpr int kSegBlocks = i8::kSegment / kBlock;
constexpr int kACols = kBlock / 2;                 // tensor-memory columns of a converted block

struct I8Args {
    int N, K, M;
    int nsplit, nkb, groups;
    int sw_stages, sx_stages;
    const float* sx;                               // [M], written ahead
    const float* sw;                               // [N]
    uint16_t* y;
    uint8_t* ws;
};

__device__ __forceinline__ void cluster_sync_all()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t map_to_rank(uint32_t local_addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local_addr), "r"(rank));
    return r;
}

__device__ __forceinline__ int4 ld_dsmem_s32x4(uint32_t addr)
{
    int4 v;
    asm("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// kind::f16 with binary16 A (tensor memory) and B (shared memory), fp32 accumulate, M = 128, N = n.
__host__ __device__ constexpr uint32_t idesc_f16(int n)
{
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

__device__ __forceinline__ void mma_f16_ta(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Four consecutive rows n.. of token t.
__device__ __forceinline__ void store4(const I8Args& a, int t, int n, int4 v, float sx)
{
    uint16_t* dst = a.y + static_cast<size_t>(t) * a.N + n;
    const int s[4] = {v.x, v.y, v.z, v.w};
    if (n + 3 < a.N && (a.N % 4) == 0) {
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = i8::output(s[i], sx, a.sw[n + i]);
        *reinterpret_cast<uint2*>(dst) = make_uint2(h[0] | (static_cast<uint32_t>(h[1]) << 16), h[2] | (static_cast<uint32_t>(h[3]) << 16));
    } else {
        for (int i = 0; i < 4; ++i)
            if (n + i < a.N) dst[i] = i8::output(s[i], sx, a.sw[n + i]);
    }
}

template <int MP>
__global__ void __launch_bounds__(kThreads, MP <= 32 ? 2 : 1)
    i8_tc_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, I8Args a)
{
    constexpr int kXBox = MP * 128, kXStage = 2 * kXBox;
    constexpr uint32_t kA0 = 2 * MP < 64 ? 64 : 2 * MP;             // first column of the converted blocks
    constexpr uint32_t kCols = MP <= 64 ? 256 : 512;               // two accumulators, two converted blocks
    static_assert(kA0 + 2 * kACols <= kCols, "tensor memory");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int SW = a.sw_stages, SX = a.sx_stages;
    uint8_t* xring = smem + SW * kWBox;
    float* sxs = reinterpret_cast<float*>(xring + SX * kXStage);    // [MP]
    uint64_t* bars = reinterpret_cast<uint64_t*>(sxs + MP);
    const int nbars = 2 * SW + 2 * SX + 8;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + nbars);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
    const uint32_t wfull = tc::su32(bars), wempty = wfull + 8 * SW, xfull = wempty + 8 * SW, xempty = xfull + 8 * SX;
    const uint32_t afull = xempty + 8 * SX, aempty = afull + 16, dfull = aempty + 16, dempty = dfull + 16;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool clustered = a.nsplit > 1;
    const int split = clustered ? static_cast<int>(cluster_rank()) : 0;
    const int unit = static_cast<int>(blockIdx.x) / a.nsplit;
    // groups of one tile run side by side, so the tile's weights come from memory once
    const int tile = unit / a.groups, group = unit - tile * a.groups;
    const int t0 = group * MP, rows_here = min(MP, a.M - t0);
    const int kb0 = static_cast<int>(static_cast<long long>(split) * a.nkb / a.nsplit);
    const int nkb = static_cast<int>(static_cast<long long>(split + 1) * a.nkb / a.nsplit) - kb0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < SW; ++s) {
            tc::bar_init(wfull + 8 * s, 1);
            tc::bar_init(wempty + 8 * s, 4);                        // one per converting warp
        }
        for (int s = 0; s < SX; ++s) {
            tc::bar_init(xfull + 8 * s, 1);
            tc::bar_init(xempty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            tc::bar_init(afull + 8 * b, 4);
            tc::bar_init(aempty + 8 * b, 1);
            tc::bar_init(dfull + 8 * b, 1);
            tc::bar_init(dempty + 8 * b, 4);                        // one per epilogue warp
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::su32(tmem_holder)),
                     "r"(kCols));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_launch_dependents();

    // After a wait that ran out: the copies in flight of a ring whose last `issued` loads went round
    // `stages` slots are waited for, again with a limit, before the CTA may leave.
    auto drain = [&](uint32_t full, int issued, int stages) {
        volatile int own = 0;
        for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
            tc::bar_wait_for(full + 8 * (i % stages), static_cast<uint32_t>(i / stages) & 1u, &own, 100000000ull);
    };

    const int q = warp & 3;                                         // tensor-memory lane quarter
    const uint32_t tlane = tmem + (static_cast<uint32_t>(q * 32) << 16);
    int tot[MP];
    if (warp == 0) {
        if (tc::elect_one()) {
            const uint64_t once = a.groups == 1 ? tc::policy_evict_first() : 0;
            int i = 0;
            for (; i < nkb; ++i) {                                  // weights: nothing to wait for
                const int s = i % SW;
                if (i >= SW && !tc::bar_wait(wempty + 8 * s, static_cast<uint32_t>(i / SW - 1) & 1u, abort_flag)) break;
                tc::bar_expect_tx(wfull + 8 * s, kWBox);
                if (a.groups == 1)
                    tc::tma_2d_hint(tc::su32(smem + s * kWBox), &tmW, (kb0 + i) * kBlock, tile * kTileRows, wfull + 8 * s, once);
                else
                    tc::tma_2d(tc::su32(smem + s * kWBox), &tmW, (kb0 + i) * kBlock, tile * kTileRows, wfull + 8 * s);
            }
            if (*abort_flag) drain(wfull, i, SW);
        }
        pdl_wait();
    } else if (warp == 10) {
        pdl_wait();
        if (tc::elect_one()) {
            int i = 0;
            for (; i < nkb; ++i) {
                const int s = i % SX;
                if (i >= SX && !tc::bar_wait(xempty + 8 * s, static_cast<uint32_t>(i / SX - 1) & 1u, abort_flag)) break;
                const uint32_t dst = tc::su32(xring + s * kXStage);
                tc::bar_expect_tx(xfull + 8 * s, kXStage);
                tc::tma_2d(dst, &tmX, (kb0 + i) * kBlock, t0, xfull + 8 * s);
                tc::tma_2d(dst + kXBox, &tmX, (kb0 + i) * kBlock + 64, t0, xfull + 8 * s);
            }
            if (*abort_flag) drain(xfull, i, SX);
        }
    } else if (warp == 1) {
        if (tc::elect_one()) {
            for (int i = 0; i < nkb; ++i) {
                const int s = i % SX, b = i & 1, seg = i / kSegBlocks, d = seg & 1, in = i % kSegBlocks;
                if (!tc::bar_wait(xfull + 8 * s, static_cast<uint32_t>(i / SX) & 1u, abort_flag)) break;
                if (!tc::bar_wait(afull + 8 * b, static_cast<uint32_t>(i / 2) & 1u, abort_flag)) break;
                if (in == 0 && seg >= 2 && !tc::bar_wait(dempty + 8 * d, static_cast<uint32_t>(seg / 2 - 1) & 1u, abort_flag)) break;
                tc::fence_after();
                const uint64_t x0 = tc::sw128_desc(tc::su32(xring + s * kXStage));
#pragma unroll
                for (int kk = 0; kk < kBlock / 16; ++kk)
                    mma_f16_ta(tmem + static_cast<uint32_t>(d * MP), tmem + kA0 + static_cast<uint32_t>(b * kACols + kk * 8),
                               x0 + static_cast<uint64_t>((kk / 4) * (kXBox / 16) + (kk % 4) * 2), idesc_f16(MP), (in > 0 || kk > 0) ? 1u : 0u);
                tc::commit(xempty + 8 * s);
                tc::commit(aempty + 8 * b);
                if (in == kSegBlocks - 1 || i == nkb - 1) tc::commit(dfull + 8 * d);
            }
        }
        pdl_wait();
    } else if (warp < 6) {
        // Convert: this lane's weight row, 16 bytes at a time from their swizzled places.
        const int row = q * 32 + lane;
        for (int i = 0; i < nkb; ++i) {
            const int s = i % SW, b = i & 1;
            if (!tc::bar_wait(wfull + 8 * s, static_cast<uint32_t>(i / SW) & 1u, abort_flag)) break;
            const uint8_t* src = smem + s * kWBox;
            uint4 raw[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) raw[c] = *reinterpret_cast<const uint4*>(src + tc::sw128_offset(row, c));
            if (i >= 2 && !tc::bar_wait(aempty + 8 * b, static_cast<uint32_t>(i / 2 - 1) & 1u, abort_flag)) break;
            tc::fence_after();
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                uint32_t v[16];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const uint4 r = raw[2 * h + c];
                    i8::to_halves(r.x, v[8 * c], v[8 * c + 1]);
                    i8::to_halves(r.y, v[8 * c + 2], v[8 * c + 3]);
                    i8::to_halves(r.z, v[8 * c + 4], v[8 * c + 5]);
                    i8::to_halves(r.w, v[8 * c + 6], v[8 * c + 7]);
                }
                tc::tmem_st16(tlane + kA0 + static_cast<uint32_t>(b * kACols + h * 16), v);
            }
            __syncwarp();
            if (lane == 0) tc::bar_arrive(wempty + 8 * s);          // (every lane's bytes are in registers)
            tc::tmem_st_wait();
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(afull + 8 * b);
        }
        pdl_wait();
    } else {
        pdl_wait();
        for (int t = threadIdx.x - 192; t < rows_here; t += 128) sxs[t] = ld_cg_f32(a.sx + t0 + t);
        asm volatile("bar.sync 1, 128;" ::: "memory");
#pragma unroll
        for (int j = 0; j < MP; ++j) tot[j] = 0;
        const int nseg = (nkb + kSegBlocks - 1) / kSegBlocks;
        bool good = true;
#pragma unroll 1
        for (int seg = 0; seg < nseg; ++seg) {
            const int d = seg & 1;
            if (!tc::bar_wait(dfull + 8 * d, static_cast<uint32_t>(seg / 2) & 1u, abort_flag)) {
                good = false;
                break;
            }
            tc::fence_after();
#pragma unroll
            for (int c = 0; c < MP / 16; ++c) {
                uint32_t v[16];
                tc::tmem_ld16(tlane + static_cast<uint32_t>(d * MP + c * 16), v);
#pragma unroll
                for (int j = 0; j < 16; ++j) tot[c * 16 + j] += __float2int_rn(__uint_as_float(v[j]));
            }
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::bar_arrive(dempty + 8 * d);
        }
        good = good && !*abort_flag;
        const int row = q * 32 + lane, n = tile * kTileRows + row;
        if (good && !clustered) {
            // A lane holds one weight row, a warp 32 of them: 64 bytes of one token's output a store.
            const float sw = n < a.N ? a.sw[n] : 0.0f;
            uint16_t* dst = a.y + static_cast<size_t>(t0) * a.N + n;
#pragma unroll
            for (int j = 0; j < MP; ++j)
                if (j < rows_here && n < a.N) dst[static_cast<size_t>(j) * a.N] = i8::output(tot[j], sxs[j], sw);
        } else if (good) {
            int* P = reinterpret_cast<int*>(smem);                  // [token][row] in the idle weight ring
#pragma unroll
            for (int j = 0; j < MP; ++j)
                if (j < rows_here) P[j * kTileRows + row] = tot[j];
        }
    }
    if (clustered) {
        cluster_sync_all();                                         // every rank's integers are in place
        if (warp >= 6 && warp < 10 && !*abort_flag) {
            const int lo = rows_here * split / a.nsplit, hi = rows_here * (split + 1) / a.nsplit;
            uint32_t peer[kMaxRanks];
#pragma unroll
            for (int r = 0; r < kMaxRanks; ++r) peer[r] = r < a.nsplit ? map_to_rank(tc::su32(smem), r) : 0u;
            const int n = tile * kTileRows + lane * 4;
#pragma unroll 1
            for (int t = lo + warp - 6; t < hi; t += 4) {
                int4 p[kMaxRanks];
#pragma unroll
                for (int r = 0; r < kMaxRanks; ++r)
                    p[r] = r < a.nsplit ? ld_dsmem_s32x4(peer[r] + static_cast<uint32_t>((t * kTileRows + lane * 4) * 4)) : make_int4(0, 0, 0, 0);
                int4 v = p[0];
#pragma unroll
                for (int r = 1; r < kMaxRanks; ++r) v = make_int4(v.x + p[r].x, v.y + p[r].y, v.z + p[r].z, v.w + p[r].w);
                store4(a, t0 + t, n, v, sxs[t]);
            }
        }
        cluster_sync_all();                                         // no rank leaves while others read its integers
    }
    tc::fence_before();
    __syncthreads();
    if (*abort_flag && threadIdx.x == 0) set_status(a.ws, DG_DEVERR_WAIT_TIMEOUT);
    if (warp == 1) {
        tc::fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols));
    }
}

// ------------------------------------------------------------------------ host

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// 2-D tiled map, 128-byte swizzle, over bytes or binary16.
bool encode_2d(CUtensorMap* m, const void* ptr, uint64_t inner, uint64_t outer, uint32_t box_inner, uint32_t box_outer, bool half)
{
    std::call_once(g_encode_once, [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
        cudaGetLastError();
    });
    if (!g_encode) return false;
    const cuuint64_t dims[2] = {inner, outer};
    const cuuint64_t strides[1] = {inner * (half ? 2 : 1)};
    const cuuint32_t box[2] = {box_inner, box_outer};
    const cuuint32_t estr[2] = {1, 1};
    return g_encode(m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr),
                    dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

const void* kernel_of(int mp)
{
    switch (mp) {
    case 16: return reinterpret_cast<const void*>(&i8_tc_kernel<16>);
    case 32: return reinterpret_cast<const void*>(&i8_tc_kernel<32>);
    case 64: return reinterpret_cast<const void*>(&i8_tc_kernel<64>);
    case 128: return reinterpret_cast<const void*>(&i8_tc_kernel<128>);
    default: return nullptr;
    }
}

size_t smem_bytes(int mp, int sw, int sx)
{
    return 1024 + static_cast<size_t>(sw) * kWBox + static_cast<size_t>(sx) * mp * 256 + mp * 4 + (2 * sw + 2 * sx + 8) * 8 + 16;
}

}  // namespace

size_t i8_workspace_bytes(int M, int K)
{
    return kWsData + (static_cast<size_t>(M) * K * 2 + 255) / 256 * 256 + (static_cast<size_t>(M) * 4 + 255) / 256 * 256;
}

dg_status launch_i8_linear(const DeviceInfo* dev, const dg_choice& c, const void* x, const void* Wq, const float* sw, void* y,
                           int M, int N, int K, void* ws, size_t ws_bytes, cudaStream_t stream)
{
    if (ws_bytes < i8_workspace_bytes(M, K)) return DG_ERR_WORKSPACE_TOO_SMALL;
    for (int i = 0; i < 6; ++i)
        if (c.params[i] < 0 || (i > 2 && c.params[i] != 0)) return DG_ERR_BAD_VARIANT;
    const int tiles = (N - 1) / kTileRows + 1, nkb = (K - 1) / kBlock + 1;
    const int mp = c.params[1] > 0 ? c.params[1] : (M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128);
    const void* fn = kernel_of(mp);
    if (!fn) return DG_ERR_BAD_VARIANT;
    const int groups = (M - 1) / mp + 1;
    int ns = c.params[2];
    if (ns == 0) {
        const bool two = mp <= 32;
        const long long units = static_cast<long long>(tiles) * groups;
        ns = 1;
        for (int r = 2; r <= kMaxRanks && 2 * r <= nkb; ++r)
            if (units <= tc_cluster_capacity(dev, two, r)) ns = r;
    }
    if (ns < 1 || ns > kMaxRanks) return DG_ERR_BAD_VARIANT;
    if (ns > nkb) ns = nkb;
    const long long grid = static_cast<long long>(tiles) * groups * ns;
    if (grid > 0x7fffffffll) return DG_ERR_UNSUPPORTED_SHAPE;
    const int stw = c.params[0] > 0 ? c.params[0] : mp <= 64 ? 5 : 4, stx = mp <= 16 ? 4 : 3;
    if (stw < 2 || stw > 8) return DG_ERR_BAD_VARIANT;
    if (ns > 1 && static_cast<size_t>(stw) * kWBox < static_cast<size_t>(mp) * kTileRows * 4) return DG_ERR_BAD_VARIANT;
    size_t smem = smem_bytes(mp, stw, stx);
    // Never more CTAs on an SM than its 512 tensor-memory columns hold.
    const size_t least = mp <= 64 ? 77 * 1024 : 115 * 1024;
    if (smem < least) smem = least;
    if (smem > kMaxDynSmem) return DG_ERR_BAD_VARIANT;
    if (occupancy(fn, kThreads, smem) < 1) return DG_ERR_UNSUPPORTED_SHAPE;
    uint8_t* qws = static_cast<uint8_t*>(ws) + kWsData;
    float* sxws = reinterpret_cast<float*>(qws + (static_cast<size_t>(M) * K * 2 + 255) / 256 * 256);
    I8Args a{};
    a.N = N;
    a.K = K;
    a.M = M;
    a.nsplit = ns;
    a.nkb = nkb;
    a.groups = groups;
    a.sw_stages = stw;
    a.sx_stages = stx;
    a.sx = sxws;
    a.sw = sw;
    a.y = static_cast<uint16_t*>(y);
    a.ws = static_cast<uint8_t*>(ws);
    CUtensorMap tmW, tmX;
    if (!encode_2d(&tmW, Wq, static_cast<uint64_t>(K), static_cast<uint64_t>(N), kBlock, kTileRows, false) ||
        !encode_2d(&tmX, qws, static_cast<uint64_t>(K), static_cast<uint64_t>(M), 64, static_cast<uint32_t>(mp), true))
        return DG_ERR_CUDA;
    const dg_status st = launch_i8_quant(dev, true, x, qws, sxws, M, K, true, stream);
    if (st != DG_OK) return st;
    void* args[] = {&tmW, &tmX, &a};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ns);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    if (launch_ordered(cfg, attr, 1, fn, args, Early::kWeights) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
