// dg_fp4.cu -- microscaled 4-bit quantisation and its inverse (dg_quant_fp4_blockscale,
// dg_dequant_fp4_blockscale).
//
// A CTA takes 128 rows x 256 columns: whole scale tiles, so the scattered scale bytes
// meet in shared memory and leave in 16-byte stores.  A lane holds 8 elements (one
// 16-byte load, one 4-byte store of codes); 2 (NV) or 4 (MX) lanes share a block and
// find its maximum by shuffles.  Bound: memory, 2 + 1/2 + 1/16 bytes an element.
#include "dg_fp4.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kCols = 256;                 // columns per CTA
constexpr int kThreads = 256;

// The outputs may be weights, which a linear of this library reads before it waits for the
// launches ahead of it: let the next launch begin only when this thread's stores are
// visible to the whole device, to plain loads and to bulk copies.
__device__ __forceinline__ void signal_written()
{
    __threadfence();
    asm volatile("fence.proxy.async.global;" ::: "memory");
    pdl_launch_dependents();
}

template <bool NV>
__global__ void __launch_bounds__(kThreads) fp4_quant_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ q,
                                                             uint8_t* __restrict__ s, const float* __restrict__ gp,
                                                             int M, int K, int col_tiles, int early)
{
    constexpr int kTiles = kCols / fp4::tile_k(NV);            // scale tiles per CTA
    constexpr int kShare = fp4::block_len(NV) / 8;             // lanes per block
    __shared__ uint4 sc[kTiles * fp4::kTileBytes / 16];
    if (early) pdl_launch_dependents();
    pdl_wait();
    const int rt = static_cast<int>(blockIdx.x) / col_tiles, ct = static_cast<int>(blockIdx.x) - rt * col_tiles;
    const float g = gp ? *gp : 1.0f, g6 = __fmul_rn(6.0f, g);
    for (int i = threadIdx.x; i < kTiles * fp4::kTileBytes / 16; i += kThreads) sc[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const int ch = threadIdx.x % (kCols / 8);                  // 8-element chunk of the column range
    const int k = ct * kCols + ch * 8;
    uint8_t* scb = reinterpret_cast<uint8_t*>(sc);
#pragma unroll 1
    for (int r = threadIdx.x / (kCols / 8); r < fp4::kTileRows; r += kThreads / (kCols / 8)) {
        const int row = rt * fp4::kTileRows + r;
        if (row >= M) break;                                   // the same row in all lanes of a warp
        const bool in = k < K;                                 // K % 32 == 0: a block is inside or outside
        uint4 raw = make_uint4(0, 0, 0, 0);
        if (in) raw = ld_stream_after(x + static_cast<size_t>(row) * K + k);
        uint32_t m = fp4::amax8(raw);
#pragma unroll
        for (int o = 1; o < kShare; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
        const fp4::Scale bs = fp4::block_scale<NV>(m, g6, g);
        if (in) {
            float v[8];
            fp4::unpack8(raw, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fp4::scaled<NV>(v[i], bs);
            const uint32_t codes = bs.live ? fp4::to_e2m1x8(v) : 0u;
            *reinterpret_cast<uint32_t*>(q + (static_cast<size_t>(row) * K + k) / 2) = codes;
            if (ch % kShare == 0) {
                const int b = ch / kShare;
                scb[(b / 4) * fp4::kTileBytes + fp4::tile_offset(r, b % 4)] = static_cast<uint8_t>(bs.byte);
            }
        }
    }
    __syncthreads();
    const int nkt = fp4::scale_tiles(K, NV);
    uint4* dst = reinterpret_cast<uint4*>(s + (static_cast<size_t>(rt) * nkt + ct * kTiles) * fp4::kTileBytes);
    const int n = min(kTiles, nkt - ct * kTiles) * (fp4::kTileBytes / 16);
    for (int i = threadIdx.x; i < n; i += kThreads) dst[i] = sc[i];
    if (!early) signal_written();
}

// y = bf16(code * (scale * g)), each step rounded to binary32 (MX without a g: exact).
template <bool NV>
__global__ void __launch_bounds__(kThreads) fp4_dequant_kernel(const uint8_t* __restrict__ q,
                                                               const uint8_t* __restrict__ s,
                                                               const float* __restrict__ gp, uint16_t* __restrict__ y,
                                                               int M, int K, int col_tiles)
{
    constexpr int kTiles = kCols / fp4::tile_k(NV);
    constexpr int kShare = fp4::block_len(NV) / 8;
    __shared__ uint4 sc[kTiles * fp4::kTileBytes / 16];
    pdl_wait();
    const int rt = static_cast<int>(blockIdx.x) / col_tiles, ct = static_cast<int>(blockIdx.x) - rt * col_tiles;
    const float g = gp ? *gp : 1.0f;
    const int nkt = fp4::scale_tiles(K, NV);
    const uint4* src = reinterpret_cast<const uint4*>(s + (static_cast<size_t>(rt) * nkt + ct * kTiles) * fp4::kTileBytes);
    const int n = min(kTiles, nkt - ct * kTiles) * (fp4::kTileBytes / 16);
    for (int i = threadIdx.x; i < n; i += kThreads) sc[i] = src[i];
    __syncthreads();
    const int ch = threadIdx.x % (kCols / 8);
    const int k = ct * kCols + ch * 8;
    const uint8_t* scb = reinterpret_cast<const uint8_t*>(sc);
    const int b = ch / kShare;
#pragma unroll 4
    for (int r = threadIdx.x / (kCols / 8); r < fp4::kTileRows; r += kThreads / (kCols / 8)) {
        const int row = rt * fp4::kTileRows + r;
        if (row >= M || k >= K) break;
        const uint32_t codes = *reinterpret_cast<const uint32_t*>(q + (static_cast<size_t>(row) * K + k) / 2);
        const uint32_t sb = scb[(b / 4) * fp4::kTileBytes + fp4::tile_offset(r, b % 4)];
        float f;
        if constexpr (NV)
            f = fp4::e4m3_value(sb);
        else
            f = sb == 0xffu ? __uint_as_float(0x7fffffffu) : fp4::pow2(static_cast<int>(sb) - 127);
        f = __fmul_rn(f, g);
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 v = fp4::from_e2m1x2(codes, j);
            w[j] = f32_to_bf16_bits(__fmul_rn(v.x, f)) | (static_cast<uint32_t>(f32_to_bf16_bits(__fmul_rn(v.y, f))) << 16);
        }
        *reinterpret_cast<uint4*>(y + static_cast<size_t>(row) * K + k) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    signal_written();
}

}  // namespace

dg_status launch_fp4_quant(bool nv, const void* x, void* q, void* s, const float* g, int M, int K, bool early,
                           cudaStream_t stream)
{
    int col_tiles = (K + kCols - 1) / kCols, now = early ? 1 : 0;
    const long long grid = ((static_cast<long long>(M) + fp4::kTileRows - 1) / fp4::kTileRows) * col_tiles;
    if (grid > 0x7fffffffll) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* fn = nv ? reinterpret_cast<const void*>(&fp4_quant_kernel<true>)
                        : reinterpret_cast<const void*>(&fp4_quant_kernel<false>);
    void* args[] = {&x, &q, &s, &g, &M, &K, &col_tiles, &now};
    if (launch_kernel(fn, static_cast<unsigned>(grid), kThreads, 0, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

dg_status launch_fp4_dequant(bool nv, const void* q, const void* s, const float* g, void* y, int M, int K,
                             cudaStream_t stream)
{
    int col_tiles = (K + kCols - 1) / kCols;
    const long long grid = ((static_cast<long long>(M) + fp4::kTileRows - 1) / fp4::kTileRows) * col_tiles;
    if (grid > 0x7fffffffll) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* fn = nv ? reinterpret_cast<const void*>(&fp4_dequant_kernel<true>)
                        : reinterpret_cast<const void*>(&fp4_dequant_kernel<false>);
    void* args[] = {&q, &s, &g, &y, &M, &K, &col_tiles};
    if (launch_kernel(fn, static_cast<unsigned>(grid), kThreads, 0, stream, args) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
