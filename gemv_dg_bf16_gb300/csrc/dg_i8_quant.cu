// dg_i8_quant.cu -- rows of bf16 to 8-bit integer codes with one scale a row
// (dg_quant_i8_rowscale, and ahead of dg_gemv_i8_rowscale with the codes as binary16, in tiles).
//
// W warps share a row and hold it in registers, 16 bytes a lane and load: one pass over
// memory, the maximum by shuffles (and shared memory where W > 1), the codes from the registers.
// Rows longer than 16 * 4096 elements are read again for the codes.  A warp a row where the rows
// fill the GPU; few rows take four warps each, whose loads are then a quarter as many in a line.
// Bytes bind many rows: 24576 x 4096 takes 44.8 us with outputs in turn over 400 MB, 6.74 TB/s of reads and writes
// together (a copy's 6.69 are half writes, these a third).  128 KB of loads in flight an SM are best: a warp has 16 of
// them in four CTAs of 104 registers (in five CTAs of 96 it took 48.8), or 8 where that is a row of 2048 (24576 x 2048:
// 23.6 us in turn, into one output 19.3, most of which then stays in L2; with 16 27.5).  Few rows are a launch and a
// chain of latencies: 16 x 4096 1.8 us.
#include "dg_i8.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

struct QuantArgs {
    const uint16_t* x;
    uint8_t* q;                             // int8 codes [M, K], or binary16 codes in tiles
    float* s;
    int M, K, early;
    int mp;                                 // tiles: tokens of a group
};

// Eight codes of a row from element k on.  Tiles are what the linear loads at once (i8::tile_offset).
template <bool HALF>
__device__ __forceinline__ void put8(const QuantArgs& a, long long row, int k, uint4 v, const i8::RowScale& o)
{
    if constexpr (HALF)
        *reinterpret_cast<uint4*>(a.q + i8::tile_offset(static_cast<int>(row), k, a.mp, a.K)) = i8::halves8(v, o);
    else
        *reinterpret_cast<uint2*>(a.q + row * a.K + k) = i8::codes8(v, o);
}

// kVec: 16-byte loads a thread holds.
template <int W, int kVec, bool HALF>
__global__ void __launch_bounds__(W < 4 ? 128 : W * 32) i8_quant_kernel(QuantArgs a)
{
    constexpr int kRows = W < 4 ? 4 / W : 1;                    // rows per CTA
    __shared__ uint32_t part[W];
    if (a.early) pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = static_cast<long long>(blockIdx.x) * kRows + warp / W;
    if (row >= a.M) return;                                     // (W > 1: a CTA has one row)
    const int nv = a.K / 8, first = (warp % W) * 32 + lane;
    const uint16_t* x = a.x + row * a.K;
    uint4 raw[kVec];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = first + i * W * 32;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (v < nv) raw[i] = ld_stream_after(x + 8 * static_cast<size_t>(v));
    }
#pragma unroll
    for (int i = 0; i < kVec; ++i) m = __vmaxu2(m, i8::amax8(raw[i]));
#pragma unroll 1
    for (int v = first + kVec * W * 32; v < nv; v += W * 32)
        m = __vmaxu2(m, i8::amax8(ld_stream_after(x + 8 * static_cast<size_t>(v))));
    m = max(m & 0xffffu, m >> 16);
    m = __reduce_max_sync(kFull, m);
    if constexpr (W > 1) {
        if (lane == 0) part[warp] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) m = max(m, part[i]);
    }
    const i8::RowScale o = i8::row_scale(m);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int v = first + i * W * 32;
        if (v < nv) put8<HALF>(a, row, 8 * v, raw[i], o);
    }
#pragma unroll 1
    for (int v = first + kVec * W * 32; v < nv; v += W * 32)
        put8<HALF>(a, row, 8 * v, ld_stream_after(x + 8 * static_cast<size_t>(v)), o);
    if constexpr (HALF)                                         // zeros to the end of the last block
        for (int v = nv + first; v < (a.K + 127) / 128 * 16; v += W * 32) put8<true>(a, row, 8 * v, make_uint4(0, 0, 0, 0), o);
    if (first == 0) a.s[row] = o.s;
}

template <bool HALF>
const void* quant_fn(int w, int K)
{
    if (w == 16) return reinterpret_cast<const void*>(&i8_quant_kernel<16, 16, HALF>);
    if (w == 4) return reinterpret_cast<const void*>(&i8_quant_kernel<4, 16, HALF>);
    if constexpr (!HALF)                                        // (the linear has too few rows for it)
        if (K > 2048) return reinterpret_cast<const void*>(&i8_quant_kernel<1, 16, HALF>);
    return reinterpret_cast<const void*>(&i8_quant_kernel<1, 8, HALF>);
}

}  // namespace

dg_status launch_i8_quant(const DeviceInfo* dev, const void* x, void* q, float* s, int M, int K, int mp, cudaStream_t stream)
{
    int w = K <= 4096 ? 1 : K <= 16384 ? 4 : 16;
    if (w == 1 && M < 8 * dev->sm_count && K > 1024) w = 4;
    const int rows = w == 1 ? 4 : 1;
    QuantArgs a{static_cast<const uint16_t*>(x), static_cast<uint8_t*>(q), s, M, K, mp > 0, mp};
    void* args[] = {&a};
    if (launch_kernel(mp > 0 ? quant_fn<true>(w, K) : quant_fn<false>(w, K), static_cast<unsigned>((M - 1) / rows + 1),
                      w == 1 ? 128u : static_cast<unsigned>(w * 32), 0, stream, args, Early::kNothing) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
