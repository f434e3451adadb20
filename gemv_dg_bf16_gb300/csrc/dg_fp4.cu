// dg_fp4.cu -- microscaled 4-bit quantisation and its inverse (dg_quant_fp4_blockscale,
// dg_dequant_fp4_blockscale).
//
// A warp takes 4 rows of a 256-column range, 32 rows apart, a lane 8 elements of each (one
// 16-byte and one 4-byte access); 2 (NV) or 4 (MX) lanes share a block and find its maximum
// by shuffles, and 8 or 16 lanes put together the 16 scale bytes that those rows have side
// by side in a scale tile (4-byte stores of them, one row at a time, cost 4 us on 16 rows).
// No shared memory and no barrier: every row's loads are in flight before the first is used.
// The outputs may be weights, which a linear reads before it waits for what is ahead of it: the
// entry points' kernels let no launch begin before they have completed, and note on the stream
// that weights were written (weights_written).  Inside the linear, which waits for the codes,
// the quantisation lets it begin at once (`early`).
// The inputs are not __restrict__: loads of what the launch ahead may have written must stay
// behind pdl_wait() and off the non-coherent path.
// Bound: memory, 2 + 1/2 + 1/16 (or 1/32) bytes an element and direction.  24576 x 4096 in MX:
// there 47 us and back 38, of 37.5 for the bytes each; 103 and 71 instructions for 8 elements,
// the former's conversions keeping the ALU 70 % busy.  In NV: there 63 us (a division a block and
// lane, two more operations an element) and back 39, of 38.  16 x 4096 there and back: 2.6 us.
#include "dg_fp4.cuh"
#include "dg_internal.h"

namespace dg {
namespace {

constexpr int kCols = 256;                 // columns per CTA (32 lanes x 8)
constexpr int kWarps = 8;
constexpr int kRows = 4;                   // rows per warp, 32 apart, all in flight
constexpr int kStep = 32;                  // rows r, r + 32, r + 64, r + 96 of a scale tile share 16 bytes
constexpr int kRowCtas = kStep / kWarps;   // CTAs over a scale tile's 128 rows
static_assert(kRows * kStep == fp4::kTileRows && kStep % kWarps == 0, "a warp's rows are one 16-byte piece");

// Where a warp works: its first row, its 16-byte piece in scale tile kt of that tile row.
struct Place {
    int row0, col_tile;
    int rows;              // rows of the tile from row0 on, every 32nd this warp's
    size_t scales;

    // tile_rows: rows that share a scale tile (the rest of its 128 are past the end)
    __device__ Place(int col_tiles, int lane, int word_lanes, int tiles_per_cta, int nkt, int tile_rows, int M)
    {
        const int rc = static_cast<int>(blockIdx.x) / col_tiles;
        col_tile = static_cast<int>(blockIdx.x) - rc * col_tiles;
        const int tile = rc / kRowCtas, r = (rc % kRowCtas) * kWarps + (threadIdx.x >> 5);
        row0 = tile * tile_rows + r;
        rows = min(tile_rows - r, M - row0);
        scales = (static_cast<size_t>(tile) * nkt + col_tile * tiles_per_cta + lane / word_lanes) * fp4::kTileBytes +
                 fp4::tile_offset(r, 0);
    }
};

template <bool NV>
__global__ void __launch_bounds__(kWarps * 32) fp4_quant_kernel(const uint16_t* x, uint8_t* __restrict__ q,
                                                                uint8_t* __restrict__ s, const float* gp, int M, int K,
                                                                int col_tiles, int tile_rows, int early)
{
    constexpr int kShare = fp4::block_len(NV) / 8;             // lanes per block
    constexpr int kWord = 4 * kShare;                          // lanes per scale word
    constexpr int kTiles = kCols / fp4::tile_k(NV);            // scale tiles per CTA
    if (early) pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, nkt = fp4::scale_tiles(K, NV);
    const Place at(col_tiles, lane, kWord, kTiles, nkt, tile_rows, M);
    const int k = at.col_tile * kCols + lane * 8;
    const bool in = k < K;                                     // K % 32 == 0: a block is inside or outside
    const float g = gp ? *gp : 1.0f, g6 = __fmul_rn(6.0f, g);
    uint4 raw[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        raw[i] = make_uint4(0, 0, 0, 0);
        if (in && i * kStep < at.rows)
            raw[i] = ld_stream_after(x + static_cast<size_t>(at.row0 + i * kStep) * K + k);
    }
    uint32_t words[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int row = at.row0 + i * kStep;
        words[i] = 0;                                          // scale bytes of rows and blocks past the end
        if (i * kStep >= at.rows) continue;                    // (the same in every lane)
        uint32_t m = fp4::amax8(raw[i]);
#pragma unroll
        for (int o = 1; o < kShare; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
        const fp4::Scale bs = fp4::block_scale<NV>(m, g6, g);
        float v[8];
        fp4::unpack8(raw[i], v);
        const uint32_t codes = fp4::encode8<NV>(v, bs);
        if (in) *reinterpret_cast<uint32_t*>(q + (static_cast<size_t>(row) * K + k) / 2) = codes;
        uint32_t w = in ? bs.byte << (8 * ((lane / kShare) & 3)) : 0u;
#pragma unroll
        for (int o = kShare; o < kWord; o <<= 1) w |= __shfl_xor_sync(kFull, w, o);
        words[i] = w;
    }
    if (lane % kWord == 0 && at.col_tile * kTiles + lane / kWord < nkt)
        *reinterpret_cast<uint4*>(s + at.scales) = make_uint4(words[0], words[1], words[2], words[3]);
}

// y = bf16(code * (scale * g)), each step rounded to binary32 (MX: exact).
template <bool NV>
__global__ void __launch_bounds__(kWarps * 32) fp4_dequant_kernel(const uint8_t* q, const uint8_t* s, const float* gp,
                                                                  uint16_t* y, int M, int K, int col_tiles)
{
    constexpr int kShare = fp4::block_len(NV) / 8;
    constexpr int kWord = 4 * kShare;
    constexpr int kTiles = kCols / fp4::tile_k(NV);
    pdl_wait();
    const int lane = threadIdx.x & 31, nkt = fp4::scale_tiles(K, NV);
    const Place at(col_tiles, lane, kWord, kTiles, nkt, fp4::kTileRows, M);
    const int k = at.col_tile * kCols + lane * 8;
    const float g = gp ? *gp : 1.0f;
    if (k < K && at.rows > 0) {
        uint32_t codes[kRows];
        const uint4 sc = *reinterpret_cast<const uint4*>(s + at.scales);
        const uint32_t word[kRows] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            codes[i] = 0;
            if (i * kStep < at.rows)
                codes[i] = *reinterpret_cast<const uint32_t*>(q + (static_cast<size_t>(at.row0 + i * kStep) * K + k) / 2);
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            const int row = at.row0 + i * kStep;
            if (i * kStep >= at.rows) break;
            const uint32_t sb = (word[i] >> (8 * ((lane / kShare) & 3))) & 0xffu;
            float f;
            if constexpr (NV)
                f = fp4::e4m3_value(sb);
            else
                f = sb == 0xffu ? __uint_as_float(0x7fffffffu) : fp4::pow2(static_cast<int>(sb) - 127);
            f = __fmul_rn(f, g);
            float v[8];
            fp4::from_e2m1x8(codes[i], v);
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 p = __floats2bfloat162_rn(__fmul_rn(v[2 * j], f), __fmul_rn(v[2 * j + 1], f));
                memcpy(&w[j], &p, sizeof w[j]);
            }
            *reinterpret_cast<uint4*>(y + static_cast<size_t>(row) * K + k) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

}  // namespace

dg_status launch_fp4_quant(bool nv, const void* x, void* q, void* s, const float* g, int M, int K, int tile_rows,
                           bool early, cudaStream_t stream)
{
    int col_tiles = (K + kCols - 1) / kCols, now = early ? 1 : 0;
    const long long grid = ((static_cast<long long>(M) + tile_rows - 1) / tile_rows) * kRowCtas * col_tiles;
    if (grid > 0x7fffffffll) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* fn = nv ? reinterpret_cast<const void*>(&fp4_quant_kernel<true>)
                        : reinterpret_cast<const void*>(&fp4_quant_kernel<false>);
    void* args[] = {&x, &q, &s, &g, &M, &K, &col_tiles, &tile_rows, &now};
    if (launch_kernel(fn, static_cast<unsigned>(grid), kWarps * 32, 0, stream, args, Early::kNothing) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

dg_status launch_fp4_dequant(bool nv, const void* q, const void* s, const float* g, void* y, int M, int K,
                             cudaStream_t stream)
{
    int col_tiles = (K + kCols - 1) / kCols;
    const long long grid = ((static_cast<long long>(M) + fp4::kTileRows - 1) / fp4::kTileRows) * kRowCtas * col_tiles;
    if (grid > 0x7fffffffll) return DG_ERR_UNSUPPORTED_SHAPE;
    const void* fn = nv ? reinterpret_cast<const void*>(&fp4_dequant_kernel<true>)
                        : reinterpret_cast<const void*>(&fp4_dequant_kernel<false>);
    void* args[] = {&q, &s, &g, &y, &M, &K, &col_tiles};
    if (launch_kernel(fn, static_cast<unsigned>(grid), kWarps * 32, 0, stream, args, Early::kNothing) != cudaSuccess) {
        cudaGetLastError();
        return DG_ERR_CUDA;
    }
    return DG_OK;
}

}  // namespace dg
