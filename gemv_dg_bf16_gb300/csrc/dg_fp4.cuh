// dg_fp4.cuh -- the microscaled 4-bit formats: block quantisation, codes, scale layout.
//
// A row of K elements is cut into blocks along K, each held as e2m1 codes (0, 1/2, 1,
// 3/2, 2, 3, 4, 6 and their negatives) under one 8-bit scale:
//   MX  32 elements, scale 2^e as e8m0 (byte e + 127), e = floor(log2 amax) - 2
//       (OCP Microscaling Formats v1.0, section 6.3), -127 for an all-zero block;
//       code = e2m1(x * 2^-e), an exact product
//   NV  16 elements, scale s as e4m3, under one fp32 scale g of the whole tensor:
//       s = e4m3(amax / (6 g)), code = e2m1(x / (s g)), 0 where s is 0
// Products and quotients are binary32 and correctly rounded; e2m1() and e4m3() round to
// nearest even and saturate.  A block with an infinity or a NaN gets the format's NaN
// scale (e8m0 0xFF, e4m3 0x7F) and zero codes, so it dequantises to NaN throughout.
//
// Codes: two a byte, the element of lower index in the low nibble.  Scales: tiles of
// 128 rows x 4 blocks, 512 bytes each, [ceil(rows/128)][ceil(blocks/4)]; row r, block b
// is byte (r % 32) * 16 + (r % 128) / 32 * 4 + b % 4 of its tile -- what one
// tcgen05.cp (32 lanes x 16 bytes) takes to tensor memory.  Rows and blocks past the
// end hold zero.
#pragma once

#include "dg_tc_common.cuh"

namespace dg {
namespace fp4 {

constexpr int kTileRows = 128;             // rows of a scale tile
constexpr int kTileBytes = 512;
constexpr int kMaxLen = 0x7fffff00;        // rows, and elements of a row: indices past the end stay in 32 bits

__host__ __device__ constexpr int block_len(bool nv) { return nv ? 16 : 32; }
__host__ __device__ constexpr int tile_k(bool nv) { return 4 * block_len(nv); }     // K elements of a scale tile
__host__ __device__ constexpr int scale_tiles(int K, bool nv)
{
    return K / tile_k(nv) + (K % tile_k(nv) != 0);
}
__host__ __device__ constexpr size_t scale_bytes(int rows, int K, bool nv)
{
    return static_cast<size_t>(rows / kTileRows + (rows % kTileRows != 0)) * scale_tiles(K, nv) * kTileBytes;
}
// Byte of row r (0..127), block b (0..3) inside a tile.
__host__ __device__ constexpr int tile_offset(int r, int b) { return (r % 32) * 16 + (r / 32) * 4 + b; }

__device__ __forceinline__ float e4m3_value(uint32_t code) { return e4m3x2_to_f32(code).x; }

// 2^e, -127 <= e <= 127.
__device__ __forceinline__ float pow2(int e)
{
    return __uint_as_float(e > -127 ? static_cast<uint32_t>(e + 127) << 23 : 0x00400000u);
}

// The scale of a block: its byte, what the elements are divided by (NV) or multiplied
// with (MX), and whether any code is non-zero at all.
struct Scale {
    uint32_t byte;
    float f;           // MX: 2^-e; NV: s g
    bool live;
    bool plain;        // NV: operands or quotients leave the range that encode8's division is for
};

// amax_bits: the largest |x| of the block, as bits (an integer maximum keeps NaN on top).
template <bool NV>
__device__ __forceinline__ Scale block_scale(uint32_t amax_bits, float g6, float g)
{
    Scale r;
    if (amax_bits >= 0x7f800000u) {
        r.byte = NV ? 0x7fu : 0xffu;
        r.f = 1.0f;
        r.live = false;
        r.plain = false;
    } else if constexpr (NV) {
        const uint32_t c = tc::to_e4m3x2(__fdiv_rn(__uint_as_float(amax_bits), g6), 0.0f) & 0xffu;
        r.byte = c;
        r.f = __fmul_rn(e4m3_value(c), g);
        r.live = c != 0;
        r.plain = !(r.f >= 0x1p-100f && r.f <= 0x1p100f && __uint_as_float(amax_bits) <= r.f * 0x1p20f);
    } else {
        // bf16 magnitudes: the exponent field, or the leading bit of a subnormal
        int e = static_cast<int>(amax_bits >> 23) - 127 - 2;
        if (amax_bits < 0x00800000u || e < -127) e = -127;
        r.byte = static_cast<uint32_t>(e + 127);
        r.f = pow2(-e);
        r.live = amax_bits != 0;
        r.plain = false;
    }
    return r;
}

// Eight values -> eight codes (element i in nibble i).
__device__ __forceinline__ uint32_t to_e2m1x8(const float (&v)[8])
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

// Codes of eight elements of a block.  NV divides by s g: with r the correctly rounded
// reciprocal and q within an ulp of x / f, q - r (q f - x) in fused steps is the correctly
// rounded quotient (P. W. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990) -- three instructions an element for a division's dozen.
// (With x - q f the quotient of -0 would come out as +0.)
// Where the remainder or the quotient could leave the normal range (divisors outside
// 2^-100 .. 2^100, a scale that saturated far below its block): plain division.
template <bool NV>
__device__ __forceinline__ uint32_t encode8(float (&v)[8], const Scale& s)
{
    if constexpr (NV) {
        if (!s.plain) {
            const float r = __frcp_rn(s.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = __fmul_rn(v[i], r);
                v[i] = __fmaf_rn(-__fmaf_rn(q, s.f, -v[i]), r, q);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], s.f);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], s.f);
    }
    const uint32_t c = to_e2m1x8(v);
    return s.live ? c : 0u;
}

// Eight codes -> fp32 (exact).
__device__ __forceinline__ void from_e2m1x8(uint32_t codes, float (&v)[8])
{
    uint32_t h[4];
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        __half2 p;
        memcpy(&p, &h[j], sizeof p);
        const float2 f = __half22float2(p);
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
    }
}

// Eight bf16 values of one 16-byte load as fp32.
__device__ __forceinline__ void unpack8(const uint4& a, float (&v)[8])
{
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}

// Largest magnitude of eight bf16 values, as fp32 bits: bf16 magnitudes order as 16-bit
// integers, two a word.
__device__ __forceinline__ uint32_t amax8(const uint4& a)
{
    const uint32_t m = __vmaxu2(__vmaxu2(a.x & 0x7fff7fffu, a.y & 0x7fff7fffu),
                                __vmaxu2(a.z & 0x7fff7fffu, a.w & 0x7fff7fffu));
    return max(m & 0xffff0000u, m << 16);
}

}  // namespace fp4
}  // namespace dg
