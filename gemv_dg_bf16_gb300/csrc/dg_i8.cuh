// dg_i8.cuh -- 8-bit integer codes with one scale a row, and their exact products.
//
// A row of bf16 values with largest magnitude amax >= 0 becomes, in binary32 (every step one
// correctly rounded operation, so that codes and scales are defined to the last bit):
//   A = max(amax, 2^-100),  r = 127 * (1 / A),  s = A * fl(1 / 127),  q = round-to-nearest-even(x * r)
// |q| <= 127: amax * r is 127 to a relative 2^-21, so within 2^-14 (1 / A may be subnormal, where it has 22 bits at
// least).  The floor keeps r finite; an all-zero row has codes 0.  A row that holds an infinity or a NaN has
// codes 0 and scale NaN.
//
// Products are exact.  An 8-bit integer is exact in binary16, a product of two in binary32, and a
// sum of at most 1024 of them is at most 1024 * 127 * 128 < 2^24, so that a chain of f16 MMAs
// with binary32 accumulators over 1024 elements of K has no rounding; such segments are
// added up as 32-bit integers (K <= 131072: |sum| < 2^31).  Whatever cuts K, the tokens or the rows, the
// sum is the same integer: every variant, batch and split gives the same bits.
#pragma once

#include "dg_common.cuh"

namespace dg {
namespace i8 {

constexpr int kMaxK = 131072;            // 131072 * 127 * 128 < 2^31
constexpr int kSegment = 1024;           // K elements of one exact chain in binary32
constexpr float kMagic = 12582912.0f;    // 1.5 * 2^23: v + kMagic holds rint(v) in its low bits

struct RowScale {
    float r, s;
    bool live;
};

// Largest magnitude of eight bf16 values as bits in each half (an integer maximum keeps
// infinities and NaN on top).
__device__ __forceinline__ uint32_t amax8(uint4 v)
{
    constexpr uint32_t kAbs = 0x7fff7fffu;
    return __vmaxu2(__vmaxu2(v.x & kAbs, v.y & kAbs), __vmaxu2(v.z & kAbs, v.w & kAbs));
}

// bits: the row's largest magnitude as a bf16 pattern.
__device__ __forceinline__ RowScale row_scale(uint32_t bits)
{
    RowScale o;
    o.live = bits < 0x7f80u;
    const float a = fmaxf(__uint_as_float(bits << 16), 0x1p-100f);
    o.r = __fmul_rn(127.0f, __fdiv_rn(1.0f, a));
    o.s = o.live ? __fmul_rn(a, 1.0f / 127.0f) : __uint_as_float(0x7fffffffu);
    return o;
}

// rint(x r) + kMagic: its low byte is the code.
__device__ __forceinline__ float coded(float x, float r) { return __fadd_rn(__fmul_rn(x, r), kMagic); }

// Eight values -> eight code bytes, or eight codes as binary16.
__device__ __forceinline__ uint2 codes8(uint4 v, const RowScale& o)
{
    if (!o.live) return make_uint2(0, 0);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        b[j] = __byte_perm(__float_as_uint(coded(bf16_lo(w[j]), o.r)), __float_as_uint(coded(bf16_hi(w[j]), o.r)), 0x0040);
    return make_uint2(__byte_perm(b[0], b[1], 0x5410), __byte_perm(b[2], b[3], 0x5410));
}

__device__ __forceinline__ uint4 halves8(uint4 v, const RowScale& o)
{
    if (!o.live) return make_uint4(0, 0, 0, 0);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2 p = __floats2half2_rn(coded(bf16_lo(w[j]), o.r) - kMagic, coded(bf16_hi(w[j]), o.r) - kMagic);
        memcpy(&h[j], &p, sizeof h[j]);
    }
    return make_uint4(h[0], h[1], h[2], h[3]);
}

// Where the linear's activations have element k (of K) of token t: per group of mp tokens and block of 128 elements two
// boxes of 64 elements, mp rows of 128 bytes, each in the swizzled order in which the MMA reads shared memory -- so
// that a block is one contiguous copy.
__device__ __forceinline__ size_t tile_offset(int t, int k, int mp, int K)
{
    const int group = t / mp, row = t - group * mp, nkb = (K + 127) / 128;
    return ((static_cast<size_t>(group) * nkb + k / 128) * 2 + (k >> 6 & 1)) * static_cast<size_t>(mp * 128) +
           static_cast<size_t>((row >> 3) * 1024 + (row & 7) * 128 + (((k >> 3) & 7) ^ (row & 7)) * 16);
}

// Four code bytes -> two pairs of binary16: 0x6400 | (q + 128) is 1152 + q.
__device__ __forceinline__ void to_halves(uint32_t codes, uint32_t& lo, uint32_t& hi)
{
    const uint32_t u = codes ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(0x64806480u));
}

// y = bf16(sum * (s_token * s_row)), each step rounded to binary32.
__device__ __forceinline__ uint16_t output(int sum, float sx, float sw)
{
    return f32_to_bf16_bits(__fmul_rn(__int2float_rn(sum), __fmul_rn(sx, sw)));
}

}  // namespace i8
}  // namespace dg
