// dg_route.cuh -- the routing's division: correctly rounded reciprocals and quotients in three
// and three more instructions (P. W. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990), where the compiler's division takes a dozen.
#pragma once

#include "dg_common.cuh"

namespace dg {
namespace route {

constexpr float kLeastY = 0x1p-60f, kLeastE = 0x1p-90f;

// 1 / y, correctly rounded, for kLeastY <= y < 2^125: one Newton step in fused operations on a
// reciprocal within an ulp.  Equal to IEEE division for every mantissa at fourteen exponents
// from -60 to 124.
__device__ __forceinline__ float recip_rn(float y)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
    return __fmaf_rn(r, __fmaf_rn(-y, r, 1.0f), r);
}

// e / y, correctly rounded, from r = recip_rn(y), for e = 0 or e >= kLeastE (no remainder is
// subnormal) with a quotient of at most 2^60.
__device__ __forceinline__ float quotient_rn(float e, float y, float r)
{
    const float q = __fmul_rn(e, r);
    return __fmaf_rn(__fmaf_rn(-q, y, e), r, q);
}

}  // namespace route
}  // namespace dg
