// ssm_common.cuh -- device helpers of the state-space operators.
#pragma once

#include "serial_common.cuh"
#include "ssm_internal.h"

namespace gdn {
namespace ssm {

using mla::load8;
using mla::raw8;
using mla::rows_of;
using mla::store8;
using mla::values;
using rec::ex2_approx;
using rec::f2;
using rec::fma2;
using rec::mul2;

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float rcp(float x)     // 1 / x to about an ulp; 0 for an infinite x
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2_approx(-kLog2e * x)); }

// log(1 + exp(v)) and its derivative.  With e = exp(-|v|) in (0, 1] it is max(v, 0) + log(1 + e), and
// log(1 + e) = 2 atanh(s) = 2 s (1 + s^2 / 3 + s^4 / 5 + ...) for s = e / (2 + e) <= 1 / 3, whose terms past s^12 / 13
// add less than 2e-8 of it: small step sizes keep their relative accuracy, which log2 of 1 + e would lose.
__device__ __forceinline__ float softplus(float v, float& slope)
{
    const float e = ex2_approx(-kLog2e * fabsf(v)), s = e * rcp(2.f + e), q = s * s, r = rcp(1.f + e);
    float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    p = fmaf(q, p, 1.f / 9.f);
    p = fmaf(q, p, 1.f / 7.f);
    p = fmaf(q, p, 1.f / 5.f);
    p = fmaf(q, p, 1.f / 3.f);
    p = fmaf(q, p, 1.f);
    slope = v >= 0.f ? r : e * r;
    return fmaf(2.f * s, p, fmaxf(v, 0.f));
}

// 16 bytes to shared memory, zeros unless ok
__device__ __forceinline__ void cp_async16_zero(void* to, const void* from, bool ok)
{
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to), n = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(from), "r"(n) : "memory");
}

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

}  // namespace ssm
}  // namespace gdn
