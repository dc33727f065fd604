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
using rec::add2;
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

__device__ __forceinline__ float max_nan(float a, float b)     // the larger one, NaN if either is
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
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

// the last of [0, n) whose key, which ascends, is at most k (0 if none is)
template <typename Key>
__device__ __forceinline__ int last_at_most(int n, int k, Key key)
{
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (key(mid) <= k) lo = mid;
        else hi = mid;
    }
    return lo;
}
__device__ __forceinline__ int offset_of(const int* cu, int b, int rows) { return min(max(cu[b], 0), rows); }
// whose place k is: a sequence and its piece of L rows (which may lie past its end)
struct Place {
    int b, piece;
};
__device__ __forceinline__ Place place_of(const int* cu, int B, int rows, int L, int k)
{
    auto key = [&](int b) { return offset_of(cu, b, rows) / L + b; };
    const int b = last_at_most(B, k, key), first = key(b);
    return {b, k < first ? places(B, rows, L) : k - first};
}

// 16 bytes to shared memory, zeros unless ok
__device__ __forceinline__ void cp_async16_zero(void* to, const void* from, bool ok)
{
    const uint32_t s = (uint32_t)__cvta_generic_to_shared(to), n = ok ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(s), "l"(from), "r"(n) : "memory");
}

// four values as two packed pairs
struct Four {
    float2 a, b;
};
__device__ __forceinline__ Four four(const float (&x)[4]) { return {f2(x[0], x[1]), f2(x[2], x[3])}; }
__device__ __forceinline__ Four mul(Four x, Four y) { return {mul2(x.a, y.a), mul2(x.b, y.b)}; }
__device__ __forceinline__ Four fma(Four x, Four y, Four z) { return {fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)}; }
__device__ __forceinline__ Four add(Four x, Four y) { return {add2(x.a, y.a), add2(x.b, y.b)}; }
__device__ __forceinline__ Four all(float x) { return {f2(x, x), f2(x, x)}; }
__device__ __forceinline__ float2 sigmoid2(float2 x)
{
    const float2 e = mul2(x, f2(-kLog2e, -kLog2e)), d = add2(f2(ex2_approx(e.x), ex2_approx(e.y)), f2(1.f, 1.f));
    return f2(rcp(d.x), rcp(d.y));
}
__device__ __forceinline__ Four sigmoid4(Four x) { return {sigmoid2(x.a), sigmoid2(x.b)}; }

__device__ __forceinline__ void store4(float* p, const float (&x)[4])
{
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4])
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// four values as they lie in memory
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ Four get() const { return {f2(v.x, v.y), f2(v.z, v.w)}; }
};
template <>
struct Raw4<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ Four get() const
    {
        return {f2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u)), f2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u))};
    }
};
__device__ __forceinline__ Raw4<float> raw4(const float* p) { return {*reinterpret_cast<const float4*>(p)}; }
__device__ __forceinline__ Raw4<__nv_bfloat16> raw4(const __nv_bfloat16* p) { return {*reinterpret_cast<const uint2*>(p)}; }
template <typename IO>
__device__ __forceinline__ void put(IO* p, Four x)
{
    const float v[4] = {x.a.x, x.a.y, x.b.x, x.b.y};
    store4(p, v);
}

}  // namespace ssm
}  // namespace gdn
