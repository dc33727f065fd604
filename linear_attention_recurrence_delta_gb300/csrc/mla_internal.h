// mla_internal.h -- shared declarations of the latent-attention operators (not part of the ABI).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdn_mla.h"
#include "gdn_internal.h"

namespace gdn {
namespace mla {

struct PrepArgs {
    gdn_mla_prep_t s;
    const void* kv;
    long long kv_tok;
    const float *w, *rot;
    const int *pos, *seq, *table;
    gdn_mla_view_t qr, lat, kr, qr_out;
    // gradients
    gdn_mla_view_t dlat, dkr, dqr, dqr_out;
    void* dkv;
    long long dkv_tok;
    float* dw;
    float* partial;       // [prep_bwd_blocks][dc]
};

struct AttnArgs {
    gdn_mla_attn_t s;
    gdn_mla_view_t qn, qr, kn, kr, v;
    const int *cu_q, *cu_k;
    void* o;
    float* lse;           // natural logarithm, [H, Nq]
    // gradients
    const void* dO;
    gdn_mla_view_t dqn, dqr, dkn, dkr, dv;
    float* delta;         // workspace: rowsum(dO * o), [H, Nq]
    float* dkr_part;      // workspace: each key head's share of dkr, [Hkv, Nk, dr]
    uint32_t* status;
};

struct DecodeArgs {
    gdn_mla_cache_t s;
    gdn_mla_view_t qc, qr;
    const void* cache;
    const int *table, *len;
    void* o;
    float* lse;
    uint32_t* status;     // words 0 and 1: what gdn_last_device_status reads
    uint32_t* cta_err;    // one word a worker CTA
    float* part_o;        // [groups][slots][rows][dc], normalised
    float* part_l;        // [groups][slots][rows], log2 of the sum
    int rows;             // query rows (t, h) a group holds
    int groups;
    int ctas;             // worker CTAs a group has
    int slots;            // ctas + B
};

// A decode call's rows in groups (a cache tile is read once a group) and its workers.
struct DecodePlan {
    int rows, groups, ctas, slots;
    size_t err_off, o_off, l_off, total;
};
DecodePlan decode_plan(const gdn_mla_cache_t& s);

constexpr int kDecodeTile = 64;    // cache rows a step of a decode worker covers
constexpr int kDecodeRows = 80;    // query rows that one takes at most on the tensor cores

int prep_bwd_blocks(int N);

cudaError_t launch_prep(const PrepArgs& a, cudaStream_t st);
cudaError_t launch_prep_bwd(const PrepArgs& a, cudaStream_t st);
cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t st);        // bf16
cudaError_t launch_attn_bwd_tc(const AttnArgs& a, cudaStream_t st);    // bf16
cudaError_t launch_delta(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_dkr(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attn_f32(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_attn_bwd_f32(const AttnArgs& a, cudaStream_t st);
cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st);
cudaError_t launch_decode_tc(const DecodeArgs& a, cudaStream_t st);   // bf16 workers, without the join

#ifdef __CUDACC__
// the rows of sequence b: cu's, cut to T rows and held inside [0, N], or the b-th T rows
struct Rows {
    int first, n;
};
__device__ __forceinline__ Rows rows_of(const int* cu, int b, int T, int N)
{
    if (!cu) return {b * T, T};
    const int a = min(max(cu[b], 0), N), e = min(max(cu[b + 1], 0), N);
    return {a, min(max(e - a, 0), T)};
}

// eight consecutive values, 16-byte aligned (bf16: one load, f32: two)
__device__ __forceinline__ void load8(const float* p, float (&x)[8])
{
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8])
{
    const uint4 r = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
// the same eight values as they lie in memory, to be held while others are worked on
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> raw8(const T* p)
{
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; i++) r.v[i] = reinterpret_cast<const uint4*>(p)[i];
    return r;
}
__device__ __forceinline__ void values(const Raw8<float>& r, float (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 2; i++) {
        x[4 * i] = __uint_as_float(r.v[i].x);
        x[4 * i + 1] = __uint_as_float(r.v[i].y);
        x[4 * i + 2] = __uint_as_float(r.v[i].z);
        x[4 * i + 3] = __uint_as_float(r.v[i].w);
    }
}
__device__ __forceinline__ void values(const Raw8<__nv_bfloat16>& r, float (&x)[8])
{
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8])
{
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
#endif

}  // namespace mla
}  // namespace gdn
