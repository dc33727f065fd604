// mla_attn_f32.cu -- attention over expanded keys and values on the CUDA cores: the form for f32 I/O.
//
// A CTA holds 64 queries (or, for the key gradients, 64 keys) and walks the other side in tiles of 64 through shared
// memory; each of 256 threads owns a 4 x 4 block of a 64 x 64 score tile and 4 rows of the results.  fp32 FMAs bound
// it: tf32 products would be faster but keep 10 bits.
#include "mla_internal.h"

namespace gdn {
namespace mla {

namespace {

constexpr int kThreads = 256, kTile = 64, kSP = kTile + 4;   // row pitch = 4 mod 32 words: 16-byte reads of
                                                             // consecutive rows meet no bank twice

__host__ __device__ inline int pitch_of(int d) { return (d + 63) / 64 * 64 + 4; }

// rows [r0, r0 + 64) of a tensor given as a main part of width d1 and a shared part of width d2 behind it; rows past
// n and columns past d1 + d2 as zeros
__device__ __forceinline__ void load_tile(float* s, int pitch, const float* a, long long tok_a, int d1, const float* b,
                                          long long tok_b, int d2, int r0, int n)
{
    const int per = (pitch - 4) >> 3;
    for (int i = threadIdx.x; i < kTile * per; i += kThreads) {
        const int r = i / per, c = (i - r * per) << 3;
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (r0 + r < n) {
            if (c < d1)
                load8(a + (long long)(r0 + r) * tok_a + c, x);
            else if (c < d1 + d2)
                load8(b + (long long)(r0 + r) * tok_b + (c - d1), x);
        }
        store8(s + r * pitch + c, x);
    }
}

// acc[i][j] = A[4 ty + i] . B[tx + 16 j]
__device__ __forceinline__ void dots(float (&acc)[4][4], const float* A, const float* B, int pitch, int d, int ty, int tx)
{
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) acc[i][j] = 0.f;
    for (int c = 0; c < d; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[i] = *reinterpret_cast<const float4*>(A + (4 * ty + i) * pitch + c);
            y[i] = *reinterpret_cast<const float4*>(B + (tx + 16 * i) * pitch + c);
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++)
                acc[i][j] += x[i].x * y[j].x + x[i].y * y[j].y + x[i].z * y[j].z + x[i].w * y[j].w;
    }
}

// acc[i][4 j + e] += sum_k P[k][4 ty + i] (TRANSPOSED) or P[4 ty + i][k] times B[k][64 j + 4 tx + e]
template <bool TRANSPOSED, int NJ>
__device__ __forceinline__ void accumulate(float (&acc)[4][4 * NJ], const float* P, const float* B, int pitch, int nj,
                                           int ty, int tx)
{
    for (int k = 0; k < kTile; k++) {
        float p[4];
        if (TRANSPOSED) {
            const float4 v = *reinterpret_cast<const float4*>(P + k * kSP + 4 * ty);
            p[0] = v.x; p[1] = v.y; p[2] = v.z; p[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) p[i] = P[(4 * ty + i) * kSP + k];
        }
#pragma unroll
        for (int j = 0; j < NJ; j++)
            if (j < nj) {
                const float4 b = *reinterpret_cast<const float4*>(B + k * pitch + 64 * j + 4 * tx);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    acc[i][4 * j] += p[i] * b.x;
                    acc[i][4 * j + 1] += p[i] * b.y;
                    acc[i][4 * j + 2] += p[i] * b.z;
                    acc[i][4 * j + 3] += p[i] * b.w;
                }
            }
    }
}

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d)
{
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}

// reduction over the 16 threads that share four rows
__device__ __forceinline__ float row_max(float x)
{
#pragma unroll
    for (int m = 8; m; m >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, m));
    return x;
}
__device__ __forceinline__ float row_sum(float x)
{
#pragma unroll
    for (int m = 8; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// one head's slice of a view, from row `first`
__device__ __forceinline__ float* head_of(const gdn_mla_view_t& v, int first, int h)
{
    return (float*)v.p + (long long)first * v.tok + (long long)h * v.head;
}

__global__ void __launch_bounds__(kThreads) fwd_kernel(const AttnArgs a)
{
    extern __shared__ float smem[];
    const gdn_mla_attn_t& s = a.s;
    const int h = blockIdx.y, b = blockIdx.z, g = h / (s.H / s.Hkv), q0 = blockIdx.x * kTile;
    const Rows rq = rows_of(a.cu_q, b, s.Tq, s.Nq), rk = rows_of(a.cu_k, b, s.Tk, s.Nk);
    if (q0 >= rq.n) return;
    const int d = s.dn + s.dr, pq = pitch_of(d), pv = pitch_of(s.dv), nj = (s.dv + 63) >> 6;
    float *Q = smem, *K = Q + kTile * pq, *V = K + kTile * pq, *P = V + kTile * pv;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = rk.n - rq.n;
    const int end = s.causal ? min(rk.n, min(q0 + kTile, rq.n) + off) : rk.n;
    load_tile(Q, pq, head_of(a.qn, rq.first, h), a.qn.tok, s.dn, head_of(a.qr, rq.first, h), a.qr.tok, s.dr, q0,
                 rq.n);
    float m[4], l[4], o[4][8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; j++) o[i][j] = 0.f;
    }
    for (int k0 = 0; k0 < end; k0 += kTile) {
        __syncthreads();
        load_tile(K, pq, head_of(a.kn, rk.first, g), a.kn.tok, s.dn, head_of(a.kr, rk.first, 0), a.kr.tok, s.dr, k0,
                     rk.n);
        load_tile(V, pv, head_of(a.v, rk.first, g), a.v.tok, s.dv, (const float*)nullptr, 0, 0, k0, rk.n);
        __syncthreads();
        float x[4][4];
        dots(x, Q, K, pq, d, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int last = s.causal ? min(rk.n - 1, q0 + 4 * ty + i + off) : rk.n - 1;
            float t = m[i];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x[i][j] = k0 + tx + 16 * j <= last ? x[i][j] * s.scale : -INFINITY;
                t = fmaxf(t, x[i][j]);
            }
            t = row_max(t);
            const float base = t == -INFINITY ? 0.f : t, keep = expf(m[i] - base);
            m[i] = t;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x[i][j] = expf(x[i][j] - base);
                sum += x[i][j];
                P[(4 * ty + i) * kSP + tx + 16 * j] = x[i][j];
            }
            l[i] = l[i] * keep + row_sum(sum);
#pragma unroll
            for (int j = 0; j < 8; j++) o[i][j] *= keep;
        }
        __syncthreads();
        accumulate<false, 2>(o, P, V, pv, nj, ty, tx);
    }
    float* out = (float*)a.o + ((long long)rq.first * s.H + h) * s.dv;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = q0 + 4 * ty + i;
        if (r >= rq.n) continue;
        const float inv = l[i] > 0.f ? 1.f / l[i] : 0.f;
        if (tx == 0 && a.lse) a.lse[(long long)h * s.Nq + rq.first + r] = l[i] > 0.f ? m[i] + logf(l[i]) : -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int c = 64 * j + 4 * tx;
            if (c < s.dv)
                store4(out + (long long)r * s.H * s.dv + c, o[i][4 * j] * inv, o[i][4 * j + 1] * inv, o[i][4 * j + 2] * inv,
                       o[i][4 * j + 3] * inv);
        }
    }
}

// p and ds = p (dO . v - delta) scale of one thread's 4 x 4 block of a tile; zero where the query does not see the key
__device__ __forceinline__ void grads(float (&x)[4][4], float (&y)[4][4], const AttnArgs& a, const Rows& rq, const Rows& rk, int h,
                                      int q0, int k0, int ty, int tx)
{
    const gdn_mla_attn_t& s = a.s;
    const int off = rk.n - rq.n;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = q0 + 4 * ty + i;
        const int last = r >= rq.n ? -1 : s.causal ? min(rk.n - 1, r + off) : rk.n - 1;
        const long long at = (long long)h * s.Nq + rq.first + min(r, rq.n - 1);
        const float lse = a.lse[at], delta = a.delta[at];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const bool seen = k0 + tx + 16 * j <= last;
            x[i][j] = seen ? expf(x[i][j] * s.scale - lse) : 0.f;
            // a query that sees one key has a constant weight: zero, not the difference of two roundings
            y[i][j] = seen && last > 0 ? x[i][j] * (y[i][j] - delta) * s.scale : 0.f;
        }
    }
}

__global__ void __launch_bounds__(kThreads) dq_kernel(const AttnArgs a)
{
    extern __shared__ float smem[];
    const gdn_mla_attn_t& s = a.s;
    const int h = blockIdx.y, b = blockIdx.z, g = h / (s.H / s.Hkv), q0 = blockIdx.x * kTile;
    const Rows rq = rows_of(a.cu_q, b, s.Tq, s.Nq), rk = rows_of(a.cu_k, b, s.Tk, s.Nk);
    if (q0 >= rq.n) return;
    const int d = s.dn + s.dr, pq = pitch_of(d), pv = pitch_of(s.dv), nj = (d + 63) >> 6;
    float *Q = smem, *K = Q + kTile * pq, *V = K + kTile * pq, *D = V + kTile * pv, *S = D + kTile * pv;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int end = s.causal ? min(rk.n, min(q0 + kTile, rq.n) + rk.n - rq.n) : rk.n;
    load_tile(Q, pq, head_of(a.qn, rq.first, h), a.qn.tok, s.dn, head_of(a.qr, rq.first, h), a.qr.tok, s.dr, q0,
                 rq.n);
    load_tile(D, pv, (const float*)a.dO + ((long long)rq.first * s.H + h) * s.dv, (long long)s.H * s.dv, s.dv,
                 (const float*)nullptr, 0, 0, q0, rq.n);
    float dq[4][12] = {};
    for (int k0 = 0; k0 < end; k0 += kTile) {
        __syncthreads();
        load_tile(K, pq, head_of(a.kn, rk.first, g), a.kn.tok, s.dn, head_of(a.kr, rk.first, 0), a.kr.tok, s.dr, k0,
                     rk.n);
        load_tile(V, pv, head_of(a.v, rk.first, g), a.v.tok, s.dv, (const float*)nullptr, 0, 0, k0, rk.n);
        __syncthreads();
        float x[4][4], y[4][4];
        dots(x, Q, K, pq, d, ty, tx);
        dots(y, D, V, pv, s.dv, ty, tx);
        grads(x, y, a, rq, rk, h, q0, k0, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) S[(4 * ty + i) * kSP + tx + 16 * j] = y[i][j];
        __syncthreads();
        accumulate<false, 3>(dq, S, K, pq, nj, ty, tx);
    }
    float *on = head_of(a.dqn, rq.first, h), *orr = head_of(a.dqr, rq.first, h);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = q0 + 4 * ty + i;
        if (r >= rq.n) continue;
#pragma unroll
        for (int j = 0; j < 3; j++) {
            const int c = 64 * j + 4 * tx;
            const float* v = &dq[i][4 * j];
            if (c < s.dn)
                store4(on + (long long)r * a.dqn.tok + c, v[0], v[1], v[2], v[3]);
            else if (c < d)
                store4(orr + (long long)r * a.dqr.tok + (c - s.dn), v[0], v[1], v[2], v[3]);
        }
    }
}

__global__ void __launch_bounds__(kThreads) dkv_kernel(const AttnArgs a)
{
    extern __shared__ float smem[];
    const gdn_mla_attn_t& s = a.s;
    const int g = blockIdx.y, b = blockIdx.z, G = s.H / s.Hkv, k0 = blockIdx.x * kTile;
    const Rows rq = rows_of(a.cu_q, b, s.Tq, s.Nq), rk = rows_of(a.cu_k, b, s.Tk, s.Nk);
    if (k0 >= rk.n) return;
    const int d = s.dn + s.dr, pq = pitch_of(d), pv = pitch_of(s.dv), njk = (d + 63) >> 6, njv = (s.dv + 63) >> 6;
    float *Q = smem, *K = Q + kTile * pq, *V = K + kTile * pq, *D = V + kTile * pv, *P = D + kTile * pv,
          *S = P + kTile * kSP;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    // the first query that sees key k0
    const int first = s.causal ? max(0, k0 - (rk.n - rq.n)) / kTile * kTile : 0;
    load_tile(K, pq, head_of(a.kn, rk.first, g), a.kn.tok, s.dn, head_of(a.kr, rk.first, 0), a.kr.tok, s.dr, k0, rk.n);
    load_tile(V, pv, head_of(a.v, rk.first, g), a.v.tok, s.dv, (const float*)nullptr, 0, 0, k0, rk.n);
    float dk[4][12] = {}, dv[4][8] = {};
    for (int h = g * G; h < (g + 1) * G; h++)
        for (int q0 = first; q0 < rq.n; q0 += kTile) {
            __syncthreads();
            load_tile(Q, pq, head_of(a.qn, rq.first, h), a.qn.tok, s.dn, head_of(a.qr, rq.first, h), a.qr.tok,
                         s.dr, q0, rq.n);
            load_tile(D, pv, (const float*)a.dO + ((long long)rq.first * s.H + h) * s.dv, (long long)s.H * s.dv, s.dv,
                         (const float*)nullptr, 0, 0, q0, rq.n);
            __syncthreads();
            float x[4][4], y[4][4];
            dots(x, Q, K, pq, d, ty, tx);
            dots(y, D, V, pv, s.dv, ty, tx);
            grads(x, y, a, rq, rk, h, q0, k0, ty, tx);
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    P[(4 * ty + i) * kSP + tx + 16 * j] = x[i][j];
                    S[(4 * ty + i) * kSP + tx + 16 * j] = y[i][j];
                }
            __syncthreads();
            accumulate<true, 2>(dv, P, D, pv, njv, ty, tx);
            accumulate<true, 3>(dk, S, Q, pq, njk, ty, tx);
        }
    float *on = head_of(a.dkn, rk.first, g), *ov = head_of(a.dv, rk.first, g);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const int r = k0 + 4 * ty + i;
        if (r >= rk.n) continue;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int c = 64 * j + 4 * tx;
            if (c < s.dv)
                store4(ov + (long long)r * a.dv.tok + c, dv[i][4 * j], dv[i][4 * j + 1], dv[i][4 * j + 2], dv[i][4 * j + 3]);
        }
#pragma unroll
        for (int j = 0; j < 3; j++) {
            const int c = 64 * j + 4 * tx;
            const float* v = &dk[i][4 * j];
            if (c < s.dn)
                store4(on + (long long)r * a.dkn.tok + c, v[0], v[1], v[2], v[3]);
            else if (c < d)
                store4(a.dkr_part + ((long long)g * s.Nk + rk.first + r) * s.dr + (c - s.dn), v[0], v[1], v[2], v[3]);
        }
    }
}

template <typename F>
cudaError_t with_smem(F f, size_t bytes)
{
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

}  // namespace

cudaError_t launch_attn_f32(const AttnArgs& a, cudaStream_t st)
{
    const gdn_mla_attn_t& s = a.s;
    const int pq = pitch_of(s.dn + s.dr), pv = pitch_of(s.dv);
    const size_t bytes = (size_t)kTile * (2 * pq + pv + kSP) * sizeof(float);
    const cudaError_t e = with_smem(fwd_kernel, bytes);
    if (e != cudaSuccess) return e;
    fwd_kernel<<<dim3((s.Tq + kTile - 1) / kTile, s.H, s.B), kThreads, bytes, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_attn_bwd_f32(const AttnArgs& a, cudaStream_t st)
{
    const gdn_mla_attn_t& s = a.s;
    const int pq = pitch_of(s.dn + s.dr), pv = pitch_of(s.dv);
    const size_t bytes = (size_t)kTile * (2 * pq + 2 * pv + 2 * kSP) * sizeof(float);
    cudaError_t e;
    if (s.Tq > 0) {
        if ((e = launch_delta(a, st)) != cudaSuccess) return e;
        if ((e = with_smem(dq_kernel, bytes)) != cudaSuccess) return e;
        dq_kernel<<<dim3((s.Tq + kTile - 1) / kTile, s.H, s.B), kThreads, bytes, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (s.Tk > 0) {
        if ((e = with_smem(dkv_kernel, bytes)) != cudaSuccess) return e;
        dkv_kernel<<<dim3((s.Tk + kTile - 1) / kTile, s.Hkv, s.B), kThreads, bytes, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if (s.dr > 0) return launch_dkr(a, st);
    }
    return cudaSuccess;
}

}  // namespace mla
}  // namespace gdn
