// mla_attn_f32.cu -- attention over expanded keys and values on the CUDA cores: the form for f32 I/O.
//
// A CTA holds 16 RI queries (or, for the key gradients, keys) and walks the other side in tiles of 64 rows through
// shared memory, the next tile on its way by cp.async where two fit; each of 256 threads owns an RI x 4 block of a
// score tile and RI rows of the results.  fp32 FMAs bound it: tf32 products would be faster but keep 10 bits.
// RI is as large as leaves every SM a CTA: four rows a thread reuse each operand from shared memory four times, but a
// small batch then fills a fraction of the SMs (times at both ends at pick_rows below).
#include "mla_internal.h"

namespace gdn {
namespace mla {

namespace {

constexpr int kThreads = 256, kTile = 64, kSP = kTile + 4;   // row pitch = 4 mod 32 words: 16-byte reads of
                                                             // consecutive rows meet no bank twice
constexpr size_t kRoom = 227 * 1024;

__host__ __device__ inline int pitch_of(int d) { return (d + 63) / 64 * 64 + 4; }

template <int BYTES>
__device__ __forceinline__ void copy_async(float* dst, const float* src, bool in)
{
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst), n = in ? BYTES : 0;
    if (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(d), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// asks for rows [r0, r0 + ROWS) of a tensor given as a main part of width d1 and a shared part of width d2 behind it;
// rows past n and columns past d1 + d2 become zeros
template <int ROWS>
__device__ __forceinline__ void ask_tile(float* s, int pitch, const float* a, long long tok_a, int d1, const float* b,
                                         long long tok_b, int d2, int r0, int n)
{
    const int per = (pitch - 4) >> 2;
    for (int i = threadIdx.x; i < ROWS * per; i += kThreads) {
        const int r = i / per, c = (i - r * per) << 2;
        const bool row = r0 + r < n, first = c < d1, in = row && c < d1 + d2;
        const float* src = first ? a + (long long)(r0 + r) * tok_a + c : b + (long long)(r0 + r) * tok_b + (c - d1);
        copy_async<16>(s + r * pitch + c, in ? src : a, in);
    }
}

// acc[i][j] = A[RA ty + i] . B[tx + 16 j]
template <int RA, int RB>
__device__ __forceinline__ void dots(float (&acc)[RA][RB], const float* A, const float* B, int pitch, int d, int ty, int tx)
{
#pragma unroll
    for (int i = 0; i < RA; i++)
#pragma unroll
        for (int j = 0; j < RB; j++) acc[i][j] = 0.f;
#pragma unroll 2
    for (int c = 0; c < d; c += 4) {
        float4 x[RA], y[RB];
#pragma unroll
        for (int i = 0; i < RA; i++) x[i] = *reinterpret_cast<const float4*>(A + (RA * ty + i) * pitch + c);
#pragma unroll
        for (int j = 0; j < RB; j++) y[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * pitch + c);
#pragma unroll
        for (int i = 0; i < RA; i++)
#pragma unroll
            for (int j = 0; j < RB; j++)
                acc[i][j] += x[i].x * y[j].x + x[i].y * y[j].y + x[i].z * y[j].z + x[i].w * y[j].w;
    }
}

// acc[i][4 j + e] += sum_k P(k, RI ty + i) B[k][64 j + 4 tx + e] over 64 rows of B; P is stored a held row after another
// (pitch kSP), or TRANSPOSED a walked row after another (pitch 16 RI + 4)
template <bool TRANSPOSED, int RI, int NJ>
__device__ __forceinline__ void accumulate(float (&acc)[RI][4 * NJ], const float* P, const float* B, int pitch, int nj, int ty,
                                           int tx)
{
#pragma unroll 2
    for (int k = 0; k < kTile; k += 4) {
        float p[RI][4];
        if (TRANSPOSED) {
#pragma unroll
            for (int e = 0; e < 4; e++)
#pragma unroll
                for (int i = 0; i < RI; i++) p[i][e] = P[(k + e) * (16 * RI + 4) + RI * ty + i];
        } else {
#pragma unroll
            for (int i = 0; i < RI; i++)
                *reinterpret_cast<float4*>(p[i]) = *reinterpret_cast<const float4*>(P + (RI * ty + i) * kSP + k);
        }
#pragma unroll
        for (int j = 0; j < NJ; j++)
            if (j < nj) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float4 b = *reinterpret_cast<const float4*>(B + (k + e) * pitch + 64 * j + 4 * tx);
#pragma unroll
                    for (int i = 0; i < RI; i++) {
                        acc[i][4 * j] += p[i][e] * b.x;
                        acc[i][4 * j + 1] += p[i][e] * b.y;
                        acc[i][4 * j + 2] += p[i][e] * b.z;
                        acc[i][4 * j + 3] += p[i][e] * b.w;
                    }
                }
            }
    }
}

__device__ __forceinline__ void store4(float* p, const float* v, float f)
{
    *reinterpret_cast<float4*>(p) = make_float4(v[0] * f, v[1] * f, v[2] * f, v[3] * f);
}

// reduction over the 16 threads that share rows
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

// The walk over `n` tiles: ask(i, buffer) requests tile i, work(i, buffer) uses it.  stages: 1 or 2 buffers.
template <typename Ask, typename Work>
__device__ __forceinline__ void walk(int n, int stages, Ask ask, Work work)
{
    if (n > 0) ask(0, 0);
    copies_commit();
    for (int i = 0; i < n; i++) {
        const int buf = stages == 2 ? i & 1 : 0;
        if (stages == 2 && i + 1 < n) {
            ask(i + 1, buf ^ 1);
            copies_commit();
            copies_wait<1>();
        } else {
            copies_wait<0>();
        }
        __syncthreads();
        work(i, buf);
        __syncthreads();
        if (stages == 1 && i + 1 < n) {
            ask(i + 1, 0);
            copies_commit();
        }
    }
}

template <int RI>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const AttnArgs a, int stages)
{
    extern __shared__ float smem[];
    constexpr int kHeld = 16 * RI;
    const gdn_mla_attn_t& s = a.s;
    const int h = blockIdx.y, b = blockIdx.z, g = h / (s.H / s.Hkv), q0 = blockIdx.x * kHeld;
    const Rows rq = rows_of(a.cu_q, b, s.Tq, s.Nq), rk = rows_of(a.cu_k, b, s.Tk, s.Nk);
    if (q0 >= rq.n) return;
    const int d = s.dn + s.dr, pq = pitch_of(d), pv = pitch_of(s.dv), nj = (s.dv + 63) >> 6;
    float *Q = smem, *P = Q + kHeld * pq, *K = P + kHeld * kSP, *V = K + stages * kTile * pq;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = rk.n - rq.n;
    const int end = s.causal ? min(rk.n, min(q0 + kHeld, rq.n) + off) : rk.n;
    ask_tile<kHeld>(Q, pq, head_of(a.qn, rq.first, h), a.qn.tok, s.dn, head_of(a.qr, rq.first, h), a.qr.tok, s.dr, q0, rq.n);
    float m[RI], l[RI], o[RI][8];
#pragma unroll
    for (int i = 0; i < RI; i++) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 8; j++) o[i][j] = 0.f;
    }
    const auto ask = [&](int t, int buf) {
        ask_tile<kTile>(K + buf * kTile * pq, pq, head_of(a.kn, rk.first, g), a.kn.tok, s.dn, head_of(a.kr, rk.first, 0), a.kr.tok,
                        s.dr, t * kTile, rk.n);
        ask_tile<kTile>(V + buf * kTile * pv, pv, head_of(a.v, rk.first, g), a.v.tok, s.dv, head_of(a.v, rk.first, g), 0, 0,
                        t * kTile, rk.n);
    };
    const auto work = [&](int t, int buf) {
        const int k0 = t * kTile;
        float x[RI][4];
        dots<RI, 4>(x, Q, K + buf * kTile * pq, pq, d, ty, tx);
#pragma unroll
        for (int i = 0; i < RI; i++) {
            const int last = s.causal ? min(rk.n - 1, q0 + RI * ty + i + off) : rk.n - 1;
            float top = m[i];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x[i][j] = k0 + tx + 16 * j <= last ? x[i][j] * s.scale : -INFINITY;
                top = fmaxf(top, x[i][j]);
            }
            top = row_max(top);
            const float base = top == -INFINITY ? 0.f : top, keep = expf(m[i] - base);
            m[i] = top;
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x[i][j] = expf(x[i][j] - base);
                sum += x[i][j];
                P[(RI * ty + i) * kSP + tx + 16 * j] = x[i][j];
            }
            l[i] = l[i] * keep + row_sum(sum);
#pragma unroll
            for (int j = 0; j < 8; j++) o[i][j] *= keep;
        }
        __syncwarp();     // a row's weights come from its own 16 threads
        accumulate<false, RI, 2>(o, P, V + buf * kTile * pv, pv, nj, ty, tx);
    };
    walk((max(end, 0) + kTile - 1) / kTile, stages, ask, work);
    float* out = (float*)a.o + ((long long)rq.first * s.H + h) * s.dv;
#pragma unroll
    for (int i = 0; i < RI; i++) {
        const int r = q0 + RI * ty + i;
        if (r >= rq.n) continue;
        const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
        if (tx == 0 && a.lse) a.lse[(long long)h * s.Nq + rq.first + r] = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int c = 64 * j + 4 * tx;
            if (c < s.dv) store4(out + (long long)r * s.H * s.dv + c, &o[i][4 * j], inv);
        }
    }
}

// p = exp(scale s - lse) and ds = p (dp - delta) for one pair; zero where the query does not see the key
__device__ __forceinline__ void pair_grads(float& x, float& y, float scale, float lse, float delta, int key, int last)
{
    const bool seen = key <= last;
    x = seen ? expf(x * scale - lse) : 0.f;
    // a query that sees one key has a constant weight: zero, not the difference of two roundings
    y = seen && last > 0 ? x * (y - delta) : 0.f;
}

template <int RI>
__global__ void __launch_bounds__(kThreads) dq_kernel(const AttnArgs a, int stages)
{
    cudaGridDependencySynchronize();     // launched as a dependent of the kernel before it
    extern __shared__ float smem[];
    constexpr int kHeld = 16 * RI;
    const gdn_mla_attn_t& s = a.s;
    const int h = blockIdx.y, b = blockIdx.z, g = h / (s.H / s.Hkv), q0 = blockIdx.x * kHeld;
    const Rows rq = rows_of(a.cu_q, b, s.Tq, s.Nq), rk = rows_of(a.cu_k, b, s.Tk, s.Nk);
    if (q0 >= rq.n) return;
    const int d = s.dn + s.dr, pq = pitch_of(d), pv = pitch_of(s.dv), nj = (d + 63) >> 6;
    float *Q = smem, *D = Q + kHeld * pq, *S = D + kHeld * pv, *K = S + kHeld * kSP, *V = K + stages * kTile * pq;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = rk.n - rq.n, end = s.causal ? min(rk.n, min(q0 + kHeld, rq.n) + off) : rk.n;
    const float* dO = (const float*)a.dO + ((long long)rq.first * s.H + h) * s.dv;
    ask_tile<kHeld>(Q, pq, head_of(a.qn, rq.first, h), a.qn.tok, s.dn, head_of(a.qr, rq.first, h), a.qr.tok, s.dr, q0, rq.n);
    ask_tile<kHeld>(D, pv, dO, (long long)s.H * s.dv, s.dv, dO, 0, 0, q0, rq.n);
    float lse[RI], delta[RI], dq[RI][12] = {};
    int last[RI];
#pragma unroll
    for (int i = 0; i < RI; i++) {
        const int r = q0 + RI * ty + i;
        const long long at = (long long)h * s.Nq + rq.first + min(r, rq.n - 1);
        lse[i] = a.lse[at];
        delta[i] = a.delta[at];
        last[i] = r >= rq.n ? -1 : s.causal ? min(rk.n - 1, r + off) : rk.n - 1;
    }
    const auto ask = [&](int t, int buf) {
        ask_tile<kTile>(K + buf * kTile * pq, pq, head_of(a.kn, rk.first, g), a.kn.tok, s.dn, head_of(a.kr, rk.first, 0), a.kr.tok,
                        s.dr, t * kTile, rk.n);
        ask_tile<kTile>(V + buf * kTile * pv, pv, head_of(a.v, rk.first, g), a.v.tok, s.dv, head_of(a.v, rk.first, g), 0, 0,
                        t * kTile, rk.n);
    };
    const auto work = [&](int t, int buf) {
        float x[RI][4], y[RI][4];
        dots<RI, 4>(x, Q, K + buf * kTile * pq, pq, d, ty, tx);
        dots<RI, 4>(y, D, V + buf * kTile * pv, pv, s.dv, ty, tx);
#pragma unroll
        for (int i = 0; i < RI; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) {
                pair_grads(x[i][j], y[i][j], s.scale, lse[i], delta[i], t * kTile + tx + 16 * j, last[i]);
                S[(RI * ty + i) * kSP + tx + 16 * j] = y[i][j];
            }
        __syncwarp();
        accumulate<false, RI, 3>(dq, S, K + buf * kTile * pq, pq, nj, ty, tx);
    };
    walk((max(end, 0) + kTile - 1) / kTile, stages, ask, work);
    float *on = head_of(a.dqn, rq.first, h), *op = head_of(a.dqr, rq.first, h);
#pragma unroll
    for (int i = 0; i < RI; i++) {
        const int r = q0 + RI * ty + i;
        if (r >= rq.n) continue;
#pragma unroll
        for (int j = 0; j < 3; j++) {
            const int c = 64 * j + 4 * tx;
            if (c < s.dn)
                store4(on + (long long)r * a.dqn.tok + c, &dq[i][4 * j], s.scale);
            else if (c < d)
                store4(op + (long long)r * a.dqr.tok + (c - s.dn), &dq[i][4 * j], s.scale);
        }
    }
}

template <int RI>
__global__ void __launch_bounds__(kThreads) dkv_kernel(const AttnArgs a, int stages)
{
    cudaGridDependencySynchronize();     // launched as a dependent of the kernel before it
    extern __shared__ float smem[];
    constexpr int kHeld = 16 * RI, kPP = kHeld + 4;
    const gdn_mla_attn_t& s = a.s;
    const int g = blockIdx.y, b = blockIdx.z, G = s.H / s.Hkv, k0 = blockIdx.x * kHeld;
    const Rows rq = rows_of(a.cu_q, b, s.Tq, s.Nq), rk = rows_of(a.cu_k, b, s.Tk, s.Nk);
    if (k0 >= rk.n) return;
    const int d = s.dn + s.dr, pq = pitch_of(d), pv = pitch_of(s.dv), njk = (d + 63) >> 6, njv = (s.dv + 63) >> 6;
    float *K = smem, *V = K + kHeld * pq, *P = V + kHeld * pv, *S = P + kTile * kPP, *L = S + kTile * kPP,
          *Q = L + stages * 2 * kTile, *D = Q + stages * kTile * pq;
    const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
    const int off = rk.n - rq.n;
    const int first = s.causal ? max(0, k0 - off) / kTile : 0;      // the first tile whose queries see key k0
    const int per = max(0, (rq.n + kTile - 1) / kTile - first);
    ask_tile<kHeld>(K, pq, head_of(a.kn, rk.first, g), a.kn.tok, s.dn, head_of(a.kr, rk.first, 0), a.kr.tok, s.dr, k0, rk.n);
    ask_tile<kHeld>(V, pv, head_of(a.v, rk.first, g), a.v.tok, s.dv, head_of(a.v, rk.first, g), 0, 0, k0, rk.n);
    float dk[RI][12] = {}, dv[RI][8] = {};
    const auto ask = [&](int t, int buf) {
        const int h = g * G + t / per, q0 = (first + t % per) * kTile;
        const float* dO = (const float*)a.dO + ((long long)rq.first * s.H + h) * s.dv;
        ask_tile<kTile>(Q + buf * kTile * pq, pq, head_of(a.qn, rq.first, h), a.qn.tok, s.dn, head_of(a.qr, rq.first, h),
                        a.qr.tok, s.dr, q0, rq.n);
        ask_tile<kTile>(D + buf * kTile * pv, pv, dO, (long long)s.H * s.dv, s.dv, dO, 0, 0, q0, rq.n);
        if (tid < 2 * kTile) {     // lse and delta of the tile's queries
            const int r = q0 + (tid & (kTile - 1));
            const float* src = (tid < kTile ? a.lse : a.delta) + (long long)h * s.Nq + rq.first;
            copy_async<4>(L + buf * 2 * kTile + tid, src + min(r, rq.n - 1), r < rq.n);
        }
    };
    const auto work = [&](int t, int buf) {
        const int q0 = (first + t % per) * kTile;
        const float* lse = L + buf * 2 * kTile;
        float x[4][RI], y[4][RI];
        dots<4, RI>(x, Q + buf * kTile * pq, K, pq, d, ty, tx);
        dots<4, RI>(y, D + buf * kTile * pv, V, pv, s.dv, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int r = q0 + 4 * ty + i;
            const int last = r >= rq.n ? -1 : s.causal ? min(rk.n - 1, r + off) : rk.n - 1;
            const float lr = lse[4 * ty + i], dr = lse[kTile + 4 * ty + i];
#pragma unroll
            for (int j = 0; j < RI; j++) {
                pair_grads(x[i][j], y[i][j], s.scale, lr, dr, k0 + tx + 16 * j, last);
                P[(4 * ty + i) * kPP + tx + 16 * j] = x[i][j];
                S[(4 * ty + i) * kPP + tx + 16 * j] = y[i][j];
            }
        }
        __syncthreads();
        accumulate<true, RI, 2>(dv, P, D + buf * kTile * pv, pv, njv, ty, tx);
        accumulate<true, RI, 3>(dk, S, Q + buf * kTile * pq, pq, njk, ty, tx);
    };
    walk(per * G, stages, ask, work);
    float *on = head_of(a.dkn, rk.first, g), *ov = head_of(a.dv, rk.first, g);
#pragma unroll
    for (int i = 0; i < RI; i++) {
        const int r = k0 + RI * ty + i;
        if (r >= rk.n) continue;
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int c = 64 * j + 4 * tx;
            if (c < s.dv) store4(ov + (long long)r * a.dv.tok + c, &dv[i][4 * j], 1.f);
        }
#pragma unroll
        for (int j = 0; j < 3; j++) {
            const int c = 64 * j + 4 * tx;
            if (c < s.dn)
                store4(on + (long long)r * a.dkn.tok + c, &dk[i][4 * j], s.scale);
            else if (c < d)
                store4(a.dkr_part + ((long long)g * s.Nk + rk.first + r) * s.dr + (c - s.dn), &dk[i][4 * j], s.scale);
        }
    }
}

// Rows a thread for `rows` held rows in each of `units` (head, sequence) pairs: the most that give every SM a CTA.
// A training step with 4, 2 and 1 rows, us: 2 x 333 tokens under 4 heads 228 / 174 / 156, 2 x 1024 under 8 672 / 681 / 864,
// 4 x 2048 under 8 3323 / 3704 / 5464.
int pick_rows(int rows, long long units)
{
    for (int r = 4; r > 1; r >>= 1)
        if ((long long)((rows + 16 * r - 1) / (16 * r)) * units >= 152) return r;
    return 1;
}

// launches kernel(a, stages) with as many buffers of the walked side as fit
template <typename F>
cudaError_t start(F kernel, const AttnArgs& a, dim3 grid, size_t held, size_t walked, bool dependent, cudaStream_t st)
{
    const int stages = (held + 2 * walked) * sizeof(float) <= kRoom ? 2 : 1;
    const size_t bytes = (held + stages * walked) * sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a, stages);
}

}  // namespace

cudaError_t launch_attn_f32(const AttnArgs& a, cudaStream_t st)
{
    const gdn_mla_attn_t& s = a.s;
    const int pq = pitch_of(s.dn + s.dr), pv = pitch_of(s.dv), r = pick_rows(s.Tq, (long long)s.H * s.B), held = 16 * r;
    const dim3 grid((s.Tq + held - 1) / held, s.H, s.B);
    const size_t h = (size_t)held * (pq + kSP), w = (size_t)kTile * (pq + pv);
    return start(r == 4 ? fwd_kernel<4> : r == 2 ? fwd_kernel<2> : fwd_kernel<1>, a, grid, h, w, false, st);
}

cudaError_t launch_attn_bwd_f32(const AttnArgs& a, cudaStream_t st)
{
    const gdn_mla_attn_t& s = a.s;
    const int pq = pitch_of(s.dn + s.dr), pv = pitch_of(s.dv);
    cudaError_t e;
    if (s.Tq > 0) {
        if ((e = launch_delta(a, st)) != cudaSuccess) return e;
        const int r = pick_rows(s.Tq, (long long)s.H * s.B), held = 16 * r;
        const dim3 grid((s.Tq + held - 1) / held, s.H, s.B);
        const size_t h = (size_t)held * (pq + pv + kSP), w = (size_t)kTile * (pq + pv);
        e = start(r == 4 ? dq_kernel<4> : r == 2 ? dq_kernel<2> : dq_kernel<1>, a, grid, h, w, true, st);
        if (e != cudaSuccess) return e;
    }
    if (s.Tk > 0) {
        const int r = pick_rows(s.Tk, (long long)s.Hkv * s.B), held = 16 * r;
        const dim3 grid((s.Tk + held - 1) / held, s.Hkv, s.B);
        const size_t h = (size_t)held * (pq + pv) + (size_t)2 * kTile * (held + 4), w = (size_t)kTile * (pq + pv + 2);
        e = start(r == 4 ? dkv_kernel<4> : r == 2 ? dkv_kernel<2> : dkv_kernel<1>, a, grid, h, w, s.Tq > 0, st);
        if (e != cudaSuccess) return e;
        if (s.dr > 0) return launch_dkr(a, st);
    }
    return cudaSuccess;
}

}  // namespace mla
}  // namespace gdn
