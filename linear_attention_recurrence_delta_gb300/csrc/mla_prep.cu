// mla_prep.cu -- latent norm, rotation of the position parts and the cache write, with their gradients.
//
// Elementwise but for one sum a token, so HBM bounds it: each input is read once and each output written once, in
// 16-byte pieces.  A warp holds a token's whole latent in registers (its sum of squares is one warp reduction); a
// thread rotates 8 pairs of a query head.  Both kinds of block run in one launch, because a decoding step is bound
// by launches, not bytes.
#include "mla_internal.h"

namespace gdn {
namespace mla {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxVec = 4;     // 8-value vectors of a latent a lane holds: dc <= 1024

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// Rotates pairs 8u .. 8u+7 of a row of width dr by the angles of `rot`'s row (backwards if BACK).
template <typename T, bool BACK>
__device__ __forceinline__ void rotate8(const T* x, T* y, const float* rot, int u, int dr, bool interleaved)
{
    const int half = dr >> 1;
    const int ia = interleaved ? 16 * u : 8 * u, ib = interleaved ? ia + 8 : half + 8 * u;
    float a[8], b[8], c[8], s[8];
    load8(x + ia, a);
    load8(x + ib, b);
    load8(rot + 8 * u, c);
    load8(rot + half + 8 * u, s);
    float p[8], q[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        if (BACK) s[i] = -s[i];
        p[i] = a[i];
        q[i] = b[i];
    }
    if (interleaved) {   // a pair is two neighbours: gather the firsts into p and the seconds into q
#pragma unroll
        for (int i = 0; i < 4; i++) {
            p[i] = a[2 * i];
            q[i] = a[2 * i + 1];
            p[i + 4] = b[2 * i];
            q[i + 4] = b[2 * i + 1];
        }
    }
    float v[8], w[8];
#pragma unroll
    for (int i = 0; i < 8; i++) {
        v[i] = p[i] * c[i] - q[i] * s[i];
        w[i] = p[i] * s[i] + q[i] * c[i];
    }
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            a[2 * i] = v[i];
            a[2 * i + 1] = w[i];
            b[2 * i] = v[i + 4];
            b[2 * i + 1] = w[i + 4];
        }
        store8(y + ia, a);
        store8(y + ib, b);
    } else {
        store8(y + ia, v);
        store8(y + ib, w);
    }
}

// one thread of the queries' share: 8 pairs of one head
template <typename T, bool BACK>
__device__ __forceinline__ void rotate_query(const PrepArgs& a, const gdn_mla_view_t& in, const gdn_mla_view_t& out,
                                             long long unit)
{
    const int per = a.s.dr >> 4;
    const long long nh = unit / per;
    const int u = (int)(unit - nh * per);
    const long long n = nh / a.s.H;
    const int h = (int)(nh - n * a.s.H);
    if (n >= a.s.N) return;
    const int pos = a.pos[n];
    T* y = (T*)out.p + n * out.tok + h * out.head;
    if (pos < 0 || pos >= a.s.npos) {
        if (BACK) {
            const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            store8(y + 16 * u, z);
            store8(y + 16 * u + 8, z);
        }
        return;
    }
    rotate8<T, BACK>((const T*)in.p + n * in.tok + h * in.head, y, a.rot + (long long)pos * a.s.dr, u, a.s.dr,
                     a.s.interleaved != 0);
}

// blocks [0, lat_blocks): a warp a token; the rest: a thread 8 pairs of a query head
template <typename T>
__global__ void __launch_bounds__(kThreads) prep_kernel(const PrepArgs a, int lat_blocks)
{
    if ((int)blockIdx.x >= lat_blocks) {
        rotate_query<T, false>(a, a.qr, a.qr_out, (long long)(blockIdx.x - lat_blocks) * kThreads + threadIdx.x);
        return;
    }
    const int lane = threadIdx.x & 31;
    const long long n = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (n >= a.s.N) return;
    const int dc = a.s.dc, dr = a.s.dr, nv = dc >> 3;
    const int pos = a.pos[n];
    const bool paged = a.s.page > 0;
    const T* x = (const T*)a.kv + n * a.kv_tok;
    float v[kMaxVec][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxVec; k++)
        if (lane + 32 * k < nv) {
            load8(x + 8 * (lane + 32 * k), v[k]);
#pragma unroll
            for (int i = 0; i < 8; i++) ss += v[k][i] * v[k][i];
        }
    if (pos < 0 || pos >= a.s.npos) return;
    T *lat, *kr;
    if (paged) {
        const int b = a.seq[n], at = pos / a.s.page;
        if (b < 0 || b >= a.s.B || at >= a.s.maxpages) return;
        const int page = a.table[(long long)b * a.s.maxpages + at];
        if (page < 0 || page >= a.s.npages) return;
        lat = (T*)a.lat.p + ((long long)page * a.s.page + (pos - at * a.s.page)) * (dc + dr);
        kr = lat + dc;
    } else {
        lat = (T*)a.lat.p + n * a.lat.tok;
        kr = (T*)a.kr.p + n * a.kr.tok;
    }
    const float r = rsqrtf(warp_sum(ss) / (float)dc + a.s.eps);
#pragma unroll
    for (int k = 0; k < kMaxVec; k++)
        if (lane + 32 * k < nv) {
            float w[8];
            const float* wp = a.w + 8 * (lane + 32 * k);
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = v[k][i] * r * wp[i];
            store8(lat + 8 * (lane + 32 * k), w);
        }
    if (lane < (dr >> 4))
        rotate8<T, false>(x + dc, kr, a.rot + (long long)pos * dr, lane, dr, a.s.interleaved != 0);
}

// Gradients: with r = rsqrt(mean x^2 + eps) and g = dy w,  dx = r (g - x r^2 mean(g x)),  dw = sum_n dy x r.
// A block's warps walk tokens a fixed way apart and keep their share of dw in registers; the shares are added in a
// fixed order here and in sum_dw_kernel.
template <typename T>
__global__ void __launch_bounds__(kThreads) prep_bwd_kernel(const PrepArgs a, int lat_blocks)
{
    if ((int)blockIdx.x >= lat_blocks) {
        rotate_query<T, true>(a, a.dqr, a.dqr_out, (long long)(blockIdx.x - lat_blocks) * kThreads + threadIdx.x);
        return;
    }
    __shared__ float red[kWarps][kMaxVec * 256 / 4];   // a quarter of a latent's widest share at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int dc = a.s.dc, dr = a.s.dr, nv = dc >> 3;
    float dw[kMaxVec][8] = {};
    for (long long n = (long long)blockIdx.x * kWarps + warp; n < a.s.N; n += (long long)lat_blocks * kWarps) {
        const int pos = a.pos[n];
        T* dx = (T*)a.dkv + n * a.dkv_tok;
        if (pos < 0 || pos >= a.s.npos) {
            const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int i = lane; i < (dc + dr) >> 3; i += 32) store8(dx + 8 * i, z);
            continue;
        }
        const T* x = (const T*)a.kv + n * a.kv_tok;
        const T* dy = (const T*)a.dlat.p + n * a.dlat.tok;
        float v[kMaxVec][8], g[kMaxVec][8];
        float ss = 0.f, gx = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxVec; k++)
            if (lane + 32 * k < nv) {
                load8(x + 8 * (lane + 32 * k), v[k]);
                load8(dy + 8 * (lane + 32 * k), g[k]);
                const float* wp = a.w + 8 * (lane + 32 * k);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    ss += v[k][i] * v[k][i];
                    gx += g[k][i] * wp[i] * v[k][i];
                }
            }
        const float r = rsqrtf(warp_sum(ss) / (float)dc + a.s.eps);
        const float m = warp_sum(gx) / (float)dc * r * r;
#pragma unroll
        for (int k = 0; k < kMaxVec; k++)
            if (lane + 32 * k < nv) {
                const float* wp = a.w + 8 * (lane + 32 * k);
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    d[i] = r * (g[k][i] * wp[i] - v[k][i] * m);
                    dw[k][i] += g[k][i] * (v[k][i] * r);
                }
                store8(dx + 8 * (lane + 32 * k), d);
            }
        if (lane < (dr >> 4))
            rotate8<T, true>((const T*)a.dkr.p + n * a.dkr.tok, dx + dc, a.rot + (long long)pos * dr, lane, dr,
                             a.s.interleaved != 0);
    }
#pragma unroll
    for (int k = 0; k < kMaxVec; k++) {
        if (256 * k >= dc) break;
#pragma unroll
        for (int i = 0; i < 8; i++) red[warp][8 * lane + i] = dw[k][i];
        __syncthreads();
        const int c = 256 * k + threadIdx.x;
        if (c < dc) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; w++) s += red[w][threadIdx.x];
            a.partial[(long long)blockIdx.x * dc + c] = s;
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(1024) sum_dw_kernel(const float* part, float* dw, int blocks, int dc)
{
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < dc)
        for (int b = threadIdx.y; b < blocks; b += 32) s += part[(long long)b * dc + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dc) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i++) t += red[i][threadIdx.x];
        dw[c] = t;
    }
}

long long query_blocks(const gdn_mla_prep_t& s)
{
    return ((long long)s.N * s.H * (s.dr >> 4) + kThreads - 1) / kThreads;
}

}  // namespace

// blocks that walk the tokens of the backward pass: two resident on each SM, or one a token's warp
int prep_bwd_blocks(int N)
{
    const int need = (N + kWarps - 1) / kWarps;
    return need < 1 ? 1 : (need < 2 * 152 ? need : 2 * 152);
}

cudaError_t launch_prep(const PrepArgs& a, cudaStream_t st)
{
    const int lat = (a.s.N + kWarps - 1) / kWarps;
    const long long grid = lat + query_blocks(a.s);
    if (grid == 0) return cudaSuccess;
    if (a.s.io == GDN_BF16)
        prep_kernel<__nv_bfloat16><<<(unsigned)grid, kThreads, 0, st>>>(a, lat);
    else
        prep_kernel<float><<<(unsigned)grid, kThreads, 0, st>>>(a, lat);
    return cudaGetLastError();
}

cudaError_t launch_prep_bwd(const PrepArgs& a, cudaStream_t st)
{
    const int lat = prep_bwd_blocks(a.s.N);
    const long long grid = lat + query_blocks(a.s);
    if (a.s.io == GDN_BF16)
        prep_bwd_kernel<__nv_bfloat16><<<(unsigned)grid, kThreads, 0, st>>>(a, lat);
    else
        prep_bwd_kernel<float><<<(unsigned)grid, kThreads, 0, st>>>(a, lat);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    sum_dw_kernel<<<(a.s.dc + 31) / 32, dim3(32, 32), 0, st>>>(a.partial, a.dw, lat, a.s.dc);
    return cudaGetLastError();
}

}  // namespace mla
}  // namespace gdn
