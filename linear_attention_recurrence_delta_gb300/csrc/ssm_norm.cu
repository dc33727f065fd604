// ssm_norm.cu -- residual addition and RMS norm, in the I/O type or in 8 bits, with the gradients.
//
// y = s / sqrt(mean s^2 + eps) w of s = x + res.  Each value is read once and written once, so HBM bounds it: a row
// stays in the registers of its threads, 8 values a piece, between the sum over it and the results.  32768 rows of 2048 bf16
// values: 75 us forwards (537 MB, 81 % of DRAM's time), 93 us for the gradients (the next row asked for ahead; 187 without) and
// 6 for the sum of dw's shares.  5371 rows of 4096 with a 32-bit residual, in 8 bits: 40 us (243 MB); two pieces a thread and
// more threads a row, not four (46 us), because more warps then wait for memory.
#include <cuda_fp8.h>
#include <float.h>

#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

namespace {

constexpr int kThreads = 256, kMostThreads = 512;      // of a block: as a rule, and for the widest rows
constexpr float kE4m3Top = 448.f, kScaleFloor = 1e-30f;

// What the 2^l threads of a row hold, joined in a fixed order; red: a place for each warp and kind of value, in turn one of
// two, so that a barrier is enough.
template <int K, bool MAX>
__device__ __forceinline__ void row_join(float (&x)[K], int l, float (*red)[kMostThreads / 32])
{
#pragma unroll
    for (int m = 16; m; m >>= 1)
#pragma unroll
        for (int k = 0; k < K; k++) {
            const float o = __shfl_xor_sync(0xffffffffu, x[k], m);
            x[k] = MAX ? max_nan(x[k], o) : x[k] + o;
        }
    if (l == 5) return;
    const int w = threadIdx.x >> 5, first = w >> (l - 5) << (l - 5);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; k++) red[k][w] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; k++) {
        x[k] = red[k][first];
        for (int i = 1; i < 1 << (l - 5); i++) x[k] = MAX ? max_nan(x[k], red[k][first + i]) : x[k] + red[k][first + i];
    }
}

// the value as the residual's type holds it
__device__ __forceinline__ float held(float x, const float*) { return x; }
__device__ __forceinline__ float held(float x, const __nv_bfloat16*) { return __bfloat162float(__float2bfloat16_rn(x)); }

__device__ __forceinline__ void store8_e4m3(void* p, const float (&x)[8])
{
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i], x[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[4 * i + 2], x[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | hi << 16;
    }
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// 2^l threads a row, V pieces of 8 values each
template <typename IO, typename RES, int V, bool E4M3>
__global__ void __launch_bounds__(V > 2 ? kMostThreads : kThreads) norm_kernel(const NormArgs a, int l)
{
    __shared__ float red[2][kMostThreads / 32];
    const int per = blockDim.x >> l, t = threadIdx.x & ((1 << l) - 1), D = a.s.D;
    const long long n = (long long)blockIdx.x * per + (threadIdx.x >> l);
    const bool row = n < a.s.N;
    float v[V][8];
    Raw8<IO> rx[V];
    Raw8<RES> rr[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = 8 * (t + (i << l));
        if (row && c < D) {
            rx[i] = raw8((const IO*)a.x + n * a.x_tok + c);
            if (a.res) rr[i] = raw8((const RES*)a.res + n * a.res_tok + c);
        }
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = 8 * (t + (i << l));
        const bool in = row && c < D;
#pragma unroll
        for (int k = 0; k < 8; k++) v[i][k] = 0.f;
        if (!in) continue;
        values(rx[i], v[i]);
        if (a.res) {
            float r[8];
            values(rr[i], r);
#pragma unroll
            for (int k = 0; k < 8; k++) v[i][k] += r[k];
        }
#pragma unroll
        for (int k = 0; k < 8; k++) {
            v[i][k] = held(v[i][k], (const RES*)nullptr);
            ss[0] = fmaf(v[i][k], v[i][k], ss[0]);
        }
        if (a.sum) store8((RES*)a.sum + n * a.sum_tok + c, v[i]);
    }
    row_join<1, false>(ss, l, red);
    const float inv = rsqrtf(ss[0] / D + a.s.eps);
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = 8 * (t + (i << l));
        if (!row || c >= D) continue;
        float w[8];
        load8(a.w + c, w);
#pragma unroll
        for (int k = 0; k < 8; k++) {
            v[i][k] = v[i][k] * inv * w[k];
            if (E4M3) top = max_nan(top, fabsf(v[i][k]));
        }
        if (!E4M3) store8((IO*)a.y + n * a.y_tok + c, v[i]);
    }
    if (!E4M3) return;
    if (a.s.group == 0) {
        float m[1] = {top};
        row_join<1, true>(m, l, red + 1);
        top = m[0];
        if (row && t == 0) a.scale[n] = max_nan(top, kScaleFloor) * (1.f / kE4m3Top);
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = 8 * (t + (i << l));
        if (a.s.group) {
            top = 0.f;
#pragma unroll
            for (int k = 0; k < 8; k++) top = max_nan(top, fabsf(v[i][k]));
            for (int m = a.s.group >> 4; m; m >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
            if (row && c < D && c % a.s.group == 0)
                a.scale[n * (D / a.s.group) + c / a.s.group] = max_nan(top, kScaleFloor) * (1.f / kE4m3Top);
        }
        if (!row || c >= D) continue;
        const float to = kE4m3Top / max_nan(top, kScaleFloor);
#pragma unroll
        for (int k = 0; k < 8; k++) v[i][k] *= to;
        store8_e4m3((uint8_t*)a.y + n * a.y_tok + c, v[i]);
    }
}

// One row's inputs as they lie in memory.
template <typename IO, typename RES, int V>
struct BackRow {
    Raw8<RES> s[V], ds[V];
    Raw8<IO> dy[V];
    __device__ __forceinline__ void load(const NormArgs& a, long long n, int t, int l)
    {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = 8 * (t + (i << l));
            s[i] = ds[i] = Raw8<RES>{};
            dy[i] = Raw8<IO>{};
            if (n >= a.s.N || c >= a.s.D) continue;
            s[i] = raw8((const RES*)a.res + n * a.res_tok + c);
            dy[i] = raw8((const IO*)a.dy + n * a.dy_tok + c);
            if (a.dsum) ds[i] = raw8((const RES*)a.dsum + n * a.dsum_tok + c);
        }
    }
};

// d = inv (gw - s inv^2 mean(gw s)) + ds with gw = dy w; dw's share of the block's rows stays in registers until the end.
// AHEAD: the next row is asked for before this one is worked on (rows of up to 4096 values, whose registers allow it).
template <typename IO, typename RES, int V, bool AHEAD>
__global__ void __launch_bounds__(V > 2 ? kMostThreads : kThreads, V > 2 ? 1 : 2) norm_bwd_kernel(const NormArgs a, int l)
{
    __shared__ float red[2][2][kMostThreads / 32];
    extern __shared__ __align__(16) float dws[];      // [rows a block][D], where a block takes several rows
    const int per = blockDim.x >> l, sub = threadIdx.x >> l, t = threadIdx.x & ((1 << l) - 1), D = a.s.D;
    const long long stride = (long long)gridDim.x * per;
    float dw[V][8] = {}, w[AHEAD ? V : 1][8] = {};
    if (AHEAD)
#pragma unroll
        for (int i = 0; i < V; i++)
            if (8 * (t + (i << l)) < D) load8(a.w + 8 * (t + (i << l)), w[AHEAD ? i : 0]);
    BackRow<IO, RES, V> next;
    int turn = 0;
    if (AHEAD) next.load(a, (long long)blockIdx.x * per + sub, t, l);
    for (long long n0 = (long long)blockIdx.x * per; n0 < a.s.N; n0 += stride, turn ^= 1) {
        const long long n = n0 + sub;
        if (!AHEAD) next.load(a, n, t, l);
        const BackRow<IO, RES, V> row = next;
        if (AHEAD) next.load(a, n + stride, t, l);
        float sums[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < V; i++) {
            float s[8], g[8];
            values(row.s[i], s);
            values(row.dy[i], g);
            if (!AHEAD && 8 * (t + (i << l)) < D) load8(a.w + 8 * (t + (i << l)), w[0]);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                sums[0] = fmaf(s[k], s[k], sums[0]);
                sums[1] = fmaf(g[k] * w[AHEAD ? i : 0][k], s[k], sums[1]);
            }
        }
        row_join<2, false>(sums, l, red[turn]);
        const float inv = rsqrtf(sums[0] / D + a.s.eps), back = inv * inv * (sums[1] / D);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = 8 * (t + (i << l));
            if (n >= a.s.N || c >= D) continue;
            float s[8], g[8], d[8];
            values(row.s[i], s);
            values(row.dy[i], g);
            values(row.ds[i], d);
            if (!AHEAD) load8(a.w + c, w[0]);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                dw[i][k] = fmaf(g[k] * s[k], inv, dw[i][k]);
                d[k] += inv * (g[k] * w[AHEAD ? i : 0][k] - s[k] * back);
            }
            if (a.dx) store8((IO*)a.dx + n * a.dx_tok + c, d);
            if (a.dres) store8((RES*)a.dres + n * a.dres_tok + c, d);
        }
    }
    if (per > 1) {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = 8 * (t + (i << l));
            if (c < D) store8(dws + sub * D + c, dw[i]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < D; c += blockDim.x) {
            float x = dws[c];
            for (int i = 1; i < per; i++) x += dws[i * D + c];
            a.partial[(long long)blockIdx.x * D + c] = x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = 8 * (t + (i << l));
            if (c < D) store8(a.partial + (long long)blockIdx.x * D + c, dw[i]);
        }
    }
}

// threads a row as a power of two, and pieces each
struct Split {
    int l, V, block;
};
Split split(int D)
{
    Split s;
    s.V = D <= 256 ? 1 : D <= 4096 ? 2 : 4;
    s.l = 5;
    while ((8 * s.V) << s.l < D) s.l++;
    s.block = (1 << s.l) > kThreads ? 1 << s.l : kThreads;
    return s;
}

template <typename IO, typename RES>
cudaError_t launch_typed(const NormArgs& a, cudaStream_t st)
{
    const Split p = split(a.s.D);
    const int per = p.block >> p.l;
    const unsigned grid = (unsigned)((a.s.N + per - 1) / per);
    if (a.s.out == GDN_E4M3) {
        if (p.V == 1) norm_kernel<IO, RES, 1, true><<<grid, p.block, 0, st>>>(a, p.l);
        else if (p.V == 2) norm_kernel<IO, RES, 2, true><<<grid, p.block, 0, st>>>(a, p.l);
        else norm_kernel<IO, RES, 4, true><<<grid, p.block, 0, st>>>(a, p.l);
    } else {
        if (p.V == 1) norm_kernel<IO, RES, 1, false><<<grid, p.block, 0, st>>>(a, p.l);
        else if (p.V == 2) norm_kernel<IO, RES, 2, false><<<grid, p.block, 0, st>>>(a, p.l);
        else norm_kernel<IO, RES, 4, false><<<grid, p.block, 0, st>>>(a, p.l);
    }
    return cudaGetLastError();
}

template <typename IO, typename RES>
cudaError_t launch_bwd_typed(const NormArgs& a, cudaStream_t st)
{
    const Split p = split(a.s.D);
    const int per = p.block >> p.l;
    const size_t smem = per > 1 ? (size_t)per * a.s.D * sizeof(float) : 0;
    const unsigned grid = norm_bwd_blocks(a.s);
    if (p.V == 1) norm_bwd_kernel<IO, RES, 1, true><<<grid, p.block, smem, st>>>(a, p.l);
    else if (p.V == 2) norm_bwd_kernel<IO, RES, 2, true><<<grid, p.block, smem, st>>>(a, p.l);
    else norm_bwd_kernel<IO, RES, 4, false><<<grid, p.block, smem, st>>>(a, p.l);
    return cudaGetLastError();
}

// 32 columns a block; the rows are dealt to its R warps in turn, whose sums are then added in their order
template <int R>
__global__ void __launch_bounds__(32 * R) column_sums_kernel(const ColumnSums s)
{
    cudaGridDependencySynchronize();      // launched as a dependent of the kernel that writes the shares
    __shared__ float part[R][33];
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long c = (long long)blockIdx.x * 32 + lane;
    float x = 0.f;
    if (c < s.cols)
#pragma unroll 8
        for (int r = w; r < s.rows; r += R) x += s.partial[r * s.cols + c];
    part[w][lane] = x;
    __syncthreads();
    if (w || c >= s.cols) return;
#pragma unroll
    for (int i = 1; i < R; i++) x += part[i][lane];
    if (c < s.a) {
        if (s.out_a) s.out_a[c] = s.decay ? x * max_nan(-expf(s.decay[c]), -FLT_MAX) : x;
    } else if (c < s.a + s.b) {
        if (s.out_b) s.out_b[c - s.a] = x;
    } else if (s.out_c) {
        s.out_c[c - s.a - s.b] = x;
    }
}

}  // namespace

// blocks that share the rows of a backward pass: as many as run at once, each with its row of shares of dw
int norm_bwd_blocks(const gdn_norm_t& s)
{
    const Split p = split(s.D);
    const long long need = ((long long)s.N * (1 << p.l) + p.block - 1) / p.block;
    const int most = 152 * 2 * kThreads / p.block;
    return need < 1 ? 1 : need < most ? (int)need : most;
}

cudaError_t launch_column_sums(const ColumnSums& s, cudaStream_t st)
{
    const dim3 grid((unsigned)((s.cols + 31) / 32));
    // shares of a scan's few sequences: many columns instead
    return s.rows <= 64 ? launch_after(column_sums_kernel<4>, grid, 128, 0, st, s) : launch_after(column_sums_kernel<32>, grid, 1024, 0, st, s);
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st)
{
    if (a.s.N == 0) return cudaSuccess;
    if (a.s.io == GDN_F32) return launch_typed<float, float>(a, st);
    return a.s.res == GDN_F32 ? launch_typed<__nv_bfloat16, float>(a, st) : launch_typed<__nv_bfloat16, __nv_bfloat16>(a, st);
}

cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st)
{
    const cudaError_t e = a.s.io == GDN_F32      ? launch_bwd_typed<float, float>(a, st)
                          : a.s.res == GDN_F32 ? launch_bwd_typed<__nv_bfloat16, float>(a, st)
                                               : launch_bwd_typed<__nv_bfloat16, __nv_bfloat16>(a, st);
    if (e != cudaSuccess) return e;
    ColumnSums c = {};
    c.partial = a.partial;
    c.rows = norm_bwd_blocks(a.s);
    c.cols = c.a = a.s.D;
    c.out_a = a.dw;
    return launch_column_sums(c, st);
}

}  // namespace ssm
}  // namespace gdn
