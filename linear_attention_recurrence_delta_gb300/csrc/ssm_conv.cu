// ssm_conv.cu -- short causal convolution of each channel with SiLU, its gradients, and its form for new tokens.
//
// pre[t] = bias + sum_k w[k] x[t - W + 1 + k], y = silu(pre).  A thread walks a strip of time for a few neighbouring
// channels with the last W - 1 rows in registers, so that a row is read once (and W - 1 rows more a strip, from L2);
// HBM bounds it.
#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

namespace {

constexpr int kThreads = 256;
constexpr int kStrip = 32;        // rows a thread walks forwards
constexpr int kAhead = 4;         // rows asked for together
constexpr int kBackStrip = 64;    // rows a thread walks for the gradients

__device__ __forceinline__ void load4(const float* p, float (&x)[4])
{
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&x)[4])
{
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4])
{
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&x)[4])
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// the taps of C channels: w[k][c] of [D, W]
template <int W, int C>
__device__ __forceinline__ void load_taps(const float* w, float (&t)[W][C])
{
    float raw[W * C];
#pragma unroll
    for (int i = 0; i < W * C / 4; i++) {
        const float4 v = reinterpret_cast<const float4*>(w)[i];
        raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int k = 0; k < W; k++)
#pragma unroll
        for (int c = 0; c < C; c++) t[k][c] = raw[c * W + k];
}

// one row: the output of 8 channels from the rows before it and this one, which then joins them
template <int W>
__device__ __forceinline__ void step8(const float (&taps)[W][8], const float (&bias)[8], float (&past)[W - 1][8], const float (&x)[8],
                                      int silu, float (&y)[8])
{
#pragma unroll
    for (int c = 0; c < 8; c++) {
        float p = bias[c];
#pragma unroll
        for (int k = 0; k < W - 1; k++) p = fmaf(taps[k][c], past[k][c], p);
        p = fmaf(taps[W - 1][c], x[c], p);
        y[c] = silu ? p * sigmoid(p) : p;
#pragma unroll
        for (int k = 0; k + 1 < W - 1; k++) past[k][c] = past[k + 1][c];
        past[W - 2][c] = x[c];
    }
}

// Sequence blockIdx.y; threads run over (strip, piece of 8 channels), pieces fastest.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ConvArgs a)
{
    const int D = a.s.D, pieces = D >> 3, b = blockIdx.y;
    const long long u = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int strip = (int)(u / pieces), c = (int)(u - (long long)strip * pieces) << 3;
    const Rows r = rows_of(a.cu, b, a.s.T, a.s.rows);
    const long long t0 = (long long)strip * kStrip;
    if (t0 >= r.n && strip > 0) return;
    const int end = (int)min((long long)r.n, t0 + kStrip);
    const IO* x = (const IO*)a.x.p + (long long)r.first * a.x.tok + c;
    IO* y = (IO*)a.y.p + (long long)r.first * a.y.tok + c;
    float taps[W][8], bias[8] = {}, past[W - 1][8];
    load_taps<W, 8>(a.w + (long long)c * W, taps);
    if (a.bias) load8(a.bias + c, bias);
#pragma unroll
    for (int k = 0; k < W - 1; k++) {
        const long long t = t0 - (W - 1) + k;
        if (t >= 0) load8(x + t * a.x.tok, past[k]);
        else if (a.s0) load8((const IO*)a.s0 + ((long long)b * (W - 1) + t + W - 1) * D + c, past[k]);
        else
#pragma unroll
            for (int i = 0; i < 8; i++) past[k][i] = 0.f;
    }
    for (int t = (int)t0; t < end; t += kAhead) {
        Raw8<IO> raw[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; j++)
            if (t + j < end) raw[j] = raw8(x + (long long)(t + j) * a.x.tok);
#pragma unroll
        for (int j = 0; j < kAhead; j++)
            if (t + j < end) {
                float v[8], o[8];
                values(raw[j], v);
                step8<W>(taps, bias, past, v, a.s.silu, o);
                store8(y + (long long)(t + j) * a.y.tok, o);
            }
    }
    if (a.sT && end == r.n)
#pragma unroll
        for (int k = 0; k < W - 1; k++) store8((IO*)a.sT + ((long long)b * (W - 1) + k) * D + c, past[k]);
}

// New tokens: a thread has 8 channels of a sequence.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvStepArgs a)
{
    const int D = a.s.D, pieces = D >> 3;
    const long long u = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int b = (int)(u / pieces), c = (int)(u - (long long)b * pieces) << 3;
    if (b >= a.s.B) return;
    const int src = a.src ? a.src[b] : b, dst = a.dst ? a.dst[b] : src;
    const IO* x = (const IO*)a.x.p + (long long)b * a.s.T * a.x.tok + c;
    IO* y = (IO*)a.y.p + (long long)b * a.s.T * a.y.tok + c;
    float taps[W][8], bias[8] = {}, past[W - 1][8];
    load_taps<W, 8>(a.w + (long long)c * W, taps);
    if (a.bias) load8(a.bias + c, bias);
#pragma unroll
    for (int k = 0; k < W - 1; k++) {
        if (src >= 0 && src < a.s.slots) load8((const IO*)a.state + ((long long)src * (W - 1) + k) * D + c, past[k]);
        else
#pragma unroll
            for (int i = 0; i < 8; i++) past[k][i] = 0.f;
    }
    for (int t = 0; t < a.s.T; t++) {
        float v[8], o[8];
        load8(x + t * a.x.tok, v);
        step8<W>(taps, bias, past, v, a.s.silu, o);
        store8(y + t * a.y.tok, o);
    }
    if (dst >= 0 && dst < a.s.slots)
#pragma unroll
        for (int k = 0; k < W - 1; k++) store8((IO*)a.state + ((long long)dst * (W - 1) + k) * D + c, past[k]);
}

// Gradients.  dpre = dy silu'(pre), dx[r] = sum_k w[k] dpre[r + W - 1 - k], dw[k] = sum_t dpre[t] x[t - W + 1 + k].
// A thread has 4 channels and keeps their sums of dw and dbias over the strips that its block takes: strip by strip of all
// sequences in turn, `2^l` pieces of channels by kThreads >> l strips at a time.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(const ConvArgs a, int l)
{
    __shared__ float4 share[kThreads];
    const int D = a.s.D, tx = threadIdx.x & ((1 << l) - 1), ty = threadIdx.x >> l, strips = kThreads >> l;
    const int c = 4 * ((blockIdx.x << l) + tx);
    const int each = (a.s.T + kBackStrip - 1) / kBackStrip;      // strips of a sequence, one at least
    const long long items = (long long)a.s.B * (each > 0 ? each : 1);
    float taps[W][4], bias[4] = {}, dw[W][4] = {}, db[4] = {};
    if (c < D) {
        load_taps<W, 4>(a.w + (long long)c * W, taps);
        if (a.bias) load4(a.bias + c, bias);
    }
    for (long long item = (long long)blockIdx.y * strips + ty; item < items && c < D; item += (long long)gridDim.y * strips) {
        const int b = (int)(item / (each > 0 ? each : 1)), t0 = (int)(item - (long long)b * (each > 0 ? each : 1)) * kBackStrip;
        const Rows r = rows_of(a.cu, b, a.s.T, a.s.rows);
        if (t0 >= r.n && t0 > 0) continue;
        const int end = min(r.n, t0 + kBackStrip);
        const IO* x = (const IO*)a.x.p + (long long)r.first * a.x.tok + c;
        const IO* dy = (const IO*)a.dy.p + (long long)r.first * a.dy.tok + c;
        IO* dx = (IO*)a.dx.p + (long long)r.first * a.dx.tok + c;
        float past[W - 1][4], d[W][4] = {};      // earlier rows of x; dpre of this row (last) and those before it
#pragma unroll
        for (int k = 0; k < W - 1; k++) {
            const int t = t0 - (W - 1) + k;
            if (t >= 0) load4(x + (long long)t * a.x.tok, past[k]);
            else if (a.s0) load4((const IO*)a.s0 + ((long long)b * (W - 1) + t + W - 1) * D + c, past[k]);
            else
#pragma unroll
                for (int i = 0; i < 4; i++) past[k][i] = 0.f;
        }
        for (int t = t0; t < end + W - 1; t++) {
#pragma unroll
            for (int k = 0; k + 1 < W; k++)
#pragma unroll
                for (int i = 0; i < 4; i++) d[k][i] = d[k + 1][i];
#pragma unroll
            for (int i = 0; i < 4; i++) d[W - 1][i] = 0.f;
            if (t < r.n) {
                float v[4], g[4];
                load4(x + (long long)t * a.x.tok, v);
                load4(dy + (long long)t * a.dy.tok, g);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    float p = bias[i];
#pragma unroll
                    for (int k = 0; k < W - 1; k++) p = fmaf(taps[k][i], past[k][i], p);
                    p = fmaf(taps[W - 1][i], v[i], p);
                    if (a.s.silu) {
                        const float s = sigmoid(p);
                        g[i] *= s * fmaf(p, 1.f - s, 1.f);
                    }
                    d[W - 1][i] = g[i];
                    if (t < end) {
                        db[i] += g[i];
#pragma unroll
                        for (int k = 0; k < W - 1; k++) dw[k][i] = fmaf(g[i], past[k][i], dw[k][i]);
                        dw[W - 1][i] = fmaf(g[i], v[i], dw[W - 1][i]);
                    }
#pragma unroll
                    for (int k = 0; k + 1 < W - 1; k++) past[k][i] = past[k + 1][i];
                    past[W - 2][i] = v[i];
                }
            }
            const int row = t - (W - 1);             // all rows that see it are done
            if (row < t0 && !(t0 == 0 && a.ds0)) continue;
            float o[4] = {};
#pragma unroll
            for (int k = 0; k < W; k++)
#pragma unroll
                for (int i = 0; i < 4; i++) o[i] = fmaf(taps[k][i], d[W - 1 - k][i], o[i]);
            const int kept = row - (r.n - (W - 1));  // its place in the new state
            if (a.dsT && kept >= 0) {
                float e[4];
                load4((const IO*)a.dsT + ((long long)b * (W - 1) + kept) * D + c, e);
#pragma unroll
                for (int i = 0; i < 4; i++) o[i] += e[i];
            }
            if (row >= 0) store4(dx + (long long)row * a.dx.tok, o);
            else store4((IO*)a.ds0 + ((long long)b * (W - 1) + row + W - 1) * D + c, o);
        }
    }
    // the strips' sums in their order
    float* out = a.partial + (long long)blockIdx.y * D * (W + 1);
#pragma unroll
    for (int k = 0; k <= W; k++) {
        const float(&s)[4] = k < W ? dw[k < W ? k : 0] : db;
        __syncthreads();
        share[threadIdx.x] = make_float4(s[0], s[1], s[2], s[3]);
        __syncthreads();
        if (ty == 0 && c < D) {
            float4 x = share[tx];
            for (int i = 1; i < strips; i++) {
                const float4 y = share[tx + (i << l)];
                x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
            }
            if (k < W) {
                out[(long long)c * W + k] = x.x;
                out[(long long)(c + 1) * W + k] = x.y;
                out[(long long)(c + 2) * W + k] = x.z;
                out[(long long)(c + 3) * W + k] = x.w;
            } else {
                *reinterpret_cast<float4*>(out + (long long)D * W + c) = x;
            }
        }
    }
}

// pieces of 4 channels a block takes side by side, as a power of two
int back_pieces(const gdn_conv_t& s)
{
    int l = 1;
    while (l < 5 && (4 << l) < s.D) l++;
    return l;
}

template <typename IO, int W>
cudaError_t launch_fwd_w(const ConvArgs& a, cudaStream_t st)
{
    const long long strips = (a.s.T + kStrip - 1) / kStrip, units = (strips > 0 ? strips : 1) * (a.s.D >> 3);
    conv_kernel<IO, W><<<dim3((unsigned)((units + kThreads - 1) / kThreads), a.s.B), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename IO, int W>
cudaError_t launch_step_w(const ConvStepArgs& a, cudaStream_t st)
{
    const long long units = (long long)a.s.B * (a.s.D >> 3);
    conv_step_kernel<IO, W><<<(unsigned)((units + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename IO, int W>
cudaError_t launch_bwd_w(const ConvArgs& a, cudaStream_t st)
{
    const int l = back_pieces(a.s), wide = ((a.s.D >> 2) + (1 << l) - 1) >> l;
    conv_bwd_kernel<IO, W><<<dim3(wide, conv_bwd_blocks(a.s)), kThreads, 0, st>>>(a, l);
    return cudaGetLastError();
}

#define GDN_BY_TYPE(fn, a, st)                                                                                        \
    ((a).s.io == GDN_BF16 ? ((a).s.W == 2   ? fn<__nv_bfloat16, 2>(a, st)                                             \
                             : (a).s.W == 3 ? fn<__nv_bfloat16, 3>(a, st)                                             \
                                            : fn<__nv_bfloat16, 4>(a, st))                                            \
                          : ((a).s.W == 2   ? fn<float, 2>(a, st)                                                     \
                             : (a).s.W == 3 ? fn<float, 3>(a, st)                                                     \
                                            : fn<float, 4>(a, st)))

}  // namespace

// blocks that share the strips of a block's channels: as many as run at once
int conv_bwd_blocks(const gdn_conv_t& s)
{
    const int l = back_pieces(s), wide = ((s.D >> 2) + (1 << l) - 1) >> l, strips = kThreads >> l;
    const long long each = (s.T + kBackStrip - 1) / kBackStrip, items = (long long)s.B * (each > 0 ? each : 1);
    const long long need = (items + strips - 1) / strips, most = 152 * 4 / wide;
    return need < most ? (int)need : most < 1 ? 1 : (int)most;
}

cudaError_t launch_conv(const ConvArgs& a, cudaStream_t st) { return GDN_BY_TYPE(launch_fwd_w, a, st); }
cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t st) { return GDN_BY_TYPE(launch_step_w, a, st); }
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t st)
{
    const cudaError_t e = GDN_BY_TYPE(launch_bwd_w, a, st);
    if (e != cudaSuccess) return e;
    ColumnSums c = {};
    c.partial = a.partial;
    c.rows = conv_bwd_blocks(a.s);
    c.cols = (long long)a.s.D * (a.s.W + 1);
    c.a = (long long)a.s.D * a.s.W;
    c.b = a.s.D;
    c.out_a = a.dw;
    c.out_b = a.dbias;
    return launch_column_sums(c, st);
}

}  // namespace ssm
}  // namespace gdn
