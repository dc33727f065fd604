// ssm_scan_fwd.cu -- the selective scan forwards.
//
// h[t] = exp(delta[t] A) h[t-1] + delta[t] x[t] B[t], y[t] = (h[t] . C[t] + D x[t]) silu(z[t]).  Tiles of tokens are
// staged in shared memory with their step sizes; each lane then walks the tile with its states in registers, and the
// tile's outputs leave through shared memory in rows again.  An exponential a state and token bounds it.
// Where sequences are few, segments of time run side by side: a first launch takes each segment's states from zero and
// the sum of its step sizes; since a segment turns the state h it gets into exp(A sum delta) h + (its state from zero), each
// segment of the second launch finds its own entering state from those of the segments before it.
#include "ssm_scan_common.cuh"

namespace gdn {
namespace ssm {

namespace {

template <typename IO, int LS, bool FIRST>      // FIRST: the first of the two launches
__global__ void __launch_bounds__(kScanThreads) scan_kernel(const ScanArgs a, int blocks)
{
    using L = Lay<LS>;
    constexpr int K = LS == 2 ? 16 : 32, UNITS = K * L::PP, U = (UNITS + kScanThreads - 1) / kScanThreads;
    __shared__ float2 sd[K][L::CH];            // delta, delta x
    __shared__ float sB[K][L::NS], sC[FIRST ? 1 : K][L::NS], sy[FIRST ? 1 : K][L::CH];
    const Spot p = spot<L>(a, blocks);
    const int D = a.s.D, N = a.s.N, cl = threadIdx.x / LS, q = threadIdx.x % LS, d = p.d0 + cl;
    const bool mine = cl < p.channels && 4 * q < N;
    if (FIRST && p.t0 >= p.t1) return;
    const long long at = ((long long)p.b * D + d) * N + 4 * q, all = (long long)a.s.B * D;
    float A[4], h[4] = {}, sum = 0.f;
    load_rates(a, d, 4 * q, mine, A);
    if (!FIRST && mine) {
        if (a.h0) get4(a.h0 + at, h);
        for (int s = 0; s < p.seg && (long long)s * a.seg_len < p.r.n; s++) {
            float e[4];
            const float w = a.seg_d[s * all + (long long)p.b * D + d];
            get4(a.seg_h + s * all * N + at, e);
#pragma unroll
            for (int i = 0; i < 4; i++) h[i] = fmaf(ex2_approx(w * A[i]), h[i], e[i]);
        }
    }
    float bias[U][8], skip[U][8];
#pragma unroll
    for (int u = 0; u < U; u++) {
        const int unit = u * kScanThreads + threadIdx.x, c = 8 * (unit % L::PP);
#pragma unroll
        for (int i = 0; i < 8; i++) bias[u][i] = skip[u][i] = 0.f;
        if (unit < UNITS && c < p.channels) {
            if (a.dt_bias) load8(a.dt_bias + p.d0 + c, bias[u]);
            if (!FIRST && a.D_skip) load8(a.D_skip + p.d0 + c, skip[u]);
        }
    }
    for (int t0 = p.t0; t0 < p.t1; t0 += K) {
        float x[U][8];
        __syncthreads();      // the last tile's outputs have left
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int unit = u * kScanThreads + threadIdx.x, j = unit / L::PP, c = 8 * (unit % L::PP);
            if (unit >= UNITS) continue;
            float v[8];
            const bool in = t0 + j < p.t1 && c < p.channels;
#pragma unroll
            for (int i = 0; i < 8; i++) x[u][i] = v[i] = 0.f;
            if (in) {
                const long long row = p.r.first + t0 + j;
                load8((const IO*)a.x.p + row * a.x.tok + p.d0 + c, x[u]);
                load8((const IO*)a.dt.p + row * a.dt.tok + p.d0 + c, v);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
                float slope, w = v[i] + bias[u][i];
                if (a.s.softplus) w = softplus(w, slope);
                if (!in) w = 0.f;          // a step of size zero changes nothing
                sd[j][c + i] = f2(w, w * x[u][i]);
            }
        }
        stage_vectors<L, IO, K>(a, a.Bm, p, t0, p.t1, sB);
        if (!FIRST) stage_vectors<L, IO, K>(a, a.Cm, p, t0, p.t1, sC);
        __syncthreads();
#pragma unroll 4
        for (int j = 0; j < K; j++) {
            if (!FIRST && a.saved && j % kSaveEvery == 0 && mine && t0 + j < p.t1)
                put4(a.saved + (saved_at(p, t0 + j) * D + d) * N + 4 * q, h);
            const float2 v = sd[j][cl];
            float B[4], C[4], y = 0.f;
            get4(&sB[j][4 * q], B);
            if (!FIRST) get4(&sC[j][4 * q], C);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                h[i] = fmaf(ex2_approx(v.x * A[i]), h[i], v.y * B[i]);
                if (!FIRST) y = fmaf(h[i], C[i], y);
            }
            if (FIRST) {
                sum += v.x;
            } else {
                y = lanes_sum<LS>(y);
                if (q == 0) sy[j][cl] = y;
            }
        }
        if (FIRST) continue;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int unit = u * kScanThreads + threadIdx.x, j = unit / L::PP, c = 8 * (unit % L::PP);
            if (unit >= UNITS || t0 + j >= p.t1 || c >= p.channels) continue;
            const long long row = p.r.first + t0 + j;
            float y[8];
            load8(&sy[j][c], y);
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] = fmaf(skip[u][i], x[u][i], y[i]);
            if (a.z.p) {
                float z[8];
                load8((const IO*)a.z.p + row * a.z.tok + p.d0 + c, z);
#pragma unroll
                for (int i = 0; i < 8; i++) y[i] *= z[i] * sigmoid(z[i]);
            }
            store8((IO*)a.y.p + row * a.y.tok + p.d0 + c, y);
        }
    }
    if (FIRST) {
        if (mine) put4(a.seg_h + p.seg * all * N + at, h);
        if (mine && q == 0) a.seg_d[p.seg * all + (long long)p.b * D + d] = sum;
    } else if (mine && a.hT && p.t1 == p.r.n && (p.t0 < p.t1 || p.seg == 0)) {
        put4(a.hT + at, h);
    }
}

template <typename IO, int LS>
cudaError_t launch_lanes(const ScanArgs& a, cudaStream_t st)
{
    const ScanPlan plan = scan_plan(a.s, 0);
    const dim3 grid(a.s.G * plan.blocks, a.s.B, a.segments);
    if (a.segments > 1) scan_kernel<IO, LS, true><<<grid, kScanThreads, 0, st>>>(a, plan.blocks);
    scan_kernel<IO, LS, false><<<grid, kScanThreads, 0, st>>>(a, plan.blocks);
    return cudaGetLastError();
}
template <typename IO>
cudaError_t launch_typed(const ScanArgs& a, cudaStream_t st)
{
    if (a.s.N <= 8) return launch_lanes<IO, 2>(a, st);
    if (a.s.N <= 16) return launch_lanes<IO, 4>(a, st);
    return a.s.N <= 32 ? launch_lanes<IO, 8>(a, st) : launch_lanes<IO, 16>(a, st);
}

// New tokens: a lane has 4 states of a channel, and takes the sequences blockIdx.y, blockIdx.y + gridDim.y, ... in turn.
constexpr int kStepThreads = 128;
template <typename IO, int LS>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(const ScanStepArgs a)
{
    const int N = a.s.N, D = a.s.D, q = threadIdx.x % LS;
    const int u = (blockIdx.x * kStepThreads + threadIdx.x) / LS, d = min(u, D - 1), g = d / (D / a.s.G), n = 4 * q;
    const bool mine = u < D && n < N;
    float A[4] = {}, bias = a.dt_bias ? a.dt_bias[d] : 0.f, skip = a.D_skip ? a.D_skip[d] : 0.f;
    if (mine) {
        get4(a.A_log + (long long)d * N + n, A);
#pragma unroll
        for (int i = 0; i < 4; i++) A[i] = -expf(A[i]) * kLog2e;
    }
    for (int b = blockIdx.y; b < a.s.B; b += gridDim.y) {
        const int src = a.src ? a.src[b] : b, dst = a.dst ? a.dst[b] : src;
        float h[4] = {};
        if (mine && src >= 0 && src < a.s.slots) get4(a.state + ((long long)src * D + d) * N + n, h);
        for (int t = 0; t < a.s.T; t++) {
            const long long row = (long long)b * a.s.T + t;
            const float x = rec::to_f(((const IO*)a.x.p)[row * a.x.tok + d]);
            float w = rec::to_f(((const IO*)a.dt.p)[row * a.dt.tok + d]) + bias, slope, y = 0.f;
            if (a.s.softplus) w = softplus(w, slope);
            if (mine) {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float B = rec::to_f(((const IO*)a.Bm.p)[row * a.Bm.tok + g * a.Bm.head + n + i]);
                    const float C = rec::to_f(((const IO*)a.Cm.p)[row * a.Cm.tok + g * a.Cm.head + n + i]);
                    h[i] = fmaf(ex2_approx(w * A[i]), h[i], w * x * B);
                    y = fmaf(h[i], C, y);
                }
            }
            y = lanes_sum<LS>(y);
            if (q == 0 && u < D) {
                y = fmaf(skip, x, y);
                if (a.z.p) {
                    const float z = rec::to_f(((const IO*)a.z.p)[row * a.z.tok + d]);
                    y *= z * sigmoid(z);
                }
                ((IO*)a.y.p)[row * a.y.tok + d] = rec::from_f<IO>(y);
            }
        }
        if (mine && dst >= 0 && dst < a.s.slots) put4(a.state + ((long long)dst * D + d) * N + n, h);
    }
}

template <typename IO, int LS>
cudaError_t launch_step_lanes(const ScanStepArgs& a, cudaStream_t st)
{
    const long long lanes = (long long)a.s.D * LS;
    const dim3 grid((unsigned)((lanes + kStepThreads - 1) / kStepThreads), a.s.B < 65535 ? a.s.B : 65535);
    scan_step_kernel<IO, LS><<<grid, kStepThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename IO>
cudaError_t launch_step_typed(const ScanStepArgs& a, cudaStream_t st)
{
    if (a.s.N <= 8) return launch_step_lanes<IO, 2>(a, st);
    if (a.s.N <= 16) return launch_step_lanes<IO, 4>(a, st);
    return a.s.N <= 32 ? launch_step_lanes<IO, 8>(a, st) : launch_step_lanes<IO, 16>(a, st);
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, cudaStream_t st)
{
    return a.s.io == GDN_BF16 ? launch_typed<__nv_bfloat16>(a, st) : launch_typed<float>(a, st);
}
cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t st)
{
    return a.s.io == GDN_BF16 ? launch_step_typed<__nv_bfloat16>(a, st) : launch_step_typed<float>(a, st);
}

}  // namespace ssm
}  // namespace gdn
