// ssm_scan_bwd.cu -- the gradients of the selective scan.
//
// With g = dy silu(z), dh[t] = g[t] C[t] + a[t+1] dh[t+1] and p = dh a h[t-1] (a = exp(delta A)):
//   d delta = sum_n p A + x sum_n dh B,   dx = delta sum_n dh B + g D,   dA = sum_t p delta,   dD = sum_t g x,
//   dB[t] = sum_d dh delta x,   dC[t] = sum_d g h,   dz = dy (sum_n h C + D x) silu'(z).
// Chunks of kSaveEvery tokens are walked from the last to the first: the forward left the state that enters each, so a
// chunk's states are taken again into registers and then met by dh on its way back.
// Sums over channels (dB, dC) are added within a CTA, written by it, and joined over the CTAs in a fixed order; those
// over tokens (dA_log, dD, d dt_bias) likewise over sequences and segments.
// Segments of time: as forwards, with the adjoint's recurrence in place of the state's.
#include "ssm_scan_common.cuh"

namespace gdn {
namespace ssm {

namespace {

constexpr int K = kSaveEvery, kWarps = kScanThreads / 32;

// sum over the channels of a warp (lanes of equal q); every lane gets it
template <int LS>
__device__ __forceinline__ float channels_sum(float x)
{
#pragma unroll
    for (int m = LS; m < 32; m <<= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

template <typename IO, int LS, bool FIRST>
__global__ void __launch_bounds__(kScanThreads) scan_bwd_kernel(const ScanArgs a, int blocks)
{
    using L = Lay<LS>;
    constexpr int UNITS = K * L::PP, U = (UNITS + kScanThreads - 1) / kScanThreads;
    __shared__ float4 sd[K][L::CH];            // delta, delta x, g; then sum dh B, sum p A, sum h C
    __shared__ float sB[FIRST ? 1 : K][L::NS], sC[K][L::NS];
    __shared__ float bc[FIRST ? 1 : K][kWarps][2 * L::NS];     // a warp's shares of dB and dC
    const Spot p = spot<L>(a, blocks);
    const int D = a.s.D, N = a.s.N, cl = threadIdx.x / LS, q = threadIdx.x % LS, d = p.d0 + cl, warp = threadIdx.x >> 5;
    const bool mine = cl < p.channels && 4 * q < N;
    if (FIRST && p.t0 >= p.t1) return;
    const long long at = ((long long)p.b * D + d) * N + 4 * q, all = (long long)a.s.B * D;
    float A[4], back[4] = {}, dA[4] = {}, sum = 0.f;          // back: the adjoint of the state that leaves the token
    load_rates(a, d, 4 * q, mine, A);
    if (!FIRST && mine) {
        if (a.dhT) get4(a.dhT + at, back);
        for (int s = a.segments - 1; s > p.seg; s--) {
            if ((long long)s * a.seg_len >= p.r.n) continue;
            float e[4];
            const float w = a.seg_d[s * all + (long long)p.b * D + d];
            get4(a.seg_h + s * all * N + at, e);
#pragma unroll
            for (int i = 0; i < 4; i++) back[i] = fmaf(ex2_approx(w * A[i]), back[i], e[i]);
        }
    }
    float bias[U][8], skip[U][8], dskip[U][8] = {}, dbias[U][8] = {};
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
    const int last = p.t1 > p.t0 ? p.t0 + (p.t1 - p.t0 - 1) / K * K : p.t0 - K;
    for (int t0 = last; t0 >= p.t0; t0 -= K) {
        float x[U][8], dy[U][8], step[U][8], slope[U][8];
        __syncthreads();      // the last tile's results have left
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int unit = u * kScanThreads + threadIdx.x, j = unit / L::PP, c = 8 * (unit % L::PP);
            if (unit >= UNITS) continue;
            const bool in = t0 + j < p.t1 && c < p.channels;
            const long long row = p.r.first + t0 + j;
            float v[8], g[8];
#pragma unroll
            for (int i = 0; i < 8; i++) x[u][i] = dy[u][i] = v[i] = 0.f;
            if (in) {
                load8((const IO*)a.x.p + row * a.x.tok + p.d0 + c, x[u]);
                load8((const IO*)a.dt.p + row * a.dt.tok + p.d0 + c, v);
                load8((const IO*)a.dy.p + row * a.dy.tok + p.d0 + c, dy[u]);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) g[i] = dy[u][i];
            if (in && a.z.p) {
                float z[8];
                load8((const IO*)a.z.p + row * a.z.tok + p.d0 + c, z);
#pragma unroll
                for (int i = 0; i < 8; i++) g[i] *= z[i] * sigmoid(z[i]);
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
                float w = v[i] + bias[u][i];
                slope[u][i] = 1.f;
                if (a.s.softplus) w = softplus(w, slope[u][i]);
                if (!in) w = 0.f;
                step[u][i] = w;
                sd[j][c + i] = make_float4(w, w * x[u][i], g[i], 0.f);
            }
        }
        if (!FIRST) stage_vectors<L, IO, K>(a, a.Bm, p, t0, p.t1, sB);
        stage_vectors<L, IO, K>(a, a.Cm, p, t0, p.t1, sC);
        float h[K + 1][4] = {};      // h[j]: the state that token j finds
        if (!FIRST && mine) get4(a.saved + (saved_at(p, t0) * D + d) * N + 4 * q, h[0]);
        __syncthreads();
        if (!FIRST) {
#pragma unroll
            for (int j = 0; j < K; j++) {
                const float2 v = *reinterpret_cast<const float2*>(&sd[j][cl]);
                float B[4];
                get4(&sB[j][4 * q], B);
#pragma unroll
                for (int i = 0; i < 4; i++) h[j + 1][i] = fmaf(ex2_approx(v.x * A[i]), h[j][i], v.y * B[i]);
            }
        }
#pragma unroll
        for (int j = K - 1; j >= 0; j--) {
            const float4 v = sd[j][cl];
            float C[4];
            get4(&sC[j][4 * q], C);
            if (FIRST) {
                sum += v.x;
#pragma unroll
                for (int i = 0; i < 4; i++) back[i] = ex2_approx(v.x * A[i]) * fmaf(v.z, C[i], back[i]);
                continue;
            }
            float B[4], dB[4], dC[4], du = 0.f, pa = 0.f, yc = 0.f;
            get4(&sB[j][4 * q], B);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float dh = fmaf(v.z, C[i], back[i]);
                dB[i] = dh * v.y;
                dC[i] = v.z * h[j + 1][i];
                du = fmaf(dh, B[i], du);
                yc = fmaf(h[j + 1][i], C[i], yc);
                back[i] = ex2_approx(v.x * A[i]) * dh;
                const float t = back[i] * h[j][i];
                dA[i] = fmaf(t, v.x, dA[i]);
                pa = fmaf(t, A[i], pa);
            }
            du = lanes_sum<LS>(du);
            pa = lanes_sum<LS>(pa);
            yc = lanes_sum<LS>(yc);
            if (q == 0) sd[j][cl] = make_float4(du, pa * (1.f / kLog2e), yc, 0.f);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                dB[i] = channels_sum<LS>(dB[i]);
                dC[i] = channels_sum<LS>(dC[i]);
            }
            if ((threadIdx.x & 31) < LS) {
                put4(&bc[j][warp][4 * q], dB);
                put4(&bc[j][warp][L::NS + 4 * q], dC);
            }
        }
        if (FIRST) continue;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int unit = u * kScanThreads + threadIdx.x, j = unit / L::PP, c = 8 * (unit % L::PP);
            if (unit >= UNITS || t0 + j >= p.t1 || c >= p.channels) continue;
            const long long row = p.r.first + t0 + j;
            float z[8], dx[8], ddt[8], dz[8], g[8];
#pragma unroll
            for (int i = 0; i < 8; i++) g[i] = dy[u][i];
            if (a.z.p) load8((const IO*)a.z.p + row * a.z.tok + p.d0 + c, z);
#pragma unroll
            for (int i = 0; i < 8; i++) {
                const float4 r = sd[j][c + i];
                if (a.z.p) {
                    const float s = sigmoid(z[i]);
                    dz[i] = dy[u][i] * fmaf(skip[u][i], x[u][i], r.z) * s * fmaf(z[i], 1.f - s, 1.f);
                    g[i] *= z[i] * s;
                }
                dx[i] = fmaf(r.x, step[u][i], g[i] * skip[u][i]);
                ddt[i] = fmaf(r.x, x[u][i], r.y) * slope[u][i];
                dskip[u][i] = fmaf(g[i], x[u][i], dskip[u][i]);
                dbias[u][i] += ddt[i];
            }
            store8((IO*)a.dx.p + row * a.dx.tok + p.d0 + c, dx);
            store8((IO*)a.ddt.p + row * a.ddt.tok + p.d0 + c, ddt);
            if (a.z.p) store8((IO*)a.dz.p + row * a.dz.tok + p.d0 + c, dz);
        }
        // the CTA's share of the tokens' dB and dC
        float* out = a.bcpart + ((long long)(blockIdx.x - p.g * blocks) * a.s.rows * a.s.G + p.g) * 2 * N;
        for (int u = threadIdx.x; u < K * 2 * L::NS; u += kScanThreads) {
            const int j = u / (2 * L::NS), e = u % (2 * L::NS), n = e % L::NS;
            if (t0 + j >= p.t1 || n >= N) continue;
            float s = bc[j][0][e];
#pragma unroll
            for (int w = 1; w < kWarps; w++) s += bc[j][w][e];
            out[(long long)(p.r.first + t0 + j) * a.s.G * 2 * N + (e < L::NS ? 0 : N) + n] = s;
        }
    }
    if (FIRST) {
        if (mine) put4(a.seg_h + p.seg * all * N + at, back);
        if (mine && q == 0) a.seg_d[p.seg * all + (long long)p.b * D + d] = sum;
        return;
    }
    if (mine && a.dh0 && p.seg == 0) put4(a.dh0 + at, back);
    float* w = a.wpart + ((long long)p.seg * a.s.B + p.b) * D * (N + 2);
    if (mine) put4(w + (long long)d * N + 4 * q, dA);
    // dD and d dt_bias: threads of the same piece of channels, in their order
    float* share = &sd[0][0].x;      // [threads][16]
    static_assert(sizeof(sd) >= (UNITS < kScanThreads ? UNITS : kScanThreads) * 16 * sizeof(float), "room for the shares");
    __syncthreads();
    if (threadIdx.x < UNITS) {
#pragma unroll
        for (int u = 1; u < U; u++)
#pragma unroll
            for (int i = 0; i < 8; i++) {
                dskip[0][i] += dskip[u][i];
                dbias[0][i] += dbias[u][i];
            }
        store8(share + threadIdx.x * 16, dskip[0]);
        store8(share + threadIdx.x * 16 + 8, dbias[0]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * L::CH; e += kScanThreads) {
        const int c = e % L::CH, which = e / L::CH;
        if (c >= p.channels) continue;
        float s = 0.f;
        for (int k = c / 8; k < (UNITS < kScanThreads ? UNITS : kScanThreads); k += L::PP) s += share[k * 16 + 8 * which + c % 8];
        w[(long long)D * (N + which) + p.d0 + c] = s;
    }
}

// dB and dC of the sequences' rows: the shares of the group's blocks in their order
template <typename IO>
__global__ void __launch_bounds__(256) scan_join_kernel(const ScanArgs a, int blocks)
{
    const int N = a.s.N, G = a.s.G, pieces = G * 2 * N / 8;
    const Rows r = rows_of(a.cu, blockIdx.y, a.s.T, a.s.rows);
    const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
    const int t = (int)(u / pieces), e = 8 * (int)(u - (long long)t * pieces), g = e / (2 * N), n = e - g * 2 * N;
    if (t >= r.n) return;
    const long long row = r.first + t, stride = (long long)a.s.rows * G * 2 * N;
    const float* in = a.bcpart + row * G * 2 * N + e;
    float s[8] = {};
#pragma unroll 4
    for (int k = 0; k < blocks; k++) {
        float x[8];
        load8(in + k * stride, x);
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] += x[i];
    }
    if (n < N) store8((IO*)a.dBm.p + row * a.dBm.tok + g * a.dBm.head + n, s);
    else store8((IO*)a.dCm.p + row * a.dCm.tok + g * a.dCm.head + n - N, s);
}

template <typename IO, int LS>
cudaError_t launch_lanes(const ScanArgs& a, cudaStream_t st)
{
    const ScanPlan plan = scan_plan(a.s, 1);
    const dim3 grid(a.s.G * plan.blocks, a.s.B, a.segments);
    if (a.segments > 1) scan_bwd_kernel<IO, LS, true><<<grid, kScanThreads, 0, st>>>(a, plan.blocks);
    scan_bwd_kernel<IO, LS, false><<<grid, kScanThreads, 0, st>>>(a, plan.blocks);
    const long long units = (long long)a.s.T * (a.s.G * 2 * a.s.N / 8);
    if (units > 0) scan_join_kernel<IO><<<dim3((unsigned)((units + 255) / 256), a.s.B), 256, 0, st>>>(a, plan.blocks);
    return cudaGetLastError();
}
template <typename IO>
cudaError_t launch_typed(const ScanArgs& a, cudaStream_t st)
{
    if (a.s.N <= 8) return launch_lanes<IO, 2>(a, st);
    if (a.s.N <= 16) return launch_lanes<IO, 4>(a, st);
    return a.s.N <= 32 ? launch_lanes<IO, 8>(a, st) : launch_lanes<IO, 16>(a, st);
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t st)
{
    const cudaError_t e = a.s.io == GDN_BF16 ? launch_typed<__nv_bfloat16>(a, st) : launch_typed<float>(a, st);
    if (e != cudaSuccess) return e;
    ColumnSums c = {};
    c.partial = a.wpart;
    c.rows = a.s.B * a.segments;
    c.cols = (long long)a.s.D * (a.s.N + 2);
    c.a = (long long)a.s.D * a.s.N;
    c.b = a.s.D;
    c.out_a = a.dA_log;
    c.out_b = a.dD_skip;
    c.out_c = a.ddt_bias;
    c.decay = a.A_log;
    return launch_column_sums(c, st);
}

}  // namespace ssm
}  // namespace gdn
