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

// FIRST: the first of the two launches
template <typename IO, int LS, bool FIRST>
__global__ void __launch_bounds__(32) scan_kernel(const ScanArgs a)
{
    using L = Lay<LS, LS>;
    __shared__ __align__(16) float sB[kTile][L::NS], sC[FIRST ? 1 : kTile][L::NS];
    const int lane = threadIdx.x, ng = lane / L::CL;
    const Spot p = spot<L, 1>(a);
    if (FIRST && p.t0 >= p.t1) return;
    float2 A[LS][4], h[LS][4];
    float sum = 0.f;
    load_rates<L>(a, p, lane, A);
#pragma unroll
    for (int r = 0; r < LS; r++) {
#pragma unroll
        for (int k = 0; k < 4; k++) h[r][k] = f2(0.f, 0.f);
        if (!FIRST && a.h0 && p.has(L::channel(lane, r)) && 8 * ng < a.s.N) get8(a.h0 + state_at<L>(a, p, lane, r), h[r]);
    }
    if (!FIRST)
        for (int s = 0; s < p.seg; s++) {
            if ((long long)s * a.seg_len >= p.r.n) break;
            carry<L, 1>(a, p, lane, s, A, h);
        }
    const bool in = p.has(lane), gated = a.z.p != nullptr;
    const float bias = in && a.dt_bias ? a.dt_bias[p.d0 + lane] : 0.f;
    const float skip = !FIRST && in && a.D_skip ? a.D_skip[p.d0 + lane] : 0.f;
    Column<IO> rx, rdt, rz;
    Vectors<L, IO> rB, rC;
    auto ask = [&](int t0) {
        rx.load(a.x, p, t0, lane);
        rdt.load(a.dt, p, t0, lane);
        rB.load(a.Bm, p, a.s.N, t0, lane);
        if (!FIRST) {
            rC.load(a.Cm, p, a.s.N, t0, lane);
            if (gated) rz.load(a.z, p, t0, lane);
        }
    };
    if (p.t0 < p.t1) ask(p.t0);
    for (int t0 = p.t0; t0 < p.t1; t0 += kTile) {
        float x[kTile], w[kTile], z[kTile], y[kTile], slope;
#pragma unroll
        for (int j = 0; j < kTile; j++) {
            x[j] = rec::to_f(rx.v[j]);
            if (!FIRST) z[j] = rec::to_f(rz.v[j]);
            w[j] = rec::to_f(rdt.v[j]) + bias;
        }
        if (a.s.softplus)
#pragma unroll
            for (int j = 0; j < kTile; j++) w[j] = softplus(w[j], slope);
        if (t0 + kTile > p.t1)
#pragma unroll
            for (int j = 0; j < kTile; j++)
                if (t0 + j >= p.t1) w[j] = 0.f;      // a step of size zero changes nothing
        __syncwarp();      // the last tile's vectors have been read
        rB.store(&sB[0][0], lane);
        if (!FIRST) rC.store(&sC[0][0], lane);
        __syncwarp();
        if (t0 + kTile < p.t1) ask(t0 + kTile);
        if (!FIRST && a.saved) put_state<L>(a.saved, saved_at(a, p, t0) + p.block, lane, h);
#pragma unroll
        for (int j = 0; j < kTile; j++) {
            float2 B[4], C[4];
            float part[LS];
            get8(&sB[j][8 * ng], B);
            if (!FIRST) get8(&sC[j][8 * ng], C);
            const float ux = w[j] * x[j];
#pragma unroll
            for (int r = 0; r < LS; r++) {
                const float wr = r ? __shfl_xor_sync(0xffffffffu, w[j], L::CL * r) : w[j];
                const float ur = r ? __shfl_xor_sync(0xffffffffu, ux, L::CL * r) : ux;
                float2 o = f2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    h[r][k] = fma2(ex2x2(mul2(f2(wr, wr), A[r][k])), h[r][k], mul2(f2(ur, ur), B[k]));
                    if (!FIRST) o = k ? fma2(h[r][k], C[k], o) : mul2(h[r][k], C[k]);
                }
                part[r] = o.x + o.y;
            }
            if (FIRST) {
                sum += w[j];
                continue;
            }
            y[j] = part[0];
#pragma unroll
            for (int r = 1; r < LS; r++) y[j] += __shfl_xor_sync(0xffffffffu, part[r], L::CL * r);
        }
        if (FIRST) continue;
#pragma unroll
        for (int j = 0; j < kTile; j++) y[j] = fmaf(skip, x[j], y[j]);
        if (gated)
#pragma unroll
            for (int j = 0; j < kTile; j++) y[j] *= z[j] * sigmoid(z[j]);
        IO* out = (IO*)a.y.p + (long long)(p.r.first + t0) * a.y.tok + p.d0 + lane;
#pragma unroll
        for (int j = 0; j < kTile; j++) store_if(in && t0 + j < p.t1, out + j * a.y.tok, y[j]);
    }
    if (FIRST) {
        put_state<L>(a.seg_h, segment_at<1>(a, p, p.seg), lane, h);
        a.seg_d[segment_at<1>(a, p, p.seg) * 32 + lane] = sum;
    } else if (a.hT && p.t1 == p.r.n && (p.t0 < p.t1 || p.seg == 0)) {
#pragma unroll
        for (int r = 0; r < LS; r++)
            if (p.has(L::channel(lane, r)) && 8 * ng < a.s.N) put8(a.hT + state_at<L>(a, p, lane, r), h[r]);
    }
}

template <typename IO, int LS>
cudaError_t launch_lanes(const ScanArgs& a, cudaStream_t st)
{
    const dim3 grid(a.s.G * a.ctas, a.s.B, a.segments);
    if (a.segments > 1) scan_kernel<IO, LS, true><<<grid, 32, 0, st>>>(a);
    scan_kernel<IO, LS, false><<<grid, 32, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename IO>
cudaError_t launch_typed(const ScanArgs& a, cudaStream_t st)
{
    if (a.s.N <= 8) return launch_lanes<IO, 1>(a, st);
    if (a.s.N <= 16) return launch_lanes<IO, 2>(a, st);
    return a.s.N <= 32 ? launch_lanes<IO, 4>(a, st) : launch_lanes<IO, 8>(a, st);
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
        { const float4 v = *reinterpret_cast<const float4*>(a.A_log + (long long)d * N + n); A[0] = v.x; A[1] = v.y; A[2] = v.z; A[3] = v.w; }
#pragma unroll
        for (int i = 0; i < 4; i++) A[i] = -expf(A[i]) * kLog2e;
    }
    for (int b = blockIdx.y; b < a.s.B; b += gridDim.y) {
        const int src = a.src ? a.src[b] : b, dst = a.dst ? a.dst[b] : src;
        float h[4] = {};
        if (mine && src >= 0 && src < a.s.slots) { const float4 v = *reinterpret_cast<const float4*>(a.state + ((long long)src * D + d) * N + n); h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w; }
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
            #pragma unroll
            for (int m = LS / 2; m; m >>= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
            if (q == 0 && u < D) {
                y = fmaf(skip, x, y);
                if (a.z.p) {
                    const float z = rec::to_f(((const IO*)a.z.p)[row * a.z.tok + d]);
                    y *= z * sigmoid(z);
                }
                ((IO*)a.y.p)[row * a.y.tok + d] = rec::from_f<IO>(y);
            }
        }
        if (mine && dst >= 0 && dst < a.s.slots) *reinterpret_cast<float4*>(a.state + ((long long)dst * D + d) * N + n) = make_float4(h[0], h[1], h[2], h[3]);
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
