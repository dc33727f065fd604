// ssm_scan_fwd.cu -- the selective scan forwards, and its form for new tokens.
//
// h[t] = exp(delta[t] A) h[t-1] + delta[t] x[t] B[t], y[t] = (h[t] . C[t] + D x[t]) silu(z[t]).  Tiles of kTile tokens: what goes
// by channel alone is worked out by the channel's owner, exchanged between lanes before the tile's recurrence, and the
// outputs' shares after it, so that one token's arithmetic can run among another's; the next tile is asked for meanwhile.
// Instructions bound it (about 131 a token and 32 channels of 16 states, 16 of them exponentials; the schedulers that have warps
// issue 0.65 to 0.70 a cycle, and a packed one of them takes two), not the special units (40 to 60 %) or DRAM (15 to 40 %).
// Where sequences are few, segments of time run side by side: a first launch takes each segment's states from zero and
// the sum of its step sizes; since a segment turns the state h it gets into exp(A sum delta) h + (its state from zero), each
// segment of the second launch finds its own entering state from those of the segments before it.  8 x 2048 tokens of 2048
// channels: 100 + 169 us split, 301 whole; 16001 tokens of 1536: 205 us a call, 2207 whole; nine prompts up to 1500: 135 and 213.
// The second launch begins while the first one ends: its warps get their rates, and those of first segments all their work, done
// (prompts 145 us without).
#include "ssm_scan_common.cuh"

namespace gdn {
namespace ssm {

namespace {

// FIRST: the first of the two launches
template <typename IO, class L, bool FIRST>
__global__ void __launch_bounds__(32, 16) scan_kernel(const ScanArgs a)
{
    constexpr int OT = L::OT, OWN = L::OWN, RC = L::RC, H = L::S / 2;
    __shared__ __align__(16) float sB[kTile][L::NS], sC[FIRST ? 1 : kTile][L::NS];
    __shared__ __align__(16) IO rows[2][FIRST ? 2 : 3][kTile][L::CH], vectors[2][FIRST ? 1 : 2][kTile][L::NS];      // x, dt, z; B, C
    const int lane = threadIdx.x, n = L::S * (lane / L::CL), oc = lane % L::CH, ot = lane / L::CH;
    const Spot p = spot<L, 1>(a);
    if (FIRST) cudaTriggerProgrammaticLaunchCompletion();
    if (FIRST && (p.t0 >= p.t1 || p.t1 == p.r.n)) return;      // what a sequence's last segment hands on nobody takes
    if (!FIRST && p.seg > 0 && p.t0 >= p.t1) {
        cudaGridDependencySynchronize();
        return;
    }
    States<L> A, h;
    float sum = 0.f;
    load_rates<L>(a, p, lane, A);
#pragma unroll
    for (int r = 0; r < RC; r++) {
#pragma unroll
        for (int k = 0; k < H; k++) h[r][k] = f2(0.f, 0.f);
        if (!FIRST && a.h0 && has_state<L>(a, p, lane, r)) get(a.h0 + state_at<L>(a, p, lane, r), h[r]);
    }
    if (!FIRST && p.seg > 0) {
        cudaGridDependencySynchronize();      // the first segments do not wait for the first launch
        carry<L>(a, p, lane, 0, 1, p.seg, A, h);
    }
    const bool in = p.has(oc), gated = a.z.p != nullptr;
    const float bias = in && a.dt_bias ? a.dt_bias[p.d0 + oc] : 0.f;
    const float skip = !FIRST && in && a.D_skip ? a.D_skip[p.d0 + oc] : 0.f;
    auto ask = [&](int t0, int buf) {
        ask_rows<L>(a.x, p, t0, lane, rows[buf][0]);
        ask_rows<L>(a.dt, p, t0, lane, rows[buf][1]);
        ask_vectors<L>(a.Bm, p, a.s.N, t0, lane, vectors[buf][0]);
        if (!FIRST) {
            if (gated) ask_rows<L>(a.z, p, t0, lane, rows[buf][FIRST ? 0 : 2]);
            ask_vectors<L>(a.Cm, p, a.s.N, t0, lane, vectors[buf][FIRST ? 0 : 1]);
        }
        rec::cp_async_commit();
    };
    if (p.t0 < p.t1) ask(p.t0, 0);
    int buf = 0;
    for (int t0 = p.t0; t0 < p.t1; t0 += kTile, buf ^= 1) {
        rec::cp_async_wait_all();
        __syncwarp();      // every lane's pieces are there, and the last tile's have been read
        if (t0 + kTile < p.t1) ask(t0 + kTile, buf ^ 1);
        float x[OWN], w[OWN], ux[OWN], y[OWN], slope;
#pragma unroll
        for (int i = 0; i < OWN; i++) {
            x[i] = rec::to_f(rows[buf][0][i * OT + ot][oc]);
            w[i] = rec::to_f(rows[buf][1][i * OT + ot][oc]) + bias;
        }
        if (a.s.softplus)
#pragma unroll
            for (int i = 0; i < OWN; i++) w[i] = softplus(w[i], slope);
        if (t0 + kTile > p.t1)
#pragma unroll
            for (int i = 0; i < OWN; i++)
                if (t0 + i * OT + ot >= p.t1) w[i] = 0.f;      // a step of size zero changes nothing
#pragma unroll
        for (int i = 0; i < OWN; i++) {
            ux[i] = w[i] * x[i];
            if (FIRST) sum += w[i];
        }
        widen<L>(vectors[buf][0], sB, lane);
        if (!FIRST) widen<L>(vectors[buf][FIRST ? 0 : 1], sC, lane);
        __syncwarp();
        if (!FIRST && a.saved) put_state<L>(reinterpret_cast<float4*>(a.saved) + saved_at<L>(a, p, t0) + state_offset<L>(p.block - p.g * a.blocks, lane), h);
        // exchanges between lanes before and after, so that nothing keeps one token's arithmetic from another's
        float wr[kTile][RC], ur[kTile][RC], part[OWN][OT][RC];
#pragma unroll
        for (int j = 0; j < kTile; j++)
#pragma unroll
            for (int r = 0; r < RC; r++) {
                wr[j][r] = from_owner<L>(w, j, r, lane);
                ur[j][r] = from_owner<L>(ux, j, r, lane);
            }
#pragma unroll
        for (int j = 0; j < kTile; j++) {
            float2 B[H], C[H];
            get(&sB[j][n], B);
            if (!FIRST) get(&sC[j][n], C);
#pragma unroll
            for (int r = 0; r < RC; r++) {
                float2 o = f2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < H; k++) {
                    h[r][k] = fma2(factor(f2(wr[j][r], wr[j][r]), A[r][k]), h[r][k], mul2(f2(ur[j][r], ur[j][r]), B[k]));
                    if (!FIRST) o = k ? fma2(h[r][k], C[k], o) : mul2(h[r][k], C[k]);
                }
                part[j / OT][j % OT][r] = o.x + o.y;
            }
        }
        if (!FIRST)
#pragma unroll
            for (int i = 0; i < OWN; i++) y[i] = to_owner<L>(part[i], lane);
        if (FIRST) continue;
#pragma unroll
        for (int i = 0; i < OWN; i++) y[i] = fmaf(skip, x[i], y[i]);
        if (gated)
#pragma unroll
            for (int i = 0; i < OWN; i++) {
                const float z = rec::to_f(rows[buf][FIRST ? 0 : 2][i * OT + ot][oc]);
                y[i] *= z * sigmoid(z);
            }
        IO* out = (IO*)a.y.p + (long long)(p.r.first + t0 + ot) * a.y.tok + p.d0 + oc;
#pragma unroll
        for (int i = 0; i < OWN; i++) store_if(in && t0 + i * OT + ot < p.t1, out + i * OT * a.y.tok, y[i]);
    }
    if (FIRST) {
        put_state<L>(reinterpret_cast<float4*>(a.seg_h) + state_offset<L>(segment_at(a, p, p.seg), lane), h);
#pragma unroll
        for (int m = L::CH; m < 32; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        a.seg_d[segment_at(a, p, p.seg) * L::CH + oc] = sum;
    } else if (a.hT && p.t1 == p.r.n && (p.t0 < p.t1 || p.seg == 0)) {
#pragma unroll
        for (int r = 0; r < RC; r++)
            if (has_state<L>(a, p, lane, r)) put(a.hT + state_at<L>(a, p, lane, r), h[r]);
    }
    if (!FIRST) cudaGridDependencySynchronize();
}

template <typename IO, class L>
cudaError_t launch_lanes(const ScanArgs& a, cudaStream_t st)
{
    const dim3 grid = scan_grid(a);
    if (a.segments > 1) scan_kernel<IO, L, true><<<grid, 32, 0, st>>>(a);
    else scan_kernel<IO, L, false><<<grid, 32, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess && a.segments > 1 ? launch_after(scan_kernel<IO, L, false>, grid, 32, 0, st, a) : e;
}
template <typename IO>
cudaError_t launch_typed(const ScanArgs& a, cudaStream_t st)
{
    if (a.s.N <= 8) return launch_lanes<IO, Fwd8>(a, st);
    if (a.s.N <= 16) return launch_lanes<IO, Fwd16>(a, st);
    return a.s.N <= 32 ? launch_lanes<IO, Fwd32>(a, st) : launch_lanes<IO, Fwd64>(a, st);
}

// New tokens.  LS = 1, 2, 4 or 8 lanes, CL = 32 / LS apart, hold a channel's states, 8 each, and take E <= LS sequences at a
// time, each of them owned by some of the lanes, which work out its step size and store its result.  The states' bytes bound
// it where sequences are many, next to the instructions around them: so few lanes a channel, and A taken once for all the
// sequences of a warp.  ONE: a single token each.  512 sequences of 2048 channels: 29 us (143 MB, a cold cache); with four states a
// lane, whose B, C and addresses serve half as many, 39 us, with a lane's every value worked out by itself 57.
constexpr int kStepThreads = 128;
template <typename IO, int LS, bool ONE>
__global__ void __launch_bounds__(kStepThreads, LS <= 2 ? 7 : 4) scan_step_kernel(const ScanStepArgs a)
{
    constexpr int CL = 32 / LS, E = LS < 4 ? LS : 4, REP = LS / E;
    const int N = a.s.N, D = a.s.D, T = ONE ? 1 : a.s.T, lane = threadIdx.x & 31, ng = lane / CL, own = ng / REP, n = 8 * ng;
    const int u = (blockIdx.x * (kStepThreads / 32) + (threadIdx.x >> 5)) * CL + lane % CL, d = min(u, D - 1), g = d / (D / a.s.G);
    const bool mine = u < D && n < N;
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.f, skip = a.D_skip ? a.D_skip[d] : 0.f;
    float2 A[4];
#pragma unroll
    for (int k = 0; k < 4; k++) A[k] = f2(0.f, 0.f);
    if (mine) {
        get(a.A_log + (long long)d * N + n, A);
#pragma unroll
        for (int k = 0; k < 4; k++) A[k] = rates(A[k]);
    }
    // from one sequence's rows to the next one's
    const long long dB = T * a.Bm.tok, dC = T * a.Cm.tok;
    float* state = a.state + (long long)d * N + n;
    const long long slot = (long long)D * N;
    for (int b0 = blockIdx.y * E; b0 < a.s.B; b0 += gridDim.y * E) {
        float2 h[E][4];
        int to[E];      // slots that are written
#pragma unroll
        for (int e = 0; e < E; e++) {
            int s = -1;
            if (b0 + e < a.s.B) s = a.src ? a.src[b0 + e] : b0 + e;
            to[e] = s;
            if (a.dst && b0 + e < a.s.B) to[e] = a.dst[b0 + e];
#pragma unroll
            for (int k = 0; k < 4; k++) h[e][k] = f2(0.f, 0.f);
            if (mine && (unsigned)s < (unsigned)a.s.slots) get(state + s * slot, h[e]);
        }
        const bool live = b0 + own < a.s.B;
        const int left = a.s.B - b0;
        const long long row = (long long)(live ? b0 + own : b0) * T;
        const IO* pB = (const IO*)a.Bm.p + (long long)b0 * dB + g * a.Bm.head + n;
        const IO* pC = (const IO*)a.Cm.p + (long long)b0 * dC + g * a.Cm.head + n;
#pragma unroll 1
        for (int t = 0; t < T; t++) {
            const float x = rec::to_f(((const IO*)a.x.p)[(row + t) * a.x.tok + d]);
            const float z = a.z.p ? rec::to_f(((const IO*)a.z.p)[(row + t) * a.z.tok + d]) : 0.f;
            float w = rec::to_f(((const IO*)a.dt.p)[(row + t) * a.dt.tok + d]) + bias, slope, y[E];
            Raw8<IO> B[E], C[E];
#pragma unroll
            for (int e = 0; e < E; e++) {
                B[e] = C[e] = Raw8<IO>{};
                if (mine && e < left) {
                    B[e] = raw8(pB + e * dB + t * a.Bm.tok);
                    C[e] = raw8(pC + e * dC + t * a.Cm.tok);
                }
            }
            if (a.s.softplus) w = softplus(w, slope);
            const float ux = w * x;
#pragma unroll
            for (int e = 0; e < E; e++) {
                const int from = lane % CL + CL * REP * e;
                const float we = LS == 1 ? w : __shfl_sync(0xffffffffu, w, from), ue = LS == 1 ? ux : __shfl_sync(0xffffffffu, ux, from);
                float b[8], c[8];
                values(B[e], b);
                values(C[e], c);
                float2 o = f2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    h[e][k] = fma2(factor(f2(we, we), A[k]), h[e][k], mul2(f2(ue, ue), f2(b[2 * k], b[2 * k + 1])));
                    o = fma2(h[e][k], f2(c[2 * k], c[2 * k + 1]), o);
                }
                y[e] = o.x + o.y;
            }
            const float v = fmaf(skip, x, states_sum<LS, E>(y, lane));
            store_if(live && u < D && ng % REP == 0, (IO*)a.y.p + (row + t) * a.y.tok + d, a.z.p ? v * z * sigmoid(z) : v);
        }
#pragma unroll
        for (int e = 0; e < E; e++)
            if (mine && (unsigned)to[e] < (unsigned)a.s.slots) put(state + to[e] * slot, h[e]);
    }
}

template <typename IO, int LS>
cudaError_t launch_step_lanes(const ScanStepArgs& a, cudaStream_t st)
{
    constexpr int CL = 32 / LS, E = LS < 4 ? LS : 4;
    const int wide = (a.s.D + 4 * CL - 1) / (4 * CL), groups = (a.s.B + E - 1) / E;
    const int fit = 152 * 40 / wide, turns = fit < 1 ? groups : (groups + fit - 1) / fit;
    const dim3 grid(wide, (groups + turns - 1) / turns);
    if (a.s.T == 1) scan_step_kernel<IO, LS, true><<<grid, kStepThreads, 0, st>>>(a);
    else scan_step_kernel<IO, LS, false><<<grid, kStepThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename IO>
cudaError_t launch_step_typed(const ScanStepArgs& a, cudaStream_t st)
{
    if (a.s.N <= 8) return launch_step_lanes<IO, 1>(a, st);
    if (a.s.N <= 16) return launch_step_lanes<IO, 2>(a, st);
    return a.s.N <= 32 ? launch_step_lanes<IO, 4>(a, st) : launch_step_lanes<IO, 8>(a, st);
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
