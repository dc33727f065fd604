// ssm_scan_bwd.cu -- the gradients of the selective scan.
//
// With g = dy silu(z), dh[t] = g[t] C[t] + a[t+1] dh[t+1] and p = dh a h[t-1] (a = exp(delta A)):
//   d delta = sum_n p A + x sum_n dh B,   dx = delta sum_n dh B + g D,   dA = sum_t p delta,   dD = sum_t g x,
//   dB[t] = sum_d dh delta x,   dC[t] = sum_d g h,   dz = dy (sum_n h C + D x) silu'(z).
// Tiles of kSaveEvery tokens are walked from the last to the first: the forward left the state that enters each, so a
// tile's states are taken again into registers and then met by dh on its way back.
// Sums over channels (dB, dC): a lane's two channels first, then lanes by exchanges that halve them, then the CTA's warps, whose
// sum it writes; a second launch joins the CTAs in their order.  Sums over tokens (dA_log, dD, d dt_bias) are joined likewise over
// sequences and segments.  Instructions bound it (425 a token and 32 channels of 16 states, of which 110 are
// packed multiplications and additions that the formulas need and about 60 the sums over channels), at two warps a scheduler, which
// their registers allow: 696 us for 8 x 2048 tokens of 2048 channels, 20 for the join.  With eight states a lane the sums over channels have
// twice the values (840 us); eight states of two channels a lane do not fit the registers (1311).
// Segments of time: as forwards, with the adjoint's recurrence in place of the state's.
#include "ssm_scan_common.cuh"

namespace gdn {
namespace ssm {

namespace {

// A token's values v[0 .. 2 S - 1] (states of dB, then of dC), each summed over the CL lanes that hold the same states: each
// exchange halves what a lane still holds, and LEFT whole sums stay, those from number (lane % CL) 2 S / CL on.  Plain fp32 additions of
// one token's values alone: a NaN or an infinity reaches its own token's sums and no other's.  (Products with a matrix that is one
// in the token's column and zero elsewhere, as tf32 in two parts, made NaN of every token's sums and kept 22 bits; the gradients of
// 8 x 2048 tokens of 2048 channels took 737 us a call with them and 736 so, with 8 states 591 and 529, with 32 1435 and 1360.)
template <class L>
struct ChannelSums {
    static constexpr int V = 2 * L::S, LEFT = V > L::CL ? V / L::CL : 1;
    static_assert(LEFT == 1 || LEFT == 2 || LEFT == 4, "stored together");
    float x[LEFT];
    __device__ __forceinline__ void take(float (&v)[V], int lane)
    {
        int m = L::CL / 2;
#pragma unroll
        for (int k = V / 2; k && m; k >>= 1, m >>= 1)
#pragma unroll
            for (int i = 0; i < k; i++) {
                const bool up = lane & m;
                const float keep = up ? v[i + k] : v[i], send = up ? v[i] : v[i + k];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
            }
#pragma unroll
        for (; m; m >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
#pragma unroll
        for (int i = 0; i < LEFT; i++) x[i] = v[i];
    }
    // where they go in a token's row of 2 NS sums, n being the lane's first state
    static __device__ __forceinline__ int place(int lane, int n)
    {
        const int q = lane % L::CL * V / L::CL;
        return (q < L::S ? 0 : L::NS - L::S) + n + q;
    }
    __device__ __forceinline__ void put(float* to) const
    {
        if (LEFT == 4) *reinterpret_cast<float4*>(to) = make_float4(x[0], x[LEFT / 4], x[LEFT / 2], x[LEFT - 1]);
        else if (LEFT == 2) *reinterpret_cast<float2*>(to) = make_float2(x[0], x[LEFT - 1]);
        else *to = x[0];
    }
};

// A long sum and, beside it, the sum of what its additions lost (compensated summation), which joins it at the end: unless the
// sum is infinite by then, whose difference from itself would make it a NaN.
struct Sum {
    float v = 0.f, lost = 0.f;
    __device__ __forceinline__ void add(float x)
    {
        const float t = __fadd_rn(v, x);
        lost = __fadd_rn(lost, __fsub_rn(x, __fsub_rn(t, v)));
        v = t;
    }
    __device__ __forceinline__ float value() const { return fabsf(v) < INFINITY ? v + lost : v; }
};

// What a warp keeps in shared memory.
template <typename IO, class L>
struct BackStage {
    IO rows[2][4][kTile][L::CH];                    // x, dt, z, dy as they lie in memory: this tile's and the next one's
    IO vectors[2][2][kTile][L::NS];                 // B, C
    float4 h[2][L::RC * L::S / 4][32];              // the states that enter
    float B[kTile][L::NS], C[kTile][L::NS];
};
// And the CTA's shares of dB and dC: this tile's and the last one's, a warp's row of 2 NS sums for each token.
template <class L>
struct BackParts {
    float v[2][kBackWarps][kTile][2 * L::NS];
};

// F: how the forward's lanes had the states
template <typename IO, class L, class F, bool FIRST>
__global__ void __launch_bounds__(32 * kBackWarps) scan_bwd_kernel(const ScanArgs a)
{
    using P = BackParts<L>;
    constexpr int K = kTile, RC = L::RC, OT = L::OT, OWN = L::OWN, NS = L::NS, H = L::S / 2;
    // the states of M tokens are kept in registers at a time, with their factors where that is the whole tile
    constexpr int M = RC * L::S <= 8 ? K : K / 2;
    extern __shared__ __align__(16) unsigned char smem[];
    BackStage<IO, L>* stages = reinterpret_cast<BackStage<IO, L>*>(smem);
    P& parts = *reinterpret_cast<P*>(smem + kBackWarps * sizeof(BackStage<IO, L>));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = L::S * (lane / L::CL), oc = lane % L::CH, ot = lane / L::CH;
    BackStage<IO, L>& S = stages[warp];
    const Spot p = spot<L, kBackWarps>(a);
    const int D = a.s.D, N = a.s.N;
    cudaTriggerProgrammaticLaunchCompletion();
    if (p.share >= a.shares) {
        if (!FIRST) cudaGridDependencySynchronize();
        return;
    }
    if (FIRST && (p.channels == 0 || p.t0 >= p.t1 || p.t0 == 0)) return;
    States<L> A, back, dA;                          // back: the adjoint of the state that leaves the token
    float sum = 0.f;
    load_rates<L>(a, p, lane, A);
#pragma unroll
    for (int r = 0; r < RC; r++) {
#pragma unroll
        for (int k = 0; k < H; k++) back[r][k] = dA[r][k] = f2(0.f, 0.f);
        if (!FIRST && a.dhT && has_state<L>(a, p, lane, r)) get(a.dhT + state_at<L>(a, p, lane, r), back[r]);
    }
    if (!FIRST && p.t1 < p.r.n) {                   // the last segments do not wait for the first launch
        const int last = (p.r.n - 1) / a.seg_len;
        cudaGridDependencySynchronize();
        if (p.channels > 0) carry<L>(a, p, lane, last, -1, last - p.seg, A, back);
    }
    int saved[RC][L::S / 4];
    if (!FIRST)
#pragma unroll
        for (int r = 0; r < RC; r++)
#pragma unroll
            for (int i = 0; i < L::S / 4; i++) saved[r][i] = saved_place<F>(p.d0 - p.g * (D / a.s.G) + L::channel(lane, r), n + 4 * i);
    const bool in = p.has(oc), gated = a.z.p != nullptr;
    const float bias = in && a.dt_bias ? a.dt_bias[p.d0 + oc] : 0.f, skip = !FIRST && in && a.D_skip ? a.D_skip[p.d0 + oc] : 0.f;
    Sum dskip, dbias;

    // asks for a tile
    auto ask = [&](int t0, int buf) {
        ask_rows<L>(a.dt, p, t0, lane, S.rows[buf][1]);
        ask_rows<L>(a.dy, p, t0, lane, S.rows[buf][3]);
        if (gated) ask_rows<L>(a.z, p, t0, lane, S.rows[buf][2]);
        if (!FIRST) ask_rows<L>(a.x, p, t0, lane, S.rows[buf][0]);
        if (!FIRST) ask_vectors<L>(a.Bm, p, N, t0, lane, S.vectors[buf][0]);
        ask_vectors<L>(a.Cm, p, N, t0, lane, S.vectors[buf][1]);
        if (!FIRST && p.channels > 0) {
            const float4* h = reinterpret_cast<const float4*>(a.saved) + saved_at<F>(a, p, t0);
#pragma unroll
            for (int r = 0; r < RC; r++) {
                const bool ok = p.has(L::channel(lane, r));
#pragma unroll
                for (int i = 0; i < L::S / 4; i++) cp_async16_zero(&S.h[buf][r * (L::S / 4) + i][lane], h + (ok ? saved[r][i] : 0), ok);
            }
        }
        rec::cp_async_commit();
    };

    const int last = p.t1 > p.t0 ? p.t0 + (p.t1 - p.t0 - 1) / K * K : p.t0 - K;
    int buf = 0;
    if (!FIRST && p.channels == 0)                  // a warp without channels still takes part in the CTA's sums
#pragma unroll
        for (int i = 0; i < RC * L::S / 4; i++) S.h[0][i][lane] = S.h[1][i][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (last >= p.t0) ask(last, 0);
    for (int t0 = last; t0 >= p.t0; t0 -= K, buf ^= 1) {
        rec::cp_async_wait_all();
        __syncwarp();                               // every lane's pieces are there, and the last tile's have been read
        if (t0 > p.t0) ask(t0 - K, buf ^ 1);
        float w[OWN], ux[OWN], g[OWN], slope[OWN];
#pragma unroll
        for (int i = 0; i < OWN; i++) {
            const int j = i * OT + ot;
            w[i] = rec::to_f(S.rows[buf][1][j][oc]) + bias;
            g[i] = rec::to_f(S.rows[buf][3][j][oc]);
            slope[i] = 1.f;
        }
        if (gated)
#pragma unroll
            for (int i = 0; i < OWN; i++) {
                const float z = rec::to_f(S.rows[buf][2][i * OT + ot][oc]);
                g[i] *= z * sigmoid(z);
            }
        if (a.s.softplus)
#pragma unroll
            for (int i = 0; i < OWN; i++) w[i] = softplus(w[i], slope[i]);
        if (t0 + K > p.t1)
#pragma unroll
            for (int i = 0; i < OWN; i++)
                if (t0 + i * OT + ot >= p.t1) w[i] = 0.f;      // a step of size zero changes nothing
#pragma unroll
        for (int i = 0; i < OWN; i++) {
            ux[i] = FIRST ? 0.f : w[i] * rec::to_f(S.rows[buf][0][i * OT + ot][oc]);
            if (FIRST) sum += w[i];
        }
        widen<L>(S.vectors[buf][1], S.C, lane);
        if (!FIRST) widen<L>(S.vectors[buf][0], S.B, lane);
        __syncwarp();
        if (FIRST) {
#pragma unroll
            for (int j = K - 1; j >= 0; j--) {
                float2 C[H];
                get(&S.C[j][n], C);
#pragma unroll
                for (int r = 0; r < RC; r++) {
                    const float wr = from_owner<L>(w, j, r, lane), gr = from_owner<L>(g, j, r, lane);
#pragma unroll
                    for (int k = 0; k < H; k++)
                        back[r][k] = mul2(factor(f2(wr, wr), A[r][k]), fma2(f2(gr, gr), C[k], back[r][k]));
                }
            }
            continue;
        }
        States<L> tA;                               // this tile's share of the sums over tokens
        float tskip = 0.f, tbias = 0.f;
#pragma unroll
        for (int r = 0; r < RC; r++)
#pragma unroll
            for (int k = 0; k < H; k++) tA[r][k] = f2(0.f, 0.f);
#pragma unroll
        for (int m0 = K - M; m0 >= 0; m0 -= M) {
            // the states of M tokens again: those before them only to get there, their own kept
            float2 h[M + 1][RC][H], f[M == K ? M : 1][RC][H];
            get_state<L>(&S.h[buf][0][lane], h[0]);
#pragma unroll
            for (int jj = -m0; jj < M; jj++) {
                const int j = jj + m0;
                float2 B[H];
                get(&S.B[j][n], B);
#pragma unroll
                for (int r = 0; r < RC; r++) {
                    const float wr = from_owner<L>(w, j, r, lane), ur = from_owner<L>(ux, j, r, lane);
#pragma unroll
                    for (int k = 0; k < H; k++) {
                        const float2 e = factor(f2(wr, wr), A[r][k]);
                        if (M == K) f[jj][r][k] = e;
                        h[jj < 0 ? 0 : jj + 1][r][k] = fma2(e, h[jj < 0 ? 0 : jj][r][k], mul2(f2(ur, ur), B[k]));
                    }
                }
            }
            ChannelSums<L> sums[M];
#pragma unroll
            for (int i0 = M - OT; i0 >= 0; i0 -= OT) {
                float du[OT][RC], pa[OT][RC], yc[OT][RC];
#pragma unroll
                for (int t = OT - 1; t >= 0; t--) {
                    const int jj = i0 + t, j = jj + m0;
                    float2 B[H], C[H], vB[H], vC[H];
                    get(&S.B[j][n], B);
                    get(&S.C[j][n], C);
#pragma unroll
                    for (int r = 0; r < RC; r++) {
                        const float wr = from_owner<L>(w, j, r, lane), ur = from_owner<L>(ux, j, r, lane), gr = from_owner<L>(g, j, r, lane);
                        const float2 w2 = f2(wr, wr), u2 = f2(ur, ur), g2 = f2(gr, gr);
                        float2 sdu, spa, syc;
#pragma unroll
                        for (int k = 0; k < H; k++) {
                            const float2 dh = fma2(g2, C[k], back[r][k]);
                            back[r][k] = mul2(M == K ? f[M == K ? jj : 0][r][k] : factor(w2, A[r][k]), dh);
                            const float2 q = mul2(back[r][k], h[jj][r][k]);
                            tA[r][k] = fma2(q, w2, tA[r][k]);
                            sdu = k ? fma2(dh, B[k], sdu) : mul2(dh, B[k]);
                            spa = k ? fma2(q, A[r][k], spa) : mul2(q, A[r][k]);
                            syc = k ? fma2(h[jj + 1][r][k], C[k], syc) : mul2(h[jj + 1][r][k], C[k]);
                            vB[k] = r ? fma2(dh, u2, vB[k]) : mul2(dh, u2);
                            vC[k] = r ? fma2(h[jj + 1][r][k], g2, vC[k]) : mul2(h[jj + 1][r][k], g2);
                        }
                        du[t][r] = sdu.x + sdu.y;
                        pa[t][r] = spa.x + spa.y;
                        yc[t][r] = syc.x + syc.y;
                    }
                    float v[2 * L::S];
#pragma unroll
                    for (int k = 0; k < H; k++) {
                        v[2 * k] = vB[k].x;
                        v[2 * k + 1] = vB[k].y;
                        v[L::S + 2 * k] = vC[k].x;
                        v[L::S + 2 * k + 1] = vC[k].y;
                    }
                    sums[jj].take(v, lane);
                }
                const int j = i0 + ot + m0, i = (i0 + m0) / OT;
                const float sdu = to_owner<L>(du, lane), spa = to_owner<L>(pa, lane), syc = to_owner<L>(yc, lane);
                const bool ok = in && t0 + j < p.t1;
                const long long row = p.r.first + t0 + j;
                const float x = rec::to_f(S.rows[buf][0][j][oc]), z = rec::to_f(S.rows[buf][2][j][oc]), s = sigmoid(z);
                const float dz = rec::to_f(S.rows[buf][3][j][oc]) * fmaf(skip, x, syc) * s * fmaf(z, 1.f - s, 1.f);
                const float ddt = fmaf(sdu, x, spa * (1.f / kLog2e)) * slope[i];
                store_if(ok && gated, (IO*)a.dz.p + row * a.dz.tok + p.d0 + oc, dz);
                store_if(ok, (IO*)a.dx.p + row * a.dx.tok + p.d0 + oc, fmaf(sdu, w[i], g[i] * skip));
                store_if(ok, (IO*)a.ddt.p + row * a.ddt.tok + p.d0 + oc, ddt);
                tskip = fmaf(g[i], x, tskip);       // zeros past the end
                tbias += ok ? ddt : 0.f;
            }
            const int at = ChannelSums<L>::place(lane, n);
#pragma unroll
            for (int jj = 0; jj < M; jj++) sums[jj].put(&parts.v[buf][warp][m0 + jj][at]);
        }
#pragma unroll
        for (int r = 0; r < RC; r++)
#pragma unroll
            for (int k = 0; k < H; k++) dA[r][k] = add2(dA[r][k], tA[r][k]);      // tile by tile: long sums keep their accuracy
        dskip.add(tskip);
        dbias.add(tbias);
        __syncthreads();
        float* out = a.bcpart + ((long long)(blockIdx.x - p.g * a.ctas) * a.s.rows * a.s.G + p.g) * 2 * N;
#pragma unroll
        for (int u0 = 0; u0 < K * 2 * NS; u0 += 32 * kBackWarps) {
            const int u = u0 + threadIdx.x, j = u / (2 * NS), e = u % (2 * NS), m = e % NS;
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < kBackWarps; v++) s += parts.v[buf][v][j][e];
            if (u < K * 2 * NS && t0 + j < p.t1 && m < N) out[(long long)(p.r.first + t0 + j) * a.s.G * 2 * N + (e < NS ? 0 : N) + m] = s;
        }
    }
    if (FIRST) {
        put_state<L>(reinterpret_cast<float4*>(a.seg_h) + state_offset<L>(segment_at(a, p, p.seg), lane), back);
#pragma unroll
        for (int m = L::CH; m < 32; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        a.seg_d[segment_at(a, p, p.seg) * L::CH + oc] = sum;
        return;
    }
    float* share = a.wpart + (long long)p.share * D * (N + 2);
#pragma unroll
    for (int r = 0; r < RC; r++) {
        if (!has_state<L>(a, p, lane, r)) continue;
        if (a.dh0 && p.seg == 0) put(a.dh0 + state_at<L>(a, p, lane, r), back[r]);
        put(share + (long long)(p.d0 + L::channel(lane, r)) * N + n, dA[r]);
    }
    float wskip = dskip.value(), wbias = dbias.value();
#pragma unroll
    for (int m = L::CH; m < 32; m <<= 1) {
        wskip += __shfl_xor_sync(0xffffffffu, wskip, m);
        wbias += __shfl_xor_sync(0xffffffffu, wbias, m);
    }
    if (ot == 0 && in) {
        share[(long long)D * N + p.d0 + oc] = wskip;
        share[(long long)D * (N + 1) + p.d0 + oc] = wbias;
    }
    cudaGridDependencySynchronize();
}

// dB and dC of the sequences' rows: the shares of the group's blocks in their order
template <typename IO, bool SPARSE>
__global__ void __launch_bounds__(256) scan_join_kernel(const ScanArgs a)
{
    cudaGridDependencySynchronize();
    const int N = a.s.N, G = a.s.G, pieces = G * 2 * N / 8;
    const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
    int t = (int)(u / pieces), b = blockIdx.y;
    const int e = 8 * (int)(u - (long long)t * pieces), g = e / (2 * N), n = e - g * 2 * N;
    if (SPARSE) b = last_at_most(a.s.B, t, [&](int i) { return offset_of(a.cu, i, a.s.rows); });      // t: a row of any sequence
    const Rows r = rows_of(a.cu, b, a.s.T, a.s.rows);
    if (SPARSE) t -= r.first;
    if (t < 0 || t >= r.n) return;
    const long long row = r.first + t, stride = (long long)a.s.rows * G * 2 * N;
    const float* in = a.bcpart + row * G * 2 * N + e;
    float s[8] = {};
#pragma unroll 4
    for (int k = 0; k < a.ctas; k++) {
        float x[8];
        load8(in + k * stride, x);
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] += x[i];
    }
    if (n < N) store8((IO*)a.dBm.p + row * a.dBm.tok + g * a.dBm.head + n, s);
    else store8((IO*)a.dCm.p + row * a.dCm.tok + g * a.dCm.head + n - N, s);
}

template <typename IO, class L, class F>
cudaError_t launch_lanes(const ScanArgs& a, cudaStream_t st)
{
    constexpr size_t stages = kBackWarps * sizeof(BackStage<IO, L>), whole = stages + sizeof(BackParts<L>);
    const dim3 grid = scan_grid(a);
    cudaError_t e = cudaSuccess;
    if (whole > 48 * 1024) e = cudaFuncSetAttribute(scan_bwd_kernel<IO, L, F, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)whole);
    if (e == cudaSuccess && stages > 48 * 1024 && a.segments > 1)
        e = cudaFuncSetAttribute(scan_bwd_kernel<IO, L, F, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)stages);
    if (e != cudaSuccess) return e;
    if (a.segments > 1) scan_bwd_kernel<IO, L, F, true><<<grid, 32 * kBackWarps, stages, st>>>(a);
    else scan_bwd_kernel<IO, L, F, false><<<grid, 32 * kBackWarps, whole, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (a.segments > 1 && (e = launch_after(scan_bwd_kernel<IO, L, F, false>, grid, 32 * kBackWarps, whole, st, a)) != cudaSuccess) return e;
    const long long units = (long long)(a.sparse ? a.s.rows : a.s.T) * (a.s.G * 2 * a.s.N / 8);
    const dim3 join((unsigned)((units + 255) / 256), a.sparse ? 1 : a.s.B);
    if (units == 0) return cudaSuccess;
    return launch_after(a.sparse ? scan_join_kernel<IO, true> : scan_join_kernel<IO, false>, join, 256, 0, st, a);
}
template <typename IO>
cudaError_t launch_typed(const ScanArgs& a, cudaStream_t st)
{
    if (a.s.N <= 8) return launch_lanes<IO, Back8, Fwd8>(a, st);
    if (a.s.N <= 16) return launch_lanes<IO, Back16, Fwd16>(a, st);
    return a.s.N <= 32 ? launch_lanes<IO, Back32, Fwd32>(a, st) : launch_lanes<IO, Back64, Fwd64>(a, st);
}

}  // namespace

cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t st)
{
    const cudaError_t e = a.s.io == GDN_BF16 ? launch_typed<__nv_bfloat16>(a, st) : launch_typed<float>(a, st);
    if (e != cudaSuccess) return e;
    ColumnSums c = {};
    c.partial = a.wpart;
    c.rows = a.shares;
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
