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

// Sums over lanes by matrix products with ones.  The 32 lanes' values v0, v1 are a 16 x 4 matrix whose rows 0 .. 7 are v0 of
// lanes 4 r .. 4 r + 3 and whose rows 8 .. 15 are v1 of them; times a 4 x 8 matrix that is one in a column and zero elsewhere,
// that column of acc gets the rows' sums added.  A product reads 11 bits of a value (tf32), so a value goes in as two,
// its first 11 bits and those of the rest: 22 bits.
__device__ __forceinline__ void add_column(float (&acc)[4], float2 v, uint32_t ones)
{
    const uint32_t h0 = __float_as_uint(v.x) & 0xffffe000u, h1 = __float_as_uint(v.y) & 0xffffe000u;
    const uint32_t l0 = __float_as_uint(v.x - __uint_as_float(h0)) & 0xffffe000u;
    const uint32_t l1 = __float_as_uint(v.y - __uint_as_float(h1)) & 0xffffe000u;
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %8}, {%0, %1, %2, %3};"
                 : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
                 : "r"(h0), "r"(h1), "r"(l0), "r"(l1), "r"(ones));
}

// v[t][r]: a lane's share of a sum over the states, for token t of OT and place r.  Every lane gets the whole sum for the
// channel and the token that it owns.
template <class L>
__device__ __forceinline__ float to_owner(const float (&v)[L::OT][L::RC], int lane)
{
    float w[L::OT];
#pragma unroll
    for (int t = 0; t < L::OT; t++) {
        w[t] = v[t][0];
        if (L::RC == 2) w[t] += __shfl_xor_sync(0xffffffffu, v[t][L::RC - 1], L::CL);
    }
    int m = 16;
#pragma unroll
    for (int k = L::OT / 2; k; k >>= 1, m >>= 1)
#pragma unroll
        for (int i = 0; i < k; i++) {
            const float keep = lane & m ? w[i + k] : w[i], send = lane & m ? w[i] : w[i + k];
            w[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    return w[0];
}

// what the owner of token j has, at place r
template <class L>
__device__ __forceinline__ float from_owner(const float (&own)[kTile / L::OT], int j, int r, int lane)
{
    const float v = own[j / L::OT];
    if (L::OT == 1) return r ? __shfl_xor_sync(0xffffffffu, v, L::CL * r) : v;
    return __shfl_sync(0xffffffffu, v, (j % L::OT) * L::CH + L::channel(lane, r));
}

// What a warp keeps in shared memory.
template <typename IO, class L>
struct BackStage {
    IO rows[2][4][kTile][L::CH];                    // x, dt, z, dy as they lie in memory: this tile's and the next one's
    IO vectors[2][2][kTile][L::NS];                 // B, C
    float4 h[2][2 * L::RC][32];                     // the states that enter
    float B[kTile][L::NS], C[kTile][L::NS];
};
// And the CTA's shares of dB and dC: this tile's and the last one's.  A product's rows are lanes / 4: CS of them hold the same
// states and are added later.  A token's row of shares is PART values, planes lie PLANE apart, so that the lanes that write
// them meet in few banks (none for N <= 16).
template <class L>
struct BackParts {
    static constexpr int CS = L::CL / 4, PART = 2 * L::NS + (L::LS == 1 ? 8 : 2), PLANE = (kTile * PART + 31) / 32 * 32 + 1;
    float v[2][kBackWarps][CS * PLANE];
};

template <typename IO, int LS, bool FIRST>
__global__ void __launch_bounds__(32 * kBackWarps) scan_bwd_kernel(const ScanArgs a)
{
    using L = Lay<LS, LS == 8 ? 2 : 1>;
    using P = BackParts<L>;
    constexpr int K = kTile, HALF = K / 2, RC = L::RC, OT = L::OT, OWN = K / OT, NS = L::NS, CS = P::CS, PART = P::PART, PLANE = P::PLANE;
    extern __shared__ __align__(16) unsigned char smem[];
    BackStage<IO, L>* stages = reinterpret_cast<BackStage<IO, L>*>(smem);
    P& parts = *reinterpret_cast<P*>(smem + kBackWarps * sizeof(BackStage<IO, L>));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ng = lane / L::CL, oc = lane % L::CH, ot = lane / L::CH;
    BackStage<IO, L>& S = stages[warp];
    const Spot p = spot<L, kBackWarps>(a);
    const int D = a.s.D, N = a.s.N;
    if (FIRST && (p.channels == 0 || p.t0 >= p.t1)) return;
    float2 A[RC][4], back[RC][4], dA[RC][4];        // back: the adjoint of the state that leaves the token
    float sum = 0.f;
    load_rates<L>(a, p, lane, A);
    int saved[RC];                                  // where the states of place r lie in the forward's order
#pragma unroll
    for (int r = 0; r < RC; r++) {
        const int c = L::channel(lane, r), c0 = p.d0 - p.g * (D / a.s.G), c32 = c0 % 32 + c, from = ng * L::CL + c32 % L::CL;
        saved[r] = c0 / 32 * (LS * 64) + (ng ^ (c32 / L::CL)) * 64 + from;
#pragma unroll
        for (int k = 0; k < 4; k++) back[r][k] = dA[r][k] = f2(0.f, 0.f);
        if (!FIRST && a.dhT && p.has(c) && 8 * ng < N) get8(a.dhT + state_at<L>(a, p, lane, r), back[r]);
    }
    if (!FIRST)
        for (int s = a.segments - 1; s > p.seg; s--)
            if ((long long)s * a.seg_len < p.r.n && p.channels > 0) carry<L, kBackWarps>(a, p, lane, s, A, back);
    const bool in = p.has(oc), gated = a.z.p != nullptr;
    const float bias = in && a.dt_bias ? a.dt_bias[p.d0 + oc] : 0.f, skip = !FIRST && in && a.D_skip ? a.D_skip[p.d0 + oc] : 0.f;
    float dskip = 0.f, dbias = 0.f;

    // asks for a tile: zeros from the segment's end on, past the warp's channels and past N
    auto ask = [&](int t0, int buf) {
        constexpr int PER = L::CH * sizeof(IO) / 16, UNIT = 16 / sizeof(IO);
        auto rows = [&](const gdn_mla_view_t& v, IO (*to)[L::CH]) {
#pragma unroll
            for (int u0 = 0; u0 < K * PER; u0 += 32) {
                const int u = u0 + lane, j = u / PER, c = u % PER * UNIT;
                if (u < K * PER) {
                    const bool ok = t0 + j < p.t1 && c < p.channels;
                    cp_async16_zero(&to[j][c], (const IO*)v.p + (ok ? (long long)(p.r.first + t0 + j) * v.tok + p.d0 + c : 0), ok);
                }
            }
        };
        rows(a.dt, S.rows[buf][1]);
        rows(a.dy, S.rows[buf][3]);
        if (gated) rows(a.z, S.rows[buf][2]);
        if (!FIRST) rows(a.x, S.rows[buf][0]);
        auto vectors = [&](const gdn_mla_view_t& v, IO (*to)[NS]) {
            constexpr int PERV = NS * sizeof(IO) / 16;
#pragma unroll
            for (int u0 = 0; u0 < K * PERV; u0 += 32) {
                const int u = u0 + lane, j = u / PERV, n = u % PERV * UNIT;
                if (u < K * PERV) {
                    const bool ok = t0 + j < p.t1 && n < N;
                    cp_async16_zero(&to[j][n], (const IO*)v.p + (ok ? (long long)(p.r.first + t0 + j) * v.tok + p.g * v.head + n : 0), ok);
                }
            }
        };
        if (!FIRST) vectors(a.Bm, S.vectors[buf][0]);
        vectors(a.Cm, S.vectors[buf][1]);
        if (!FIRST) {
            const float4* h = reinterpret_cast<const float4*>(a.saved) + (saved_at(a, p, t0) + (long long)p.g * a.warps) * (LS * 64);
#pragma unroll
            for (int r = 0; r < RC; r++) {
                const bool ok = p.has(L::channel(lane, r));
#pragma unroll
                for (int i = 0; i < 2; i++) cp_async16_zero(&S.h[buf][2 * r + i][lane], h + (ok ? saved[r] + 32 * i : 0), ok);
            }
        }
        rec::cp_async_commit();
    };
    // one token forwards
    auto step = [&](int j, float wr, float ur, const float2 (&B)[4], const float2 (&from)[4], float2 (&to)[4], int r) {
#pragma unroll
        for (int k = 0; k < 4; k++) to[k] = fma2(ex2x2(mul2(f2(wr, wr), A[r][k])), from[k], mul2(f2(ur, ur), B[k]));
    };

    const int last = p.t1 > p.t0 ? p.t0 + (p.t1 - p.t0 - 1) / K * K : p.t0 - K;
    int buf = 0;
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
#pragma unroll
        for (int u0 = 0; u0 < K * LS; u0 += 32) {
            const int u = u0 + lane;
            if (u < K * LS) {
                float v[8];
                load8(&S.vectors[buf][1][0][0] + 8 * u, v);
                store8(&S.C[0][0] + 8 * u, v);
                if (!FIRST) {
                    load8(&S.vectors[buf][0][0][0] + 8 * u, v);
                    store8(&S.B[0][0] + 8 * u, v);
                }
            }
        }
        __syncwarp();
        if (FIRST) {
#pragma unroll
            for (int j = K - 1; j >= 0; j--) {
                float2 C[4];
                get8(&S.C[j][8 * ng], C);
#pragma unroll
                for (int r = 0; r < RC; r++) {
                    const float wr = from_owner<L>(w, j, r, lane), gr = from_owner<L>(g, j, r, lane);
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        back[r][k] = mul2(ex2x2(mul2(f2(wr, wr), A[r][k])), fma2(f2(gr, gr), C[k], back[r][k]));
                }
            }
            continue;
        }
        float2 tA[RC][4];
#pragma unroll
        for (int r = 0; r < RC; r++)
#pragma unroll
            for (int k = 0; k < 4; k++) tA[r][k] = f2(0.f, 0.f);
#pragma unroll
        for (int half = 1; half >= 0; half--) {
            // the states of half the tile again: those before it only to get there, its own kept
            float2 h[HALF + 1][RC][4];
#pragma unroll
            for (int r = 0; r < RC; r++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float4 v = S.h[buf][2 * r + i][lane];
                    h[0][r][2 * i] = f2(v.x, v.y);
                    h[0][r][2 * i + 1] = f2(v.z, v.w);
                }
#pragma unroll
            for (int jj = -HALF * half; jj < HALF; jj++) {
                const int j = jj + HALF * half;
                float2 B[4];
                get8(&S.B[j][8 * ng], B);
#pragma unroll
                for (int r = 0; r < RC; r++)
                    step(j, from_owner<L>(w, j, r, lane), from_owner<L>(ux, j, r, lane), B, h[jj < 0 ? 0 : jj][r], h[jj < 0 ? 0 : jj + 1][r], r);
            }
            float acc[4][4] = {};
#pragma unroll
            for (int i0 = HALF - OT; i0 >= 0; i0 -= OT) {
                float du[OT][RC], pa[OT][RC], yc[OT][RC];
#pragma unroll
                for (int t = OT - 1; t >= 0; t--) {
                    const int jj = i0 + t, j = jj + HALF * half;
                    float2 B[4], C[4], vB[4], vC[4];
                    get8(&S.B[j][8 * ng], B);
                    get8(&S.C[j][8 * ng], C);
#pragma unroll
                    for (int r = 0; r < RC; r++) {
                        const float wr = from_owner<L>(w, j, r, lane), ur = from_owner<L>(ux, j, r, lane), gr = from_owner<L>(g, j, r, lane);
                        const float2 w2 = f2(wr, wr), u2 = f2(ur, ur), g2 = f2(gr, gr);
                        float2 sdu, spa, syc;
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const float2 dh = fma2(g2, C[k], back[r][k]);
                            back[r][k] = mul2(ex2x2(mul2(w2, A[r][k])), dh);
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
                    const uint32_t first = lane >> 2 == jj ? 0x3f800000u : 0u, second = lane >> 2 == HALF + jj ? 0x3f800000u : 0u;
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        add_column(acc[k], vB[k], first);
                        add_column(acc[k], vC[k], second);
                    }
                }
                const int j = i0 + ot + HALF * half, i = (i0 + HALF * half) / OT;
                const float sdu = to_owner<L>(du, lane), spa = to_owner<L>(pa, lane), syc = to_owner<L>(yc, lane);
                const bool ok = in && t0 + j < p.t1;
                const long long row = p.r.first + t0 + j;
                const float x = rec::to_f(S.rows[buf][0][j][oc]), z = rec::to_f(S.rows[buf][2][j][oc]), s = sigmoid(z);
                const float dz = rec::to_f(S.rows[buf][3][j][oc]) * fmaf(skip, x, syc) * s * fmaf(z, 1.f - s, 1.f);
                const float ddt = fmaf(sdu, x, spa * (1.f / kLog2e)) * slope[i];
                store_if(ok && gated, (IO*)a.dz.p + row * a.dz.tok + p.d0 + oc, dz);
                store_if(ok, (IO*)a.dx.p + row * a.dx.tok + p.d0 + oc, fmaf(sdu, w[i], g[i] * skip));
                store_if(ok, (IO*)a.ddt.p + row * a.ddt.tok + p.d0 + oc, ddt);
                dskip = fmaf(g[i], x, dskip);       // zeros past the end
                dbias += ok ? ddt : 0.f;
            }
            // row r of a product is lanes 4 r .., columns 2 q and 2 q + 1 are lane q's: dB of two tokens, or dC
            const int r = lane >> 2, q = lane & 3;
            float* to = parts.v[buf][warp] + r % CS * PLANE + (HALF * half + 2 * (q & 1)) * PART + (q >> 1) * NS + 8 * (r / CS);
#pragma unroll
            for (int k = 0; k < 4; k++)
#pragma unroll
                for (int e = 0; e < 4; e++) to[(e & 1) * PART + 2 * k + (e >> 1)] = acc[k][e];
        }
#pragma unroll
        for (int r = 0; r < RC; r++)
#pragma unroll
            for (int k = 0; k < 4; k++) dA[r][k] = rec::add2(dA[r][k], tA[r][k]);      // tile by tile: long sums keep their accuracy
        __syncthreads();
        float* out = a.bcpart + ((long long)(blockIdx.x - p.g * a.ctas) * a.s.rows * a.s.G + p.g) * 2 * N;
#pragma unroll
        for (int u0 = 0; u0 < K * 2 * NS; u0 += 32 * kBackWarps) {
            const int u = u0 + threadIdx.x, j = u / (2 * NS), e = u % (2 * NS), n = e % NS;
            float s = 0.f;
#pragma unroll
            for (int v = 0; v < kBackWarps; v++)
#pragma unroll
                for (int c = 0; c < CS; c++) s += parts.v[buf][v][c * PLANE + j * PART + e];
            if (t0 + j < p.t1 && n < N) out[(long long)(p.r.first + t0 + j) * a.s.G * 2 * N + (e < NS ? 0 : N) + n] = s;
        }
    }
    if (FIRST) {
        put_state<L>(a.seg_h, segment_at<kBackWarps>(a, p, p.seg), lane, back);
#pragma unroll
        for (int m = L::CH; m < 32; m <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        a.seg_d[segment_at<kBackWarps>(a, p, p.seg) * L::CH + oc] = sum;
        return;
    }
    float* share = a.wpart + ((long long)p.seg * a.s.B + p.b) * D * (N + 2);
#pragma unroll
    for (int r = 0; r < RC; r++) {
        const int c = L::channel(lane, r);
        if (!p.has(c) || 8 * ng >= N) continue;
        if (a.dh0 && p.seg == 0) put8(a.dh0 + state_at<L>(a, p, lane, r), back[r]);
        put8(share + (long long)(p.d0 + c) * N + 8 * ng, dA[r]);
    }
#pragma unroll
    for (int m = L::CH; m < 32; m <<= 1) {
        dskip += __shfl_xor_sync(0xffffffffu, dskip, m);
        dbias += __shfl_xor_sync(0xffffffffu, dbias, m);
    }
    if (ot == 0 && in) {
        share[(long long)D * N + p.d0 + oc] = dskip;
        share[(long long)D * (N + 1) + p.d0 + oc] = dbias;
    }
}

// dB and dC of the sequences' rows: the shares of the group's blocks in their order
template <typename IO>
__global__ void __launch_bounds__(256) scan_join_kernel(const ScanArgs a)
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
    for (int k = 0; k < a.ctas; k++) {
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
    using L = Lay<LS, LS == 8 ? 2 : 1>;
    constexpr size_t stages = kBackWarps * sizeof(BackStage<IO, L>), whole = stages + sizeof(BackParts<L>);
    const dim3 grid(a.s.G * a.ctas, a.s.B, a.segments);
    if (whole > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<IO, LS, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)whole);
        if (e != cudaSuccess) return e;
    }
    if (a.segments > 1) scan_bwd_kernel<IO, LS, true><<<grid, 32 * kBackWarps, stages, st>>>(a);
    scan_bwd_kernel<IO, LS, false><<<grid, 32 * kBackWarps, whole, st>>>(a);
    const long long units = (long long)a.s.T * (a.s.G * 2 * a.s.N / 8);
    if (units > 0) scan_join_kernel<IO><<<dim3((unsigned)((units + 255) / 256), a.s.B), 256, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename IO>
cudaError_t launch_typed(const ScanArgs& a, cudaStream_t st)
{
    if (a.s.N <= 8) return launch_lanes<IO, 1>(a, st);
    if (a.s.N <= 16) return launch_lanes<IO, 2>(a, st);
    return a.s.N <= 32 ? launch_lanes<IO, 4>(a, st) : launch_lanes<IO, 8>(a, st);
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
