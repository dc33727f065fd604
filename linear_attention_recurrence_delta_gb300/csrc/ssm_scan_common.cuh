// ssm_scan_common.cuh -- what the forward and the backward scan share: how a warp is laid out, and how tokens are staged.
//
// A warp takes CH neighbouring channels of one group of one sequence (or a segment of it).  LS lanes, CL = 32 / LS apart, hold
// the same RC channels (CH = RC CL), each lane S states of every one (S LS >= N; those past N stay zero).  So a write or
// read vector is fetched from shared memory S values a lane for RC channels' use, which matters: 16 bytes a lane from
// shared memory take as long as four instructions of every scheduler, broadcast or not.
// What goes by channel alone (rows of x, step sizes, gates, results) has an owner: lane l owns channel l % CH at the tokens
// whose number is l / CH modulo OT = 32 / CH.  Place r of a lane's arrays is the channel that differs from its own by r CL,
// its own for r = 0.
#pragma once

#include <float.h>

#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

constexpr int kTile = kSaveEvery;      // tokens that are loaded together

template <int S_, int LS_, int RC_>
struct Lay {
    static constexpr int S = S_, LS = LS_, RC = RC_, NS = S * LS, CL = 32 / LS, CH = RC * CL, OT = 32 / CH, OWN = kTile / OT;
    // the channel of place r, within the warp's
    static __device__ __forceinline__ int channel(int lane, int r) { return (lane % CH) ^ (CL * r); }
};
// by N up to 8, 16, 32 and 64.  Forwards few instructions a token count; backwards the channels that a lane adds up by itself
using Fwd8 = Lay<8, 1, 1>;
using Fwd16 = Lay<8, 2, 2>;
using Fwd32 = Lay<8, 4, 2>;
using Fwd64 = Lay<8, 8, 2>;
using Back8 = Lay<4, 2, 2>;
using Back16 = Lay<4, 4, 2>;
using Back32 = Lay<4, 8, 2>;
using Back64 = Lay<8, 8, 2>;
template <class L>
using States = float2[L::RC][L::S / 2];

// where a warp works
struct Spot {
    int g, b, seg;        // group, sequence, segment
    int share;            // of the shares of sums over tokens (and may lie past them: nothing to do)
    int block;            // its number among all warps' blocks of channels
    int d0, channels;     // its first channel, how many it has (0: none)
    Rows r;               // the sequence's rows
    int t0, t1;           // tokens of the segment
    __device__ __forceinline__ bool has(int channel) const { return channel < channels; }
};
// W warps a CTA, a.ctas CTAs and a.blocks blocks of CH channels a group; the grid is segments of sequences, or their places
inline dim3 scan_grid(const ScanArgs& a)
{
    const int n = places(a.s.B, a.s.rows, a.seg_len), z = (n + 65534) / 65535;
    return a.sparse ? dim3(a.s.G * a.ctas, (n + z - 1) / z, z) : dim3(a.s.G * a.ctas, a.s.B, a.segments);
}
template <class L, int W>
__device__ __forceinline__ Spot spot(const ScanArgs& a)
{
    Spot p;
    p.g = blockIdx.x / a.ctas;
    p.b = blockIdx.y;
    p.seg = blockIdx.z;
    p.share = blockIdx.z * gridDim.y + blockIdx.y;
    if (a.sparse) {
        const Place at = place_of(a.cu, a.s.B, a.s.rows, a.seg_len, p.share);
        p.b = at.b;
        p.seg = at.piece;
    }
    const int each = a.s.D / a.s.G, n = (blockIdx.x - p.g * a.ctas) * W + (threadIdx.x >> 5), c0 = min(each, n * L::CH);
    p.block = p.g * a.blocks + n;
    p.d0 = p.g * each + c0;
    p.channels = min(L::CH, each - c0);
    p.r = rows_of(a.cu, p.b, a.s.T, a.s.rows);
    p.t0 = (int)min((long long)p.r.n, (long long)p.seg * a.seg_len);
    p.t1 = (int)min((long long)p.r.n, (long long)p.t0 + a.seg_len);
    return p;
}

__device__ __forceinline__ float2 ex2x2(float2 x) { return f2(ex2_approx(x.x), ex2_approx(x.y)); }
// exp(delta A) of two states: 2^(w A2).  ex2.approx's results are 2.1e-8 low on average for exponents between -0.3 and -0.003
// (measured; their other error, 3.7e-8, has no sign).  A state that forgets over a thousand tokens would add that up a thousand
// times, so the exponent is raised by as much; 2^(that alone) is 1, and a step of size zero still changes nothing.
constexpr float kLow = 3e-8f;
__device__ __forceinline__ float2 factor(float2 w, float2 A2) { return ex2x2(fma2(w, A2, f2(kLow, kLow))); }

template <int H>
__device__ __forceinline__ void get(const float* p, float2 (&x)[H])
{
#pragma unroll
    for (int i = 0; i < H / 2; i++) {
        const float4 v = reinterpret_cast<const float4*>(p)[i];
        x[2 * i] = f2(v.x, v.y);
        x[2 * i + 1] = f2(v.z, v.w);
    }
}
template <int H>
__device__ __forceinline__ void put(float* p, const float2 (&x)[H])
{
#pragma unroll
    for (int i = 0; i < H / 2; i++) reinterpret_cast<float4*>(p)[i] = make_float4(x[2 * i].x, x[2 * i].y, x[2 * i + 1].x, x[2 * i + 1].y);
}

// Without a branch, which would keep the compiler from moving instructions of one token among another's.
__device__ __forceinline__ void store_if(bool ok, float* p, float x)
{
    asm volatile("{ .reg .pred q; setp.ne.b32 q, %2, 0; @q st.global.f32 [%0], %1; }" ::"l"(p), "f"(x), "r"((int)ok) : "memory");
}
__device__ __forceinline__ void store_if(bool ok, __nv_bfloat16* p, float x)
{
    const __nv_bfloat16 v = __float2bfloat16_rn(x);
    asm volatile("{ .reg .pred q; setp.ne.b32 q, %2, 0; @q st.global.b16 [%0], %1; }" ::"l"(p), "h"(*reinterpret_cast<const unsigned short*>(&v)), "r"((int)ok) : "memory");
}

// A tile's rows of a tensor, or of the write or read vectors, asked for by cp.async: as they lie in memory, zeros from the
// segment's end on, past the warp's channels and past N.
template <class L, typename IO>
__device__ __forceinline__ void ask_rows(const gdn_mla_view_t& v, const Spot& p, int t0, int lane, IO (*to)[L::CH])
{
    constexpr int PER = L::CH * sizeof(IO) / 16, UNIT = 16 / sizeof(IO);
#pragma unroll
    for (int u0 = 0; u0 < kTile * PER; u0 += 32) {
        const int u = u0 + lane, j = u / PER, c = u % PER * UNIT;
        if (u < kTile * PER) {
            const bool ok = t0 + j < p.t1 && c < p.channels;
            cp_async16_zero(&to[j][c], (const IO*)v.p + (ok ? (long long)(p.r.first + t0 + j) * v.tok + p.d0 + c : 0), ok);
        }
    }
}
template <class L, typename IO>
__device__ __forceinline__ void ask_vectors(const gdn_mla_view_t& v, const Spot& p, int N, int t0, int lane, IO (*to)[L::NS])
{
    constexpr int PER = L::NS * sizeof(IO) / 16, UNIT = 16 / sizeof(IO);
#pragma unroll
    for (int u0 = 0; u0 < kTile * PER; u0 += 32) {
        const int u = u0 + lane, j = u / PER, n = u % PER * UNIT;
        if (u < kTile * PER) {
            const bool ok = t0 + j < p.t1 && n < N;
            cp_async16_zero(&to[j][n], (const IO*)v.p + (ok ? (long long)(p.r.first + t0 + j) * v.tok + p.g * v.head + n : 0), ok);
        }
    }
}
// the vectors as fp32
template <class L, typename IO>
__device__ __forceinline__ void widen(const IO (*from)[L::NS], float (*to)[L::NS], int lane)
{
#pragma unroll
    for (int u0 = 0; u0 < kTile * L::NS / 8; u0 += 32) {
        const int u = u0 + lane;
        if (u < kTile * L::NS / 8) {
            float v[8];
            load8(&from[0][0] + 8 * u, v);
            store8(&to[0][0] + 8 * u, v);
        }
    }
}

// where a lane's states of place r lie in [B, D, N], and whether they exist
template <class L>
__device__ __forceinline__ long long state_at(const ScanArgs& a, const Spot& p, int lane, int r)
{
    return ((long long)p.b * a.s.D + p.d0 + L::channel(lane, r)) * a.s.N + L::S * (lane / L::CL);
}
template <class L>
__device__ __forceinline__ bool has_state(const ScanArgs& a, const Spot& p, int lane, int r)
{
    return p.has(L::channel(lane, r)) && L::S * (lane / L::CL) < a.s.N;
}

// -exp(A_log) log2(e) of two states.  Rates past fp32 count as its largest value: times any step size of use that forgets all the same,
// and times zero (a step past a sequence's end, or a state's product with a factor of zero) it is zero, as in exact arithmetic,
// where infinity times zero would make a NaN.  A NaN stays one.
__device__ __forceinline__ float2 rates(float2 A_log)
{
    return f2(max_nan(-expf(A_log.x) * kLog2e, -FLT_MAX), max_nan(-expf(A_log.y) * kLog2e, -FLT_MAX));
}

// the rates of a lane's states; zeros past N and past the warp's channels
template <class L>
__device__ __forceinline__ void load_rates(const ScanArgs& a, const Spot& p, int lane, States<L>& A)
{
#pragma unroll
    for (int r = 0; r < L::RC; r++) {
#pragma unroll
        for (int k = 0; k < L::S / 2; k++) A[r][k] = f2(0.f, 0.f);
        if (!has_state<L>(a, p, lane, r)) continue;
        get(a.A_log + (long long)(p.d0 + L::channel(lane, r)) * a.s.N + L::S * (lane / L::CL), A[r]);
#pragma unroll
        for (int k = 0; k < L::S / 2; k++) A[r][k] = rates(A[r][k]);
    }
}

// States that the kernels keep for one another lie as the lanes have them: place `at` of [places][RC][S / 4][32] float4.
template <class L>
__device__ __forceinline__ long long state_offset(long long at, int lane)
{
    return at * (L::RC * L::S / 4 * 32) + lane;
}
template <class L>
__device__ __forceinline__ void put_state(float4* q, const States<L>& h)
{
#pragma unroll
    for (int r = 0; r < L::RC; r++)
#pragma unroll
        for (int i = 0; i < L::S / 4; i++)
            q[(r * (L::S / 4) + i) * 32] = make_float4(h[r][2 * i].x, h[r][2 * i].y, h[r][2 * i + 1].x, h[r][2 * i + 1].y);
}
template <class L>
__device__ __forceinline__ void get_state(const float4* q, States<L>& h)
{
#pragma unroll
    for (int r = 0; r < L::RC; r++)
#pragma unroll
        for (int i = 0; i < L::S / 4; i++) {
            const float4 v = q[(r * (L::S / 4) + i) * 32];
            h[r][2 * i] = f2(v.x, v.y);
            h[r][2 * i + 1] = f2(v.z, v.w);
        }
}
// the place of what a segment hands on
__device__ __forceinline__ long long segment_at(const ScanArgs& a, const Spot& p, int seg)
{
    return (long long)(p.r.first / a.seg_len + p.b + seg) * (a.s.G * a.blocks) + p.block;
}
// where the states lie that enter chunk t / kSaveEvery of a sequence (neighbouring sequences' places never meet), and in
// them the four states n .. n + 3 of channel c of the group, as the forward's lanes have them
template <class F>
__device__ __forceinline__ long long saved_at(const ScanArgs& a, const Spot& p, int t)
{
    const long long place = (long long)(p.r.first / kSaveEvery) + p.b + t / kSaveEvery;
    return (place * a.s.G + p.g) * a.saved_blocks * (F::RC * F::S / 4 * 32);
}
template <class F>
__device__ __forceinline__ int saved_place(int c, int n)
{
    const int cc = c % F::CH, lane = n / F::S * F::CL + cc % F::CL, r = (lane % F::CH ^ cc) / F::CL;
    return ((c / F::CH * F::RC + r) * (F::S / 4) + n % F::S / 4) * 32 + lane;
}
// h (what enters segment s0) becomes what leaves segment s0 + (n - 1) step: for each of them in turn exp(A sum delta) h + (the
// segment's state from zero).  Four segments' values are asked for together.
template <class L>
__device__ __forceinline__ void carry(const ScanArgs& a, const Spot& p, int lane, int s0, int step, int n, const States<L>& A, States<L>& h)
{
    for (int i0 = 0; i0 < n; i0 += 4) {
        States<L> e[4];
        float w[4][L::RC];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const long long at = segment_at(a, p, s0 + min(i0 + i, n - 1) * step);
            get_state<L>(reinterpret_cast<const float4*>(a.seg_h) + state_offset<L>(at, lane), e[i]);
#pragma unroll
            for (int r = 0; r < L::RC; r++) w[i][r] = a.seg_d[at * L::CH + L::channel(lane, r)];
        }
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (i0 + i < n)
#pragma unroll
                for (int r = 0; r < L::RC; r++)
#pragma unroll
                    for (int k = 0; k < L::S / 2; k++) h[r][k] = fma2(ex2x2(mul2(f2(w[i][r], w[i][r]), A[r][k])), h[r][k], e[i][r][k]);
    }
}

// v[t][r]: a lane's share of a sum over the states, for token t of OT and place r.  Every lane gets the whole sum for the
// channel and the token that it owns.
template <class L>
__device__ __forceinline__ float to_owner(const float (&v)[L::OT][L::RC], int lane)
{
    static_assert(L::RC == 1 || L::RC == 2 || (L::RC == L::LS && L::OT == 1), "how places and tokens are dealt");
    float w[L::OT];
#pragma unroll
    for (int t = 0; t < L::OT; t++) {
        w[t] = v[t][0];
#pragma unroll
        for (int r = 1; r < L::RC; r++) w[t] += __shfl_xor_sync(0xffffffffu, v[t][r], L::CL * r);
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
__device__ __forceinline__ float from_owner(const float (&own)[L::OWN], int j, int r, int lane)
{
    const float v = own[j / L::OT];
    if (L::OT == 1) return r ? __shfl_xor_sync(0xffffffffu, v, L::CL * r) : v;
    return __shfl_sync(0xffffffffu, v, (j % L::OT) * L::CH + L::channel(lane, r));
}

// v[0 .. n - 1], n a power of two of at most LS: each summed over the LS lanes of a channel (lane = group of states * 32 / LS +
// channel), v[i] to the lanes whose group of states begins with the bits of i; each of the first log2 n exchanges halves what
// a lane still holds
template <int LS, int n>
__device__ __forceinline__ float states_sum(float (&v)[n], int lane)
{
    int m = 16;
#pragma unroll
    for (int k = n / 2; k; k >>= 1, m >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < k; i++) {
            const float keep = up ? v[i + k] : v[i], send = up ? v[i] : v[i + k];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m);
        }
    }
#pragma unroll
    for (; m > (32 / LS) / 2; m >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
    return v[0];
}

}  // namespace ssm
}  // namespace gdn
