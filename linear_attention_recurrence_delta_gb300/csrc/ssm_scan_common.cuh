// ssm_scan_common.cuh -- what the forward and the backward scan share: how a warp is laid out, and how tokens are staged.
//
// A warp takes CH neighbouring channels of one group of one sequence (or a segment of it).  LS = 1, 2, 4 or 8 lanes, CL =
// 32 / LS apart, hold the same RC channels (RC <= LS, CH = RC CL), each lane 8 states of every one (8 LS >= N; those past N
// stay zero).  So a write or read vector is fetched from shared memory 8 values a lane for RC channels' use, which
// matters: 16 bytes a lane from shared memory take as long as four instructions of every scheduler, broadcast or not.
// What goes by channel alone (rows of x, step sizes, gates, results) has an owner: lane l owns channel l % CH at the tokens
// whose number is l / CH modulo OT = 32 / CH.  Place r of a lane's arrays is the channel that differs from its own by r CL,
// its own for r = 0.
#pragma once

#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

constexpr int kTile = kSaveEvery;      // tokens that are loaded together

template <int LS_, int RC_>
struct Lay {
    static constexpr int LS = LS_, RC = RC_, NS = 8 * LS, CL = 32 / LS, CH = RC * CL, OT = 32 / CH;
    // the channel of place r, within the warp's
    static __device__ __forceinline__ int channel(int lane, int r) { return (lane % CH) ^ (CL * r); }
};

// where a warp works
struct Spot {
    int g, b, seg;        // group, sequence, segment
    int block;            // its number among all warps' blocks of channels
    int d0, channels;     // its first channel, how many it has (0: none)
    Rows r;               // the sequence's rows
    int t0, t1;           // tokens of the segment
    __device__ __forceinline__ bool has(int channel) const { return channel < channels; }
};
// W warps a CTA; a.ctas CTAs take a group's channels
template <class L, int W>
__device__ __forceinline__ Spot spot(const ScanArgs& a)
{
    Spot p;
    p.block = blockIdx.x * W + (threadIdx.x >> 5);
    p.g = blockIdx.x / a.ctas;
    p.b = blockIdx.y;
    p.seg = blockIdx.z;
    const int each = a.s.D / a.s.G, c0 = min(each, (p.block - p.g * a.ctas * W) * L::CH);
    p.d0 = p.g * each + c0;
    p.channels = min(L::CH, each - c0);
    p.r = rows_of(a.cu, p.b, a.s.T, a.s.rows);
    p.t0 = (int)min((long long)p.r.n, (long long)p.seg * a.seg_len);
    p.t1 = (int)min((long long)p.r.n, (long long)p.t0 + a.seg_len);
    return p;
}

__device__ __forceinline__ float2 ex2x2(float2 x) { return f2(ex2_approx(x.x), ex2_approx(x.y)); }
__device__ __forceinline__ void get8(const float* p, float2 (&x)[4])
{
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const float4 v = reinterpret_cast<const float4*>(p)[i];
        x[2 * i] = f2(v.x, v.y);
        x[2 * i + 1] = f2(v.z, v.w);
    }
}
__device__ __forceinline__ void put8(float* p, const float2 (&x)[4])
{
#pragma unroll
    for (int i = 0; i < 2; i++) reinterpret_cast<float4*>(p)[i] = make_float4(x[2 * i].x, x[2 * i].y, x[2 * i + 1].x, x[2 * i + 1].y);
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

// A tile of a lane's own channel: zeros from the segment's end on and past the warp's channels.
template <typename IO>
struct Column {
    IO v[kTile];
    __device__ __forceinline__ void load(const gdn_mla_view_t& view, const Spot& p, int t0, int lane)
    {
        const IO* src = (const IO*)view.p + (long long)(p.r.first + t0) * view.tok + p.d0 + lane;
        const bool in = p.has(lane);
        if (t0 + kTile <= p.t1) {
#pragma unroll
            for (int j = 0; j < kTile; j++) v[j] = in ? src[j * view.tok] : rec::from_f<IO>(0.f);
        } else {
#pragma unroll
            for (int j = 0; j < kTile; j++) v[j] = in && t0 + j < p.t1 ? src[j * view.tok] : rec::from_f<IO>(0.f);
        }
    }
};

// A tile's write or read vectors, kTile tokens of NS values, in pieces of 8.
template <class L, typename IO>
struct Vectors {
    static constexpr int PIECES = kTile * L::LS, V = (PIECES + 31) / 32;
    Raw8<IO> raw[V];
    // asked for: zeros from the segment's end on and past N
    __device__ __forceinline__ void load(const gdn_mla_view_t& v, const Spot& p, int N, int t0, int lane)
    {
        const IO* src = (const IO*)v.p + p.g * v.head;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int u = 32 * i + lane, j = u / L::LS, c = 8 * (u % L::LS);
            raw[i] = Raw8<IO>{};
            if (u < PIECES && t0 + j < p.t1 && c < N) raw[i] = raw8(src + (long long)(p.r.first + t0 + j) * v.tok + c);
        }
    }
    __device__ __forceinline__ void store(float* to, int lane) const
    {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int u = 32 * i + lane;
            if (u < PIECES) {
                float x[8];
                values(raw[i], x);
                store8(to + 8 * u, x);
            }
        }
    }
};

// where a lane's states of place r lie in [B, D, N]
template <class L>
__device__ __forceinline__ long long state_at(const ScanArgs& a, const Spot& p, int lane, int r)
{
    return ((long long)p.b * a.s.D + p.d0 + L::channel(lane, r)) * a.s.N + 8 * (lane / L::CL);
}

// -exp(A_log) log2(e) of a lane's states; zeros past N and past the warp's channels
template <class L>
__device__ __forceinline__ void load_rates(const ScanArgs& a, const Spot& p, int lane, float2 (&A)[L::RC][4])
{
    const int n = 8 * (lane / L::CL);
#pragma unroll
    for (int r = 0; r < L::RC; r++) {
#pragma unroll
        for (int k = 0; k < 4; k++) A[r][k] = f2(0.f, 0.f);
        const int c = L::channel(lane, r);
        if (!p.has(c) || n >= a.s.N) continue;
        get8(a.A_log + (long long)(p.d0 + c) * a.s.N + n, A[r]);
#pragma unroll
        for (int k = 0; k < 4; k++) A[r][k] = f2(-expf(A[r][k].x) * kLog2e, -expf(A[r][k].y) * kLog2e);
    }
}

// States that the kernels keep for one another lie as the lanes have them: place `at` of [places][RC][2][32] float4.
template <class L>
__device__ __forceinline__ void put_state(float* to, long long at, int lane, const float2 (&h)[L::RC][4])
{
    float4* q = reinterpret_cast<float4*>(to) + at * (L::RC * 64) + lane;
#pragma unroll
    for (int r = 0; r < L::RC; r++)
#pragma unroll
        for (int i = 0; i < 2; i++) q[(2 * r + i) * 32] = make_float4(h[r][2 * i].x, h[r][2 * i].y, h[r][2 * i + 1].x, h[r][2 * i + 1].y);
}
template <class L>
__device__ __forceinline__ void get_state(const float* from, long long at, int lane, float2 (&h)[L::RC][4])
{
    const float4* q = reinterpret_cast<const float4*>(from) + at * (L::RC * 64) + lane;
#pragma unroll
    for (int r = 0; r < L::RC; r++)
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const float4 v = q[(2 * r + i) * 32];
            h[r][2 * i] = f2(v.x, v.y);
            h[r][2 * i + 1] = f2(v.z, v.w);
        }
}
// the place of what a segment hands on
template <int W>
__device__ __forceinline__ long long segment_at(const ScanArgs& a, const Spot& p, int seg)
{
    return ((long long)seg * a.s.B + p.b) * (a.s.G * a.ctas * W) + p.block;
}
// the place of the states that enter chunk t / kSaveEvery of a sequence, [blocks of 32 channels] as the forward's lanes have
// them: neighbouring sequences' places never meet
__device__ __forceinline__ long long saved_at(const ScanArgs& a, const Spot& p, int t)
{
    return ((long long)(p.r.first / kSaveEvery) + p.b + t / kSaveEvery) * (a.s.G * a.warps);
}
// h (what enters segment s) becomes what leaves it: exp(A sum delta) h + (the segment's state from zero)
template <class L, int W>
__device__ __forceinline__ void carry(const ScanArgs& a, const Spot& p, int lane, int s, const float2 (&A)[L::RC][4], float2 (&h)[L::RC][4])
{
    float2 e[L::RC][4];
    const long long at = segment_at<W>(a, p, s);
    get_state<L>(a.seg_h, at, lane, e);
#pragma unroll
    for (int r = 0; r < L::RC; r++) {
        const float w = a.seg_d[at * L::CH + L::channel(lane, r)];
#pragma unroll
        for (int k = 0; k < 4; k++) h[r][k] = fma2(ex2x2(mul2(f2(w, w), A[r][k])), h[r][k], e[r][k]);
    }
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
