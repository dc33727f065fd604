// ssm_scan_common.cuh -- what the forward and the backward scan share: how a CTA is laid out, and how tokens are staged.
//
// A lane holds 4 states of one channel, LS = 2, 4, 8 or 16 neighbouring lanes a channel's 4 LS >= N states (those past N
// stay zero), a CTA of 128 threads 128 / LS neighbouring channels of one group and one sequence (or a segment of it).
#pragma once

#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

constexpr int kScanThreads = 128;

template <int LS_>
struct Lay {
    static constexpr int LS = LS_, NS = 4 * LS, CH = kScanThreads / LS, PP = CH / 8;
};

// where a thread's CTA works
struct Spot {
    int g, b, seg;        // group, sequence, segment
    int d0, channels;     // its first channel, how many of CH it has
    Rows r;               // the sequence's rows
    int t0, t1;           // tokens of the segment
};
template <class L>
__device__ __forceinline__ Spot spot(const ScanArgs& a, int blocks)
{
    Spot p;
    p.g = blockIdx.x / blocks;
    p.b = blockIdx.y;
    p.seg = blockIdx.z;
    const int each = a.s.D / a.s.G, c0 = (blockIdx.x - p.g * blocks) * L::CH;
    p.d0 = p.g * each + c0;
    p.channels = min(L::CH, each - c0);
    p.r = rows_of(a.cu, p.b, a.s.T, a.s.rows);
    p.t0 = (int)min((long long)p.r.n, (long long)p.seg * a.seg_len);
    p.t1 = (int)min((long long)p.r.n, (long long)p.t0 + a.seg_len);
    return p;
}

// The write (or read) vectors of tokens t0 .. t0 + K - 1 (zeros from t1 on and past N) as fp32 rows of NS values.
template <class L, typename IO, int K>
__device__ __forceinline__ void stage_vectors(const ScanArgs& a, const gdn_mla_view_t& v, const Spot& p, int t0, int t1,
                                              float (*to)[L::NS])
{
    const IO* src = (const IO*)v.p + p.g * v.head;
#pragma unroll
    for (int u0 = 0; u0 < K * L::NS / 8; u0 += kScanThreads) {
        const int u = u0 + threadIdx.x, j = u / (L::NS / 8), c = 8 * (u % (L::NS / 8));
        if (u < K * L::NS / 8) {
            float x[8] = {};
            if (t0 + j < t1 && c < a.s.N) load8(src + (long long)(p.r.first + t0 + j) * v.tok + c, x);
            store8(&to[j][c], x);
        }
    }
}

// -exp(A_log) log2(e) of a lane's four states; zeros past N and past the block's channels
__device__ __forceinline__ void load_rates(const ScanArgs& a, int d, int n, bool in, float (&A)[4])
{
#pragma unroll
    for (int i = 0; i < 4; i++) A[i] = 0.f;
    if (!in || n >= a.s.N) return;
    const float4 v = *reinterpret_cast<const float4*>(a.A_log + (long long)d * a.s.N + n);
    A[0] = -expf(v.x) * kLog2e;
    A[1] = -expf(v.y) * kLog2e;
    A[2] = -expf(v.z) * kLog2e;
    A[3] = -expf(v.w) * kLog2e;
}

__device__ __forceinline__ void get4(const float* p, float (&x)[4])
{
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void put4(float* p, const float (&x)[4])
{
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// the place of the state that enters chunk t / kSaveEvery of a sequence: neighbouring sequences' places never meet
__device__ __forceinline__ long long saved_at(const Spot& p, int t)
{
    return (long long)(p.r.first / kSaveEvery) + p.b + t / kSaveEvery;
}

// sum over the LS lanes of a channel
template <int LS>
__device__ __forceinline__ float lanes_sum(float x)
{
#pragma unroll
    for (int m = LS / 2; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

}  // namespace ssm
}  // namespace gdn
