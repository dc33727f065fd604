// mla_bwd_common.cu -- the elementwise passes around the attention's gradients, for both I/O types; HBM bounds them.
#include "mla_internal.h"

namespace gdn {
namespace mla {

namespace {

constexpr int kThreads = 256;

// delta[h, i] = dO[i, h] . o[i, h], a warp a row of one head
template <typename T>
__global__ void __launch_bounds__(kThreads) delta_kernel(const AttnArgs a)
{
    const gdn_mla_attn_t& s = a.s;
    const long long u = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (u >= (long long)s.Nq * s.H) return;
    const int lane = threadIdx.x & 31;
    float t = 0.f;
    if (lane * 8 < s.dv) {
        float x[8], y[8];
        load8((const T*)a.o + u * s.dv + 8 * lane, x);
        load8((const T*)a.dO + u * s.dv + 8 * lane, y);
#pragma unroll
        for (int i = 0; i < 8; i++) t += x[i] * y[i];
    }
#pragma unroll
    for (int m = 8; m; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
    if (lane == 0) a.delta[(u % s.H) * s.Nq + u / s.H] = t;
}

// dkr = the key heads' shares, added in the heads' order
template <typename T>
__global__ void __launch_bounds__(kThreads) dkr_kernel(const AttnArgs a)
{
    const gdn_mla_attn_t& s = a.s;
    const Rows rk = rows_of(a.cu_k, blockIdx.y, s.Tk, s.Nk);
    const int per = s.dr >> 3;
    const long long u = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int r = (int)(u / per), c = (int)(u - (long long)r * per) << 3;
    if (r >= rk.n) return;
    float t[8] = {};
    for (int g = 0; g < s.Hkv; g++) {
        float x[8];
        load8(a.dkr_part + ((long long)g * s.Nk + rk.first + r) * s.dr + c, x);
#pragma unroll
        for (int i = 0; i < 8; i++) t[i] += x[i];
    }
    store8((T*)a.dkr.p + (long long)(rk.first + r) * a.dkr.tok + c, t);
}

}  // namespace

cudaError_t launch_delta(const AttnArgs& a, cudaStream_t st)
{
    const long long units = (long long)a.s.Nq * a.s.H;
    const unsigned grid = (unsigned)((units + kThreads / 32 - 1) / (kThreads / 32));
    if (a.s.io == GDN_BF16)
        delta_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
    else
        delta_kernel<float><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_dkr(const AttnArgs& a, cudaStream_t st)
{
    const long long units = (long long)a.s.Tk * (a.s.dr >> 3);
    const dim3 grid((unsigned)((units + kThreads - 1) / kThreads), a.s.B);
    if (a.s.io == GDN_BF16)
        dkr_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
    else
        dkr_kernel<float><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace mla
}  // namespace gdn
