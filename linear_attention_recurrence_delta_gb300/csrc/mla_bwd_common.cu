// mla_bwd_common.cu -- the elementwise passes around the attention's gradients, for both I/O types; HBM bounds them.
#include "mla_internal.h"

namespace gdn {
namespace mla {

namespace {

constexpr int kThreads = 256;

// f32: delta[h, i] = dO[i, h] . o[i, h]: 16 threads a row of one head (dv <= 128), kRows rows each with their loads in
// flight.  (With bf16, dQ's kernel holds the rows of dO anyway and takes the sums itself.)
constexpr int kRows = 4;
__global__ void __launch_bounds__(kThreads) delta_kernel(const AttnArgs a)
{
    const gdn_mla_attn_t& s = a.s;
    const long long all = (long long)s.Nq * s.H, u0 = ((long long)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4)) * kRows;
    const int c = 8 * (threadIdx.x & 15);
    Raw8<float> x[kRows], y[kRows];
#pragma unroll
    for (int k = 0; k < kRows; k++)
        if (u0 + k < all && c < s.dv) {
            x[k] = raw8((const float*)a.o + (u0 + k) * s.dv + c);
            y[k] = raw8((const float*)a.dO + (u0 + k) * s.dv + c);
        }
#pragma unroll
    for (int k = 0; k < kRows; k++) {
        float t = 0.f;
        if (u0 + k < all && c < s.dv) {
            float v[8], w[8];
            values(x[k], v);
            values(y[k], w);
#pragma unroll
            for (int i = 0; i < 8; i++) t += v[i] * w[i];
        }
#pragma unroll
        for (int m = 8; m; m >>= 1) t += __shfl_xor_sync(0xffffffffu, t, m);
        if (c == 0 && u0 + k < all) a.delta[(u0 + k) % s.H * s.Nq + (u0 + k) / s.H] = t;
    }
}

// dkr = the key heads' shares, added in the heads' order
constexpr int kDkrThreads = 64;     // few rows: spread them over the SMs
template <typename T>
__global__ void __launch_bounds__(kDkrThreads) dkr_kernel(const AttnArgs a)
{
    cudaGridDependencySynchronize();     // launched as a dependent of the pass over the keys
    const gdn_mla_attn_t& s = a.s;
    const Rows rk = rows_of(a.cu_k, blockIdx.y, s.Tk, s.Nk);
    const int per = s.dr >> 3;
    const long long u = (long long)blockIdx.x * kDkrThreads + threadIdx.x;
    const int r = (int)(u / per), c = (int)(u - (long long)r * per) << 3;
    if (r >= rk.n) return;
    float t[8] = {};
#pragma unroll 8
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
    const int each = kThreads / 16 * kRows;
    const unsigned grid = (unsigned)((units + each - 1) / each);
    delta_kernel<<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_dkr(const AttnArgs& a, cudaStream_t st)
{
    const long long units = (long long)a.s.Tk * (a.s.dr >> 3);
    const dim3 grid((unsigned)((units + kDkrThreads - 1) / kDkrThreads), a.s.B);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kDkrThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return a.s.io == GDN_BF16 ? cudaLaunchKernelEx(&cfg, dkr_kernel<__nv_bfloat16>, a) : cudaLaunchKernelEx(&cfg, dkr_kernel<float>, a);
}

}  // namespace mla
}  // namespace gdn
