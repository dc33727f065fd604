// mla_prep.cu -- latent norm, rotation of the position parts and the cache write, with their gradients.
//
// Elementwise but for one sum a token, so HBM bounds it: each input is read once and each output written once, in
// 16-byte pieces.  A warp holds a token's whole latent in registers (its sum of squares is one warp reduction); a
// thread rotates 8 pairs of two query heads by angles that it reads once.  Forwards both kinds of block run in one
// launch, because a decoding step is bound by launches, not bytes.  32768 tokens of 256 + 64 values with 16 heads of 64:
// 41 us forwards (176 MB, 4.3 TB/s), 87 us for both passes; a decoding step of 24 tokens takes 5 us from a cold cache, and
// the call's host time more.
#include "mla_internal.h"

namespace gdn {
namespace mla {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

__device__ __forceinline__ float warp_sum(float x)
{
#pragma unroll
    for (int m = 16; m; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// eight pairs as loaded: the two 8-value pieces of a row that hold them
struct Pairs {
    float a[8], b[8];
};

// pairs 8u .. 8u+7 of a row of width dr: where its pieces lie
template <bool IL>
__device__ __forceinline__ void piece(int u, int dr, int& ia, int& ib)
{
    ia = IL ? 16 * u : 8 * u;
    ib = IL ? ia + 8 : (dr >> 1) + 8 * u;
}

// turns them by the angles c, s.  IL: a pair is two neighbours, else equal places of the two pieces
template <bool IL>
__device__ __forceinline__ void turn(Pairs& x, const float (&c)[8], const float (&s)[8])
{
#pragma unroll
    for (int i = 0; i < 8; i++) {
        float& p = IL ? (i < 4 ? x.a[2 * i] : x.b[2 * i - 8]) : x.a[i];
        float& q = IL ? (i < 4 ? x.a[2 * i + 1] : x.b[2 * i - 7]) : x.b[i];
        const float v = p * c[i] - q * s[i];
        q = p * s[i] + q * c[i];
        p = v;
    }
}

// the angles of pairs 8u .. 8u+7 at a position, the other way round if BACK
template <bool BACK>
__device__ __forceinline__ void angles(const float* rot, int u, int dr, float (&c)[8], float (&s)[8])
{
    load8(rot + 8 * u, c);
    load8(rot + (dr >> 1) + 8 * u, s);
    if (BACK) {
#pragma unroll
        for (int i = 0; i < 8; i++) s[i] = -s[i];
    }
}

// What is rotated: a thread turns 8 pairs of kHeads query heads of one token by the same angles, or 8 pairs of its key.
// (Of 1, 2 and 4 heads two are fastest: 121, 94 and 146 us for the training batch's both passes; more read the angles
// less often but hold fewer threads on an SM.)
constexpr int kHeads = 2;
__host__ __device__ inline int threads_a_token(const gdn_mla_prep_t& s)
{
    return ((s.H + kHeads - 1) / kHeads + 1) * (s.dr >> 4);
}
__host__ __device__ inline int tokens_a_block(const gdn_mla_prep_t& s)
{
    const int p = threads_a_token(s);
    return p == 0 || p > kThreads ? 1 : kThreads / p;
}

// where token n's row of the cache begins, or null
template <typename T>
__device__ __forceinline__ T* cache_row(const PrepArgs& a, long long n, int pos)
{
    const int b = a.seq[n], at = pos / a.s.page;
    if (b < 0 || b >= a.s.B || at >= a.s.maxpages) return nullptr;
    const int page = a.table[(long long)b * a.s.maxpages + at];
    if (page < 0 || page >= a.s.npages) return nullptr;
    return (T*)a.lat.p + ((long long)page * a.s.page + (pos - at * a.s.page)) * (a.s.dc + a.s.dr);
}

// Block `block` of them.  BACK: the gradients' way (dqr to dqr_out, dkr to dkv), which zeroes a skipped token's.
template <typename T, bool BACK, bool IL>
__device__ __forceinline__ void rotate_rows(const PrepArgs& a, int block)
{
    const int p = threads_a_token(a.s), each = tokens_a_block(a.s), per = a.s.dr >> 4;
    const long long n = (long long)block * each + (each > 1 ? threadIdx.x / p : 0);
    if (n >= a.s.N || (each > 1 && (int)threadIdx.x >= each * p)) return;
    const int pos = a.pos[n];      // on its way while the rows are asked for
    for (int r = each > 1 ? threadIdx.x % p : threadIdx.x; r < p; r += kThreads) {
        const int u = r % per, h = r / per * kHeads;
        const bool key = h >= a.s.H;
        const gdn_mla_view_t& in = BACK ? a.dqr : a.qr;
        const gdn_mla_view_t& out = BACK ? a.dqr_out : a.qr_out;
        const T* x = key ? (BACK ? (const T*)a.dkr.p + n * a.dkr.tok : (const T*)a.kv + n * a.kv_tok + a.s.dc)
                         : (const T*)in.p + n * in.tok + h * in.head;
        const int heads = key ? 1 : min(kHeads, a.s.H - h);
        int ia, ib;
        piece<IL>(u, a.s.dr, ia, ib);
        Raw8<T> va[kHeads], vb[kHeads];      // as loaded: converted, twice the registers would hold fewer threads
#pragma unroll
        for (int k = 0; k < kHeads; k++)
            if (k < heads) {
                va[k] = raw8(x + k * in.head + ia);
                vb[k] = raw8(x + k * in.head + ib);
            }
        const bool bad = pos < 0 || pos >= a.s.npos;
        if (bad && !BACK) return;
        float c[8] = {}, s[8] = {};
        if (!bad) angles<BACK>(a.rot + (long long)pos * a.s.dr, u, a.s.dr, c, s);
        T* y = (T*)out.p + n * out.tok + h * out.head;
        if (key) {
            if (BACK) {
                y = (T*)a.dkv + n * a.dkv_tok + a.s.dc;
            } else if (a.s.page > 0) {
                y = cache_row<T>(a, n, pos);
                if (!y) continue;
                y += a.s.dc;
            } else {
                y = (T*)a.kr.p + n * a.kr.tok;
            }
        }
#pragma unroll
        for (int k = 0; k < kHeads; k++)
            if (k < heads) {
                Pairs v;
                values(va[k], v.a);
                values(vb[k], v.b);
                turn<IL>(v, c, s);
                if (bad) {
#pragma unroll
                    for (int i = 0; i < 8; i++) v.a[i] = v.b[i] = 0.f;
                }
                store8(y + k * out.head + ia, v.a);
                store8(y + k * out.head + ib, v.b);
            }
    }
}

// blocks [0, rows_blocks): what is rotated; the rest: a warp a token's norm, NV 8-value vectors of its latent a lane
template <typename T, bool IL, int NV>
__global__ void __launch_bounds__(kThreads, NV == 4 ? 2 : sizeof(T) == 4 ? 3 : 4) prep_kernel(const PrepArgs a, int rows_blocks)
{
    if ((int)blockIdx.x < rows_blocks) {
        rotate_rows<T, false, IL>(a, blockIdx.x);
        return;
    }
    const int lane = threadIdx.x & 31;
    const long long n = (long long)(blockIdx.x - rows_blocks) * kWarps + (threadIdx.x >> 5);
    if (n >= a.s.N) return;
    const int dc = a.s.dc, nv = dc >> 3;
    const int pos = a.pos[n];
    const T* x = (const T*)a.kv + n * a.kv_tok;
    float v[NV][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < NV; k++)
        if (lane + 32 * k < nv) load8(x + 8 * (lane + 32 * k), v[k]);
    if (pos < 0 || pos >= a.s.npos) return;
    T* lat = a.s.page > 0 ? cache_row<T>(a, n, pos) : (T*)a.lat.p + n * a.lat.tok;
    if (!lat) return;
#pragma unroll
    for (int k = 0; k < NV; k++)
        if (lane + 32 * k < nv) {
#pragma unroll
            for (int i = 0; i < 8; i++) ss += v[k][i] * v[k][i];
        }
    const float r = rsqrtf(warp_sum(ss) / (float)dc + a.s.eps);
#pragma unroll
    for (int k = 0; k < NV; k++)
        if (lane + 32 * k < nv) {
            float w[8];
            const float* wp = a.w + 8 * (lane + 32 * k);
#pragma unroll
            for (int i = 0; i < 8; i++) w[i] = v[k][i] * r * wp[i];
            store8(lat + 8 * (lane + 32 * k), w);
        }
}

// Gradients: with r = rsqrt(mean x^2 + eps) and g = dy w,  dx = r (g - x r^2 mean(g x)),  dw = sum_n dy x r.
// A block's warps walk tokens a fixed way apart and keep their share of dw in registers; the shares are added in a
// fixed order here and in sum_dw_kernel.
template <typename T, int NV>
__device__ __forceinline__ void latents_bwd(const PrepArgs& a, int block, int blocks)
{
    __shared__ float red[kWarps][256];   // a quarter of the widest latent's shares at a time
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int dc = a.s.dc, nv = dc >> 3;
    float dw[NV][8] = {}, w[NV][8];
#pragma unroll
    for (int k = 0; k < NV; k++)
        if (lane + 32 * k < nv && a.s.N > 0) {     // without tokens there need be no weight
#pragma unroll
            for (int i = 0; i < 8; i++) w[k][i] = a.w[8 * (lane + 32 * k) + i];
        }
    const long long step = (long long)blocks * kWarps;
    for (long long n = (long long)block * kWarps + warp; n < a.s.N; n += step) {
        const int pos = a.pos[n];
        const bool bad = pos < 0 || pos >= a.s.npos;
        const T* x = (const T*)a.kv + n * a.kv_tok;
        const T* dy = (const T*)a.dlat.p + n * a.dlat.tok;
        T* dx = (T*)a.dkv + n * a.dkv_tok;
        float v[NV][8], g[NV][8];
        float ss = 0.f, gx = 0.f;
#pragma unroll
        for (int k = 0; k < NV; k++)
            if (lane + 32 * k < nv) {
                load8(x + 8 * (lane + 32 * k), v[k]);
                load8(dy + 8 * (lane + 32 * k), g[k]);
            }
#pragma unroll
        for (int k = 0; k < NV; k++)
            if (lane + 32 * k < nv) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    if (bad) g[k][i] = v[k][i] = 0.f;      // whatever a skipped token holds, it adds nothing
                    ss += v[k][i] * v[k][i];
                    gx += g[k][i] * w[k][i] * v[k][i];
                }
            }
        const float r = rsqrtf(warp_sum(ss) / (float)dc + a.s.eps);
        const float m = warp_sum(gx) / (float)dc * r * r;
#pragma unroll
        for (int k = 0; k < NV; k++)
            if (lane + 32 * k < nv) {
                float d[8];
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    d[i] = bad ? 0.f : r * (g[k][i] * w[k][i] - v[k][i] * m);
                    dw[k][i] += bad ? 0.f : g[k][i] * (v[k][i] * r);
                }
                store8(dx + 8 * (lane + 32 * k), d);
            }
    }
#pragma unroll
    for (int k = 0; k < NV; k++) {
        if (256 * k >= dc) break;
#pragma unroll
        for (int i = 0; i < 8; i++) red[warp][8 * lane + i] = dw[k][i];
        __syncthreads();
        const int col = 256 * k + threadIdx.x;
        if (col < dc) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < kWarps; i++) sum += red[i][threadIdx.x];
            a.partial[(long long)block * dc + col] = sum;
        }
        __syncthreads();
    }
}

// Blocks [0, latents): the norm's gradients, which take longest; the rest: what was rotated.  One launch for latents up to
// 256 wide (32768 tokens, 16 heads of 64: 94.3 to 88.2 us for both passes; f32 144 to 139); wider ones hold twice the
// registers or more, which would leave the rotation half its threads (512 wide 114.9 against 118.6 us in one launch, 1024
// wide 95.7 against 100.9), and go in two.
template <typename T, bool IL, int NV>
__global__ void __launch_bounds__(kThreads, NV == 4 ? 1 : NV == 2 ? 2 : sizeof(T) == 4 ? 3 : 4) prep_bwd_kernel(const PrepArgs a, int latents)
{
    if (NV > 1 || (int)blockIdx.x < latents)
        latents_bwd<T, NV>(a, blockIdx.x, latents);
    else
        rotate_rows<T, true, IL>(a, blockIdx.x - latents);
}

template <typename T, bool IL>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 3 : 4) rows_bwd_kernel(const PrepArgs a)
{
    rotate_rows<T, true, IL>(a, blockIdx.x);
}

__global__ void __launch_bounds__(1024) sum_dw_kernel(const float* part, float* dw, int blocks, int dc)
{
    cudaGridDependencySynchronize();     // launched as a dependent of the shares' kernel
    __shared__ float red[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < dc) {
#pragma unroll 8
        for (int b = threadIdx.y; b < blocks; b += 32) s += part[(long long)b * dc + c];
    }
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dc) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; i++) t += red[i][threadIdx.x];
        dw[c] = t;
    }
}

long long rows_blocks(const gdn_mla_prep_t& s)
{
    if (threads_a_token(s) == 0) return 0;
    const int each = tokens_a_block(s);
    return ((long long)s.N + each - 1) / each;
}

template <typename T, bool IL, int NV>
void start(const PrepArgs& a, bool backward, cudaStream_t st)
{
    const long long rows = rows_blocks(a.s);
    if (backward) {
        const int latents = prep_bwd_blocks(a.s.N);
        if (NV > 1 && rows > 0) rows_bwd_kernel<T, IL><<<(unsigned)rows, kThreads, 0, st>>>(a);
        prep_bwd_kernel<T, IL, NV><<<(unsigned)(latents + (NV > 1 ? 0 : rows)), kThreads, 0, st>>>(a, latents);
    } else {
        prep_kernel<T, IL, NV><<<(unsigned)(rows + (a.s.N + kWarps - 1) / kWarps), kThreads, 0, st>>>(a, (int)rows);
    }
}

template <typename T, bool IL>
void start(const PrepArgs& a, bool backward, cudaStream_t st)
{
    if (a.s.dc <= 256)
        start<T, IL, 1>(a, backward, st);
    else if (a.s.dc <= 512)
        start<T, IL, 2>(a, backward, st);
    else
        start<T, IL, 4>(a, backward, st);
}

cudaError_t launch(const PrepArgs& a, bool backward, cudaStream_t st)
{
    const bool il = a.s.interleaved != 0;
    if (a.s.io == GDN_BF16)
        il ? start<__nv_bfloat16, true>(a, backward, st) : start<__nv_bfloat16, false>(a, backward, st);
    else
        il ? start<float, true>(a, backward, st) : start<float, false>(a, backward, st);
    return cudaGetLastError();
}

}  // namespace

// blocks that walk the tokens of the backward pass: four on each SM, or a warp a token
int prep_bwd_blocks(int N)
{
    const int need = (N + kWarps - 1) / kWarps;
    return need < 1 ? 1 : (need < 4 * 152 ? need : 4 * 152);
}

cudaError_t launch_prep(const PrepArgs& a, cudaStream_t st) { return launch(a, false, st); }

cudaError_t launch_prep_bwd(const PrepArgs& a, cudaStream_t st)
{
    const cudaError_t e = launch(a, true, st);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.s.dc + 31) / 32);
    cfg.blockDim = dim3(32, 32);
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, sum_dw_kernel, (const float*)a.partial, a.dw, prep_bwd_blocks(a.s.N), a.s.dc);
}

}  // namespace mla
}  // namespace gdn
