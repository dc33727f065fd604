// mla_decode.cu -- attention of a few new tokens over the paged latent cache: the workers' plan, the join of their
// pieces, and the worker for f32 on the CUDA cores.
#include "mla_decode_common.cuh"

namespace gdn {
namespace mla {

DecodePlan decode_plan(const gdn_mla_cache_t& s)
{
    DecodePlan p;
    const int all = s.T * s.H;
    // Query rows of a worker on the tensor, the CUDA cores.  Fewer groups send each cache tile through fewer SMs, which
    // outweighs the shorter ring beside 80 rows.  At most 64 against 80, us: 32 sequences of 6000 rows of 512 + 64 values
    // under 72 query rows 88.2 / 73.6, under 160 (up to 6000 rows) 116.8 / 88.5, under 320 237 / 210; 160 over 256 + 64
    // 94.3 / 72.4; two sequences under 160 28.7 / 30.7.  (A load that filled both of two groups' tiles took 86.6, 172 and
    // 53.3 for the 160, 320 and 160 rows over 256 + 64.  It is not used: the library also runs on several GPUs at once, where
    // such loads are not safe.)
    const int most = s.io == GDN_BF16 ? kDecodeRows : 8;
    p.groups = (all + most - 1) / most;
    p.rows = (all + p.groups - 1) / p.groups;
    p.ctas = 152 / p.groups > 0 ? 152 / p.groups : 1;
    p.slots = p.ctas + s.B;
    const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    p.err_off = 256;
    p.l_off = up(p.err_off + (size_t)p.groups * p.ctas * 4);
    p.o_off = up(p.l_off + (size_t)p.groups * p.slots * p.rows * 4);
    p.total = up(p.o_off + (size_t)p.groups * p.slots * p.rows * s.dc * 4);
    return p;
}

namespace {

constexpr int kThreads = 256, kMaxRows = 8, kStep = 32;   // cache rows in shared memory at a time

// f32: 8 query rows a worker; a warp's lanes take a row's scores for 32 cache rows, a thread two latent columns of the
// output of all 8 rows.  FMAs bound it.
__global__ void __launch_bounds__(kThreads) decode_rows_kernel(const DecodeArgs a)
{
    extern __shared__ float smem[];
    __shared__ float P[kMaxRows][kStep], keep[kMaxRows], top[kMaxRows], sum[kMaxRows];
    __shared__ int place[3];
    const gdn_mla_cache_t& s = a.s;
    const int W = s.dc + s.dr, pitch = (W + 31) / 32 * 32 + 4;
    float *Q = smem, *K = smem + kMaxRows * pitch;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int cta = blockIdx.x, group = blockIdx.y;
    const Deal deal{a.len, s.B, s.maxpages * s.page};
    if (warp == 0) {
        const int all = deal_tiles(deal), share = deal_share(all, a.ctas);
        const int start = min((long long)share * cta, (long long)all);
        int b, tile;
        deal_find(deal, start, b, tile);
        if (lane == 0) {
            place[0] = b;
            place[1] = tile;
            place[2] = min(share, all - start);
            a.cta_err[group * a.ctas + cta] = 0;
        }
    }
    __syncthreads();
    cudaTriggerProgrammaticLaunchCompletion();   // the join's blocks may take their places
    int b = place[0], tile = place[1];
    int left = place[2];
    const int row0 = group * a.rows, rows = min(a.rows, s.T * s.H - row0);
    while (left > 0 && b < s.B) {
        const int n = deal.rows(b), tiles = deal.tiles(b);
        if (tiles == 0) {
            b++;
            continue;
        }
        const int to = min(tiles, tile + left);
        __syncthreads();
        for (int i = tid; i < kMaxRows * (pitch - 4) / 8; i += kThreads) {
            const int r = i / ((pitch - 4) / 8), c = (i - r * ((pitch - 4) / 8)) * 8;
            float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            if (r < rows && c < W) {
                const int t = (row0 + r) / s.H, h = (row0 + r) - t * s.H;
                const long long tok = (long long)b * s.T + t;
                if (c < s.dc)
                    load8((const float*)a.qc.p + tok * a.qc.tok + h * a.qc.head + c, x);
                else
                    load8((const float*)a.qr.p + tok * a.qr.tok + h * a.qr.head + (c - s.dc), x);
            }
            store8(Q + r * pitch + c, x);
        }
        if (tid < kMaxRows) {
            top[tid] = -INFINITY;
            sum[tid] = 0.f;
        }
        float o[kMaxRows][2] = {};
        const int last = min(n, to * kDecodeTile);
        for (int j0 = tile * kDecodeTile; j0 < last; j0 += kStep) {
            __syncthreads();
            for (int i = tid; i < kStep * (pitch - 4) / 8; i += kThreads) {
                const int r = i / ((pitch - 4) / 8), c = (i - r * ((pitch - 4) / 8)) * 8, j = j0 + r;
                float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (j < n && c < W) {
                    const int page = a.table[(long long)b * s.maxpages + j / s.page];
                    if (page >= 0 && page < s.npages)
                        load8((const float*)a.cache + ((long long)page * s.page + j % s.page) * W + c, x);
                }
                store8(K + r * pitch + c, x);
            }
            __syncthreads();
            {   // scores of row `warp` with cache row j0 + lane
                float x = 0.f;
                for (int c = 0; c < W; c += 4) {
                    const float4 q = *reinterpret_cast<const float4*>(Q + warp * pitch + c);
                    const float4 k = *reinterpret_cast<const float4*>(K + lane * pitch + c);
                    x += q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
                }
                const int t = (row0 + warp) / s.H;
                x = j0 + lane < n - (s.T - 1 - t) ? x * s.scale * 1.4426950408889634f : -INFINITY;
                float m = x;
#pragma unroll
                for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
                const float was = top[warp];
                m = fmaxf(m, was);
                const float base = m == -INFINITY ? 0.f : m;
                const float p = exp2f(x - base), f = exp2f(was - base);
                float l = p;
#pragma unroll
                for (int k = 16; k; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
                P[warp][lane] = p;
                __syncwarp();
                if (lane == 0) {
                    keep[warp] = f;
                    top[warp] = m;
                    sum[warp] = sum[warp] * f + l;
                }
            }
            __syncthreads();
            if (2 * tid < s.dc) {
#pragma unroll
                for (int r = 0; r < kMaxRows; r++) {
                    o[r][0] *= keep[r];
                    o[r][1] *= keep[r];
                }
#pragma unroll 4
                for (int k = 0; k < kStep; k++) {
                    const float2 v = *reinterpret_cast<const float2*>(K + k * pitch + 2 * tid);
#pragma unroll
                    for (int r = 0; r < kMaxRows; r++) {
                        o[r][0] += P[r][k] * v.x;
                        o[r][1] += P[r][k] * v.y;
                    }
                }
            }
        }
        __syncthreads();
        const bool whole = tile == 0 && to == tiles;
        const long long slot = ((long long)group * a.slots + cta + b) * a.rows;
        for (int r = 0; r < rows; r++) {
            const float inv = sum[r] > 0.f ? 1.f / sum[r] : sum[r];    // zero stays zero, a NaN a NaN
            const long long out = (long long)b * s.T * s.H + row0 + r;
            if (2 * tid < s.dc) {
                if (whole) {
                    float* p = (float*)a.o + out * s.dc + 2 * tid;
                    p[0] = o[r][0] * inv;
                    p[1] = o[r][1] * inv;
                } else {
                    *reinterpret_cast<float2*>(a.part_o + (slot + r) * s.dc + 2 * tid) =
                        make_float2(o[r][0] * inv, o[r][1] * inv);
                }
            }
            if (tid == 0) {
                const float l2 = sum[r] == 0.f ? -INFINITY : top[r] + log2f(sum[r]);
                if (!whole)
                    a.part_l[slot + r] = l2;
                else if (a.lse)
                    a.lse[out] = l2 * 0.6931471805599453f;
            }
        }
        left -= to - tile;
        tile = 0;
        b++;
    }
}

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d)
{
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d)
{
    const __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// o = sum_i 2^(l_i - l) o_i over a sequence's pieces, in their order.  Many rows fill the card with a warp a row, a
// thread 8 columns of it at a time.  Few rows (SPREAD) take a block for 128 columns of a row, a warp a quarter of the
// pieces and the quarters added in their order: one warp would walk up to 152 pieces in turn.  Sequences that one worker
// covered are written already; empty ones become zeros here.  Block (0, 0) also gathers the workers' error words.
constexpr int kJoinWarps = 4, kJoinAhead = 8;
template <typename T, bool SPREAD>
__global__ void __launch_bounds__(kJoinWarps * 32) decode_join_kernel(const DecodeArgs a)
{
    __shared__ int where[2];
    __shared__ float4 quarter[SPREAD ? kJoinWarps : 1][32];
    __shared__ float quarter_sum[SPREAD ? kJoinWarps : 1];
    const gdn_mla_cache_t& s = a.s;
    const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const Deal deal{a.len, s.B, s.maxpages * s.page};
    if (tid < 32) {      // the lengths are the caller's: read them before the workers are done
        const int share = deal_share(deal_tiles(deal), a.ctas), before = deal_before(deal, b);
        if (tid == 0) {
            where[0] = share;
            where[1] = before;
        }
    }
    __syncthreads();
    cudaGridDependencySynchronize();
    if (blockIdx.x == 0 && b == 0) {
        uint32_t err = 0;
        for (int i = tid; i < a.groups * a.ctas; i += kJoinWarps * 32) err |= a.cta_err[i];
        err = __syncthreads_or(err != 0);
        if (tid == 0) {
            a.status[0] = err ? kDevTimeout : kDevOk;
            a.status[1] = 0;
        }
    }
    const int chunks = SPREAD ? (s.dc + 127) >> 7 : 1, warp = tid >> 5;
    const int row = SPREAD ? blockIdx.x / chunks : blockIdx.x * kJoinWarps + warp;
    const int part = SPREAD ? blockIdx.x - row * chunks : 0;    // which 128 columns
    if (row >= s.T * s.H) return;
    const int tiles = deal.tiles(b);
    const long long out = (long long)b * s.T * s.H + row;
    T* o = (T*)a.o + out * s.dc;
    if (tiles == 0) {
        const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (part == 0 && (!SPREAD || warp == 0))
            for (int c = 8 * lane; c < s.dc; c += 256) store8(o + c, z);
        if (part == 0 && lane == 0 && (!SPREAD || warp == 0) && a.lse) a.lse[out] = -INFINITY;
        return;
    }
    const int c0 = where[1] / where[0], n = (where[1] + tiles - 1) / where[0] - c0 + 1;
    if (n == 1) return;
    const int group = row / a.rows, r = row - group * a.rows;
    const long long slot = (long long)group * a.slots + b + c0;
    const float* L = a.part_l + slot * a.rows + r;
    const float* O = a.part_o + (slot * a.rows + r) * s.dc;
    const long long next = (long long)a.rows * s.dc;
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, L[(long long)i * a.rows]);
#pragma unroll
    for (int k = 16; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float base = m == -INFINITY ? 0.f : m;
    if constexpr (SPREAD) {
        const int c = 128 * part + 4 * lane, from = n * warp / kJoinWarps, to = n * (warp + 1) / kJoinWarps;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
        for (int i0 = from; i0 < to; i0 += 32) {
            const float w = i0 + lane < to ? exp2f(L[(long long)(i0 + lane) * a.rows] - base) : 0.f;
            const int upto = min(32, to - i0);
            for (int i = 0; i < upto; i += kJoinAhead) {
                float4 v[kJoinAhead];
#pragma unroll
                for (int e = 0; e < kJoinAhead; e++)
                    if (c < s.dc && i + e < upto) v[e] = *reinterpret_cast<const float4*>(O + (i0 + i + e) * next + c);
#pragma unroll
                for (int e = 0; e < kJoinAhead; e++)
                    if (i + e < upto) {
                        const float f = __shfl_sync(0xffffffffu, w, i + e);
                        sum += f;
                        if (c < s.dc) x = make_float4(x.x + f * v[e].x, x.y + f * v[e].y, x.z + f * v[e].z, x.w + f * v[e].w);
                    }
            }
        }
        quarter[warp][lane] = x;
        if (lane == 0) quarter_sum[warp] = sum;
        __syncthreads();      // row, tiles and n are the block's: all of its warps come here
        if (warp) return;
        for (int k = 1; k < kJoinWarps; k++) {
            const float4 y = quarter[k][lane];
            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
            sum += quarter_sum[k];
        }
        const float inv = sum > 0.f ? 1.f / sum : sum;    // zero stays zero, a NaN a NaN
        if (c < s.dc) store4(o + c, x.x * inv, x.y * inv, x.z * inv, x.w * inv);
        if (part == 0 && lane == 0 && a.lse) a.lse[out] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
        return;
    }
    float sum = 0.f;
    for (int c = 8 * lane; c < 8 * 32 * ((s.dc + 255) / 256); c += 256) {   // every lane passes every shuffle
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        sum = 0.f;
        for (int i0 = 0; i0 < n; i0 += 32) {
            const float w = i0 + lane < n ? exp2f(L[(long long)(i0 + lane) * a.rows] - base) : 0.f;
            const int upto = min(32, n - i0);
            for (int i = 0; i < upto; i += kJoinAhead) {
                float v[kJoinAhead][8];
#pragma unroll
                for (int e = 0; e < kJoinAhead; e++)
                    if (c < s.dc && i + e < upto) load8(O + (i0 + i + e) * next + c, v[e]);
#pragma unroll
                for (int e = 0; e < kJoinAhead; e++)
                    if (i + e < upto) {
                        const float f = __shfl_sync(0xffffffffu, w, i + e);
                        sum += f;
                        if (c < s.dc) {
#pragma unroll
                            for (int k = 0; k < 8; k++) x[k] += f * v[e][k];
                        }
                    }
            }
        }
        const float inv = sum > 0.f ? 1.f / sum : sum;    // zero stays zero, a NaN a NaN
        if (c < s.dc) {
#pragma unroll
            for (int k = 0; k < 8; k++) x[k] *= inv;
            store8(o + c, x);
        }
    }
    if (lane == 0 && a.lse) a.lse[out] = sum == 0.f ? -INFINITY : (base + log2f(sum)) * 0.6931471805599453f;
}

cudaError_t run_rows(const DecodeArgs& a, cudaStream_t st)
{
    const int pitch = (a.s.dc + a.s.dr + 31) / 32 * 32 + 4;
    const size_t bytes = (size_t)(kMaxRows + kStep) * pitch * sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(decode_rows_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    decode_rows_kernel<<<dim3(a.ctas, a.groups), kThreads, bytes, st>>>(a);
    return cudaGetLastError();
}

// Launched as a dependent of the workers' kernel: its blocks find their place while the last workers finish.  A second
// launch, not the last worker of a sequence, because the workspace is the caller's and holds no counters between calls.
// The rows' pieces go to a block's warps where rows are few for the pieces that each has, about workers / B.  A warp a row
// against a block for 128 columns of a row, us of the call (sequences x lengths, rows a sequence, latent width):
// 1 x 32768, 64, 512: 47.3 / 31.0; 2 x 32768, 16, 512: 40.8 / 26.6; 8 x 32768, 16, 512: 63.7 / 61.0; 16 x 16384, 16, 512:
// 63.5 / 61.5; 4 x 32768, 160, 512: 86.5 / 84.6; 32 x 8192, 16, 512: 62.1 / 64.3; 16 x 6000, 40, 512: 39.0 / 41.1;
// 64 x 4096, 16, 256: 44.5 / 47.1.
constexpr long long kSpread = 4096;
template <typename T>
cudaError_t run_join(const DecodeArgs& a, cudaStream_t st)
{
    const bool spread = (long long)a.s.B * a.s.B * a.s.T * a.s.H <= kSpread;
    const int rows = a.s.T * a.s.H, chunks = (a.s.dc + 127) / 128;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(spread ? rows * chunks : (rows + kJoinWarps - 1) / kJoinWarps, a.s.B);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (spread) return cudaLaunchKernelEx(&cfg, decode_join_kernel<T, true>, a);
    return cudaLaunchKernelEx(&cfg, decode_join_kernel<T, false>, a);
}

}  // namespace

cudaError_t launch_decode(const DecodeArgs& a, cudaStream_t st)
{
    const bool bf16 = a.s.io == GDN_BF16;
    const cudaError_t e = bf16 ? launch_decode_tc(a, st) : run_rows(a, st);
    if (e != cudaSuccess) return e;
    return bf16 ? run_join<__nv_bfloat16>(a, st) : run_join<float>(a, st);
}

}  // namespace mla
}  // namespace gdn
