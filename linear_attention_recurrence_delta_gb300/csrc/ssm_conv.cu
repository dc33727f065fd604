// ssm_conv.cu -- short causal convolution of each channel with SiLU, its gradients, and its form for new tokens.
//
// pre[t] = bias + sum_k w[k] x[t - W + 1 + k], y = silu(pre).  A thread walks a strip of time for four neighbouring
// channels with the last rows in registers, in rings of four whose turning the unrolled loop knows, so that a row is read
// once (and W - 1 rows more a strip, from L2).  HBM bounds it, once rows are asked for well ahead, the arithmetic is packed
// and no row within a strip has a branch: 8 x 4096 rows of 2048 channels, four taps, take 50 us forwards (268 MB; 71 with
// eight channels a thread and a test a row) and 86 us back (403 MB; 252 with a row at a time), 5 for the sums of the shares.
#include "ssm_common.cuh"

namespace gdn {
namespace ssm {

namespace {

constexpr int kThreads = 256, kBackThreads = 128;
constexpr int kStrip = 32;        // rows a thread walks forwards (64: prompts 25 us for 15, few threads; 16: 153 us for 149 both ways)
constexpr int kBackStrip = 128;   // rows a thread walks for the gradients (64: 159 us for 149 both ways; 32: 197)

// the taps of C channels: w[k][c] of [D, W]
template <int W, int C>
__device__ __forceinline__ void load_taps(const float* w, float (&t)[W][C])
{
    float raw[W * C];
#pragma unroll
    for (int i = 0; i < W * C / 4; i++) {
        const float4 v = reinterpret_cast<const float4*>(w)[i];
        raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int k = 0; k < W; k++)
#pragma unroll
        for (int c = 0; c < C; c++) t[k][c] = raw[c * W + k];
}

// one row: the output of 8 channels from the rows before it and this one, which then joins them
template <int W>
__device__ __forceinline__ void step8(const float (&taps)[W][8], const float (&bias)[8], float (&past)[W - 1][8], const float (&x)[8],
                                      int silu, float (&y)[8])
{
#pragma unroll
    for (int c = 0; c < 8; c++) {
        float p = bias[c];
#pragma unroll
        for (int k = 0; k < W - 1; k++) p = fmaf(taps[k][c], past[k][c], p);
        p = fmaf(taps[W - 1][c], x[c], p);
        y[c] = silu ? p * sigmoid(p) : p;
#pragma unroll
        for (int k = 0; k + 1 < W - 1; k++) past[k][c] = past[k + 1][c];
        past[W - 2][c] = x[c];
    }
}

// Rows on their way to a thread: groups of four rows of its own four channels, by cp.async into a ring of its own in shared
// memory, so that what is in flight takes no registers and no thread waits for another.  Three groups ahead with bf16 (138 us
// for 8 x 4096 rows of 2048 channels both ways, 150 with one group ahead or with four rows in registers, 164 with seven groups
// and fewer CTAs), one with f32, whose rows are twice the bytes.
template <typename IO, int THREADS>
struct Rows4 {
    static constexpr int GROUPS = sizeof(IO) == 2 ? 4 : 2;
    Raw4<IO> v[GROUPS][4][THREADS];
    __device__ __forceinline__ static void copy(Raw4<IO>* to, const IO* from)
    {
        const uint32_t s = (uint32_t)__cvta_generic_to_shared(to);
        if (sizeof(IO) == 2) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(s), "l"(from) : "memory");
        else asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(from) : "memory");
    }
    // rows t .. t + 3 of p, those before `end`
    __device__ __forceinline__ void ask(const IO* p, long long tok, int t, int end)
    {
        Raw4<IO>* to = &v[(t >> 2) & (GROUPS - 1)][0][threadIdx.x];
        if (t + 4 <= end)
#pragma unroll
            for (int j = 0; j < 4; j++) copy(to + j * THREADS, p + (t + j) * tok);
        else
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (t + j < end) copy(to + j * THREADS, p + (t + j) * tok);
    }
    __device__ __forceinline__ Raw4<IO> get(int t, int j) const { return v[(t >> 2) & (GROUPS - 1)][j][threadIdx.x]; }
    // the oldest group, if GROUPS - 1 have been asked for
    __device__ __forceinline__ static void arrived() { asm volatile("cp.async.wait_group %0;" ::"n"(GROUPS - 2) : "memory"); }
};

template <int W>
__device__ __forceinline__ void load_taps(const float* w, Four (&t)[W])
{
    float raw[W][4];
    load_taps<W, 4>(w, raw);
#pragma unroll
    for (int k = 0; k < W; k++) t[k] = four(raw[k]);
}

// rows t0 - (W - 1) .. t0 - 1 of a sequence into a ring (t0 a multiple of 4): its own, its state's, or zeros
template <typename IO, int W>
__device__ __forceinline__ void load_past(const IO* x, long long tok, const void* s0, int b, int D, int c, int t0, Four (&ring)[4])
{
    ring[0] = all(0.f);
#pragma unroll
    for (int k = 1; k < W; k++) {
        const int t = t0 - k;
        ring[4 - k] = all(0.f);
        if (t >= 0) ring[4 - k] = raw4(x + t * tok).get();
        else if (s0) ring[4 - k] = raw4((const IO*)s0 + ((long long)b * (W - 1) + t + W - 1) * D + c).get();
    }
}

// Sequence blockIdx.y (SPARSE: whose place it is); threads run over (strip, piece of 4 channels), pieces fastest.
template <typename IO, int W, bool SILU, bool SPARSE>
__global__ void __launch_bounds__(kThreads, 3) conv_kernel(const ConvArgs a)
{
    const int D = a.s.D, pieces = D >> 2;
    const long long u = (long long)blockIdx.x * kThreads + threadIdx.x;
    int strip = (int)(u / pieces), b = blockIdx.y;
    const int c = (int)(u - (long long)strip * pieces) << 2;
    if (SPARSE) {
        const Place p = place_of(a.cu, a.s.B, a.s.rows, kStrip, strip);
        b = p.b;
        strip = p.piece;
    }
    const Rows r = rows_of(a.cu, b, a.s.T, a.s.rows);
    const long long first = (long long)strip * kStrip;
    if (first >= r.n && strip > 0) return;
    const int t0 = (int)first, end = min(r.n, t0 + kStrip);
    const IO* x = (const IO*)a.x.p + (long long)r.first * a.x.tok + c;
    IO* y = (IO*)a.y.p + (long long)r.first * a.y.tok + c;
    Four taps[W], bias = all(0.f), ring[4];
    load_taps<W>(a.w + (long long)c * W, taps);
    if (a.bias) bias = raw4(a.bias + c).get();
    using Ring = Rows4<IO, kThreads>;
    __shared__ Ring rows;
    auto row = [&](int t, int j) {
        ring[j] = rows.get(t, j).get();
        Four p = bias;
#pragma unroll
        for (int k = 0; k < W; k++) p = fma(taps[k], ring[(j + 5 - W + k) & 3], p);
        put(y + (long long)(t + j) * a.y.tok, SILU ? mul(p, sigmoid4(p)) : p);
    };
#pragma unroll
    for (int g = 0; g < Ring::GROUPS - 1; g++) {
        rows.ask(x, a.x.tok, t0 + 4 * g, end);
        rec::cp_async_commit();
    }
    load_past<IO, W>(x, a.x.tok, a.s0, b, D, c, t0, ring);
    int t = t0;
    for (; t + 4 <= end; t += 4) {
        Ring::arrived();
        rows.ask(x, a.x.tok, t + 4 * (Ring::GROUPS - 1), end);
        rec::cp_async_commit();
#pragma unroll
        for (int j = 0; j < 4; j++) row(t, j);
    }
    rec::cp_async_wait_all();
#pragma unroll
    for (int j = 0; j < 3; j++)
        if (t + j < end) row(t, j);
    if (!a.sT || end != r.n) return;
    // the last W - 1 rows: in the ring by their number modulo 4
#pragma unroll
    for (int k = 0; k < W - 1; k++) {
        const int at = (end - (W - 1) + k) & 3;
        const Four v = at == 0 ? ring[0] : at == 1 ? ring[1] : at == 2 ? ring[2] : ring[3];
        put((IO*)a.sT + ((long long)b * (W - 1) + k) * D + c, v);
    }
}

// New tokens: a thread has 8 channels of a sequence.
template <typename IO, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvStepArgs a)
{
    const int D = a.s.D, pieces = D >> 3;
    const long long u = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int b = (int)(u / pieces), c = (int)(u - (long long)b * pieces) << 3;
    if (b >= a.s.B) return;
    const int src = a.src ? a.src[b] : b, dst = a.dst ? a.dst[b] : src;
    const IO* x = (const IO*)a.x.p + (long long)b * a.s.T * a.x.tok + c;
    IO* y = (IO*)a.y.p + (long long)b * a.s.T * a.y.tok + c;
    float taps[W][8], bias[8] = {}, past[W - 1][8];
    load_taps<W, 8>(a.w + (long long)c * W, taps);
    if (a.bias) load8(a.bias + c, bias);
#pragma unroll
    for (int k = 0; k < W - 1; k++) {
        if (src >= 0 && src < a.s.slots) load8((const IO*)a.state + ((long long)src * (W - 1) + k) * D + c, past[k]);
        else
#pragma unroll
            for (int i = 0; i < 8; i++) past[k][i] = 0.f;
    }
    for (int t = 0; t < a.s.T; t++) {
        float v[8], o[8];
        load8(x + t * a.x.tok, v);
        step8<W>(taps, bias, past, v, a.s.silu, o);
        store8(y + t * a.y.tok, o);
    }
    if (dst >= 0 && dst < a.s.slots)
#pragma unroll
        for (int k = 0; k < W - 1; k++) store8((IO*)a.state + ((long long)dst * (W - 1) + k) * D + c, past[k]);
}

// Gradients.  dpre = dy silu'(pre), dx[r] = sum_k w[k] dpre[r + W - 1 - k], dw[k] = sum_t dpre[t] x[t - W + 1 + k].
// A thread has 4 channels and keeps their sums of dw and dbias over the strips that it takes: strip by strip of all sequences
// in turn, `2^l` pieces of channels by kBackThreads >> l strips at a time.
// Four CTAs an SM: three leave loads unhidden (169 us for 149 both ways), five spill (208).
template <typename IO, int W, bool SILU, bool SPARSE>
__global__ void __launch_bounds__(kBackThreads, 4) conv_bwd_kernel(const ConvArgs a, int l)
{
    __shared__ float4 share[kBackThreads];
    using Ring = Rows4<IO, kBackThreads>;
    __shared__ Ring rx, ry;
    const int D = a.s.D, tx = threadIdx.x & ((1 << l) - 1), ty = threadIdx.x >> l, strips = kBackThreads >> l;
    const int c = 4 * ((blockIdx.x << l) + tx);
    const int each = a.s.T > 0 ? (a.s.T + kBackStrip - 1) / kBackStrip : 1;      // strips of a sequence
    const long long items = SPARSE ? places(a.s.B, a.s.rows, kBackStrip) : (long long)a.s.B * each;
    Four taps[W], bias = all(0.f), dw[W], db = all(0.f);
#pragma unroll
    for (int k = 0; k < W; k++) taps[k] = dw[k] = all(0.f);
    if (c < D) {
        load_taps<W>(a.w + (long long)c * W, taps);
        if (a.bias) bias = raw4(a.bias + c).get();
    }
    for (long long item = (long long)blockIdx.y * strips + ty; item < items && c < D; item += (long long)gridDim.y * strips) {
        int b = (int)(item / each), strip = (int)(item - (long long)b * each);
        if (SPARSE) {
            const Place p = place_of(a.cu, a.s.B, a.s.rows, kBackStrip, (int)item);
            b = p.b;
            strip = p.piece;
        }
        const Rows r = rows_of(a.cu, b, a.s.T, a.s.rows);
        if (strip > 0 && (long long)strip * kBackStrip >= r.n) continue;
        const int t0 = strip * kBackStrip;
        const int end = min(r.n, t0 + kBackStrip), from = t0 == 0 && a.ds0 ? -(W - 1) : t0;      // rows whose gradients it writes
        const IO* x = (const IO*)a.x.p + (long long)r.first * a.x.tok + c;
        const IO* dy = (const IO*)a.dy.p + (long long)r.first * a.dy.tok + c;
        IO* dx = (IO*)a.dx.p + (long long)r.first * a.dx.tok + c;
        Four ring[4], d[4];                          // rows of x and of dpre, by their number modulo 4
        const int seen = min(r.n, end + W - 1);      // rows that it reads end here
        auto ask = [&](int t) {
            rx.ask(x, a.x.tok, t, seen);
            ry.ask(dy, a.dy.tok, t, seen);
            rec::cp_async_commit();
        };
        auto pre = [&](int t, int j) {               // d[j] of a row of the sequence
            ring[j] = rx.get(t, j).get();
            d[j] = ry.get(t, j).get();
            if (!SILU) return;
            Four p = bias;
#pragma unroll
            for (int k = 0; k < W; k++) p = fma(taps[k], ring[(j + 5 - W + k) & 3], p);
            const Four s = sigmoid4(p);
            d[j] = mul(d[j], mul(s, fma(p, fma(s, all(-1.f), all(1.f)), all(1.f))));
        };
        auto own = [&](int j) {                      // a row of the strip's own goes into the sums
            db = add(db, d[j]);
#pragma unroll
            for (int k = 0; k < W; k++) dw[k] = fma(d[j], ring[(j + 5 - W + k) & 3], dw[k]);
        };
        auto gradient = [&](int j) {                 // of row t + j - (W - 1): all rows that see it are done
            Four o = mul(taps[0], d[j]);
#pragma unroll
            for (int k = 1; k < W; k++) o = fma(taps[k], d[(j + 4 - k) & 3], o);
            return o;
        };
        auto edge = [&](int t) {                     // rows t .. t + 3 at an end of the strip, whatever holds of them
            Ring::arrived();
            ask(t + 4 * (Ring::GROUPS - 1));
#pragma unroll
            for (int j = 0; j < 4; j++) {
                if (t + j >= end + W - 1) break;
                d[j] = all(0.f);
                if (t + j < r.n) {
                    pre(t, j);
                    if (t + j < end) own(j);
                }
                const int row = t + j - (W - 1), kept = row - (r.n - (W - 1));      // kept: its place in the new state
                if (row < from) continue;
                Four o = gradient(j);
                if (a.dsT && kept >= 0) o = add(o, raw4((const IO*)a.dsT + ((long long)b * (W - 1) + kept) * D + c).get());
                if (row >= 0) put(dx + (long long)row * a.dx.tok, o);
                else put((IO*)a.ds0 + ((long long)b * (W - 1) + row + W - 1) * D + c, o);
            }
        };
        rec::cp_async_wait_all();                    // of the last strip
#pragma unroll
        for (int g = 0; g < Ring::GROUPS - 1; g++) ask(t0 + 4 * g);
        load_past<IO, W>(x, a.x.tok, a.s0, b, D, c, t0, ring);
#pragma unroll
        for (int k = 0; k < 4; k++) d[k] = all(0.f);
        edge(t0);
        int t = t0 + 4;
        for (; t + 4 <= end; t += 4) {               // rows within the strip, which end before the sequence does
            Ring::arrived();
            ask(t + 4 * (Ring::GROUPS - 1));
#pragma unroll
            for (int j = 0; j < 4; j++) {
                pre(t, j);
                own(j);
                put(dx + (long long)(t + j - (W - 1)) * a.dx.tok, gradient(j));
            }
        }
        for (; t < end + W - 1; t += 4) edge(t);
    }
    // the strips' sums in their order
    float* out = a.partial + (long long)blockIdx.y * D * (W + 1);
#pragma unroll
    for (int k = 0; k <= W; k++) {
        const Four s = k < W ? dw[k < W ? k : 0] : db;
        __syncthreads();
        share[threadIdx.x] = make_float4(s.a.x, s.a.y, s.b.x, s.b.y);
        __syncthreads();
        if (ty == 0 && c < D) {
            float4 x = share[tx];
            for (int i = 1; i < strips; i++) {
                const float4 y = share[tx + (i << l)];
                x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
            }
            if (k < W) {
                out[(long long)c * W + k] = x.x;
                out[(long long)(c + 1) * W + k] = x.y;
                out[(long long)(c + 2) * W + k] = x.z;
                out[(long long)(c + 3) * W + k] = x.w;
            } else {
                *reinterpret_cast<float4*>(out + (long long)D * W + c) = x;
            }
        }
    }
}

// pieces of 4 channels a block takes side by side, as a power of two
int back_pieces(const gdn_conv_t& s)
{
    int l = 1;
    while (l < 5 && (4 << l) < s.D) l++;
    return l;
}

template <typename IO, int W>
cudaError_t launch_fwd_w(const ConvArgs& a, cudaStream_t st)
{
    const bool sp = sparse(a.s.B, a.s.T, a.s.rows);
    const long long strips = sp ? places(a.s.B, a.s.rows, kStrip) : (a.s.T + kStrip - 1) / kStrip;
    const long long units = (strips > 0 ? strips : 1) * (a.s.D >> 2);
    const dim3 grid((unsigned)((units + kThreads - 1) / kThreads), sp ? 1 : a.s.B);
    if (sp && a.s.silu) conv_kernel<IO, W, true, true><<<grid, kThreads, 0, st>>>(a);
    else if (sp) conv_kernel<IO, W, false, true><<<grid, kThreads, 0, st>>>(a);
    else if (a.s.silu) conv_kernel<IO, W, true, false><<<grid, kThreads, 0, st>>>(a);
    else conv_kernel<IO, W, false, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename IO, int W>
cudaError_t launch_step_w(const ConvStepArgs& a, cudaStream_t st)
{
    const long long units = (long long)a.s.B * (a.s.D >> 3);
    conv_step_kernel<IO, W><<<(unsigned)((units + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename IO, int W>
cudaError_t launch_bwd_w(const ConvArgs& a, cudaStream_t st)
{
    const int l = back_pieces(a.s), wide = ((a.s.D >> 2) + (1 << l) - 1) >> l;
    const dim3 grid(wide, conv_bwd_blocks(a.s));
    const bool sp = sparse(a.s.B, a.s.T, a.s.rows);
    if (sp && a.s.silu) conv_bwd_kernel<IO, W, true, true><<<grid, kBackThreads, 0, st>>>(a, l);
    else if (sp) conv_bwd_kernel<IO, W, false, true><<<grid, kBackThreads, 0, st>>>(a, l);
    else if (a.s.silu) conv_bwd_kernel<IO, W, true, false><<<grid, kBackThreads, 0, st>>>(a, l);
    else conv_bwd_kernel<IO, W, false, false><<<grid, kBackThreads, 0, st>>>(a, l);
    return cudaGetLastError();
}

#define GDN_BY_TYPE(fn, a, st)                                                                                        \
    ((a).s.io == GDN_BF16 ? ((a).s.W == 2   ? fn<__nv_bfloat16, 2>(a, st)                                             \
                             : (a).s.W == 3 ? fn<__nv_bfloat16, 3>(a, st)                                             \
                                            : fn<__nv_bfloat16, 4>(a, st))                                            \
                          : ((a).s.W == 2   ? fn<float, 2>(a, st)                                                     \
                             : (a).s.W == 3 ? fn<float, 3>(a, st)                                                     \
                                            : fn<float, 4>(a, st)))

}  // namespace

// blocks that share the strips of a block's channels, each with its row of shares of dw and dbias
int conv_bwd_blocks(const gdn_conv_t& s)
{
    const int l = back_pieces(s), wide = ((s.D >> 2) + (1 << l) - 1) >> l, strips = kBackThreads >> l;
    const int T = s.T < s.rows ? s.T : s.rows;      // as the launch has it: a T past the rows is no bound
    const long long each = T > 0 ? (T + kBackStrip - 1) / kBackStrip : 1, items = (long long)s.B * each;
    const long long need = (items + strips - 1) / strips, most = 152 * 32 / wide;
    return need < most ? (int)need : most < 1 ? 1 : (int)most;
}

cudaError_t launch_conv(const ConvArgs& a, cudaStream_t st) { return GDN_BY_TYPE(launch_fwd_w, a, st); }
cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t st) { return GDN_BY_TYPE(launch_step_w, a, st); }
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t st)
{
    const cudaError_t e = GDN_BY_TYPE(launch_bwd_w, a, st);
    if (e != cudaSuccess) return e;
    ColumnSums c = {};
    c.partial = a.partial;
    c.rows = conv_bwd_blocks(a.s);
    c.cols = (long long)a.s.D * (a.s.W + 1);
    c.a = (long long)a.s.D * a.s.W;
    c.b = a.s.D;
    c.out_a = a.dw;
    c.out_b = a.dbias;
    return launch_column_sums(c, st);
}

}  // namespace ssm
}  // namespace gdn
