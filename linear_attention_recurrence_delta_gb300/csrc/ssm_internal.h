// ssm_internal.h -- what the translation units of the state-space operators share (not part of the ABI).
#pragma once

#include "../../include/gdn_ssm.h"
#include "mla_internal.h"

namespace gdn {
namespace ssm {

using mla::Raw8;
using mla::Rows;

struct NormArgs {
    gdn_norm_t s;
    const void *x, *res;      // x is the forward's input; the backward's `sum` arrives in res
    const float* w;
    void *y, *sum;
    float* scale;
    const void *dy, *dsum;
    void *dx, *dres;
    float *dw, *partial;      // partial [norm_bwd_blocks][D]
    long long x_tok, res_tok, y_tok, sum_tok, dy_tok, dsum_tok, dx_tok, dres_tok;
};

struct ConvArgs {
    gdn_conv_t s;
    gdn_mla_view_t x, y, dy, dx;
    const float *w, *bias;
    const int* cu;
    const void *s0, *dsT;
    void *sT, *ds0;
    float *dw, *dbias, *partial;   // partial [conv_bwd_blocks][D (W + 1)]
};

struct ConvStepArgs {
    gdn_conv_step_t s;
    gdn_mla_view_t x, y;
    const float *w, *bias;
    void* state;
    const int *src, *dst;
};

struct ScanArgs {
    gdn_scan_t s;
    gdn_mla_view_t x, dt, z, Bm, Cm, y, dy, dx, ddt, dz, dBm, dCm;
    const float *A_log, *D_skip, *dt_bias, *h0, *dhT;
    const int* cu;
    float *hT, *dh0, *dA_log, *dD_skip, *ddt_bias;
    float* saved;             // states entering every kSaveEvery tokens, [rows / kSaveEvery + B + 1][blocks]
    float* wpart;             // backward: [shares][D (N + 2)] of dA_log, dD_skip, ddt_bias
    float* bcpart;            // backward: [CTAs of a group][rows][G][2 N] shares of dBm, dCm
    float *seg_h, *seg_d;     // split in time: states from zero and sums of delta, [places][blocks]
    int ctas, blocks;         // CTAs that a group's channels need, and warps' blocks of channels
    int saved_blocks;         // the forward's blocks
    int segments, seg_len;    // segments a sequence is cut into, tokens of one (a multiple of the tile)
    int shares;               // rows of wpart
    bool sparse;              // segments are dealt by places
};

struct ScanStepArgs {
    gdn_scan_step_t s;
    gdn_mla_view_t x, dt, z, Bm, Cm, y;
    const float *A_log, *D_skip, *dt_bias;
    float* state;
    const int *src, *dst;
};

int norm_bwd_blocks(const gdn_norm_t& s);
int conv_bwd_blocks(const gdn_conv_t& s);

constexpr int kSaveEvery = 8;     // tokens between the states that a training forward keeps

// Work over packed sequences is dealt as B x T rows, most of which is nobody's where one sequence is far longer than the
// average or T is only a bound.  There it is dealt by places instead: piece i of L rows of sequence b has place cu[b] / L + b + i,
// which no other sequence's piece has, `places` in all, and who works at a place looks up whose it is.  16384 rows of 2048 channels with
// T = 16384, us by places and as B x T rows (16 states; the sequences equal, but for the last two batches):
//   sequences             2          5          8         16         32        128        512     9 uneven   30 uneven
//   convolution                         31    37                                       36   495
//   its gradients                       58    82                                       75   379
//   scan           291  289   301  283   298  271   304  295   277  380   210  946   246 3333   306  322   313  406
//   its gradients  886  867   939 1055   801  702   748  757   677  704   681  881   815 1651   919  886   829  831
// So by places from over four times the rows on, where most of B x T is nobody's.  Up to 16 sequences either way of the scan is
// faster by up to 14 %, as sequences and segments happen to fall to the SMs, and no ratio parts them; by places its workspace does not
// grow with what T allows.
inline bool sparse(int B, int T, int rows) { return (long long)B * (T < rows ? T : rows) > 4LL * rows; }
__host__ __device__ inline int places(int B, int rows, int L) { return rows / L + B; }

// How a scan's call is laid out: CTAs and warps' blocks of channels of a group, segments of time, workspace.
struct ScanPlan {
    int ctas, blocks;
    int segments, seg_len, shares;
    size_t h_off, d_off, w_off, bc_off, total;
};
constexpr int kBackWarps = 4;     // warps of a CTA of the backward scan
inline int fwd_channels(int N) { return N <= 16 ? 32 : N <= 32 ? 16 : 8; }      // that a warp takes forwards
inline int back_channels(int N) { return N <= 8 ? 32 : N <= 16 ? 16 : 8; }      // and backwards
ScanPlan scan_plan(const gdn_scan_t& s, int backward);
inline int state_values(int N) { return N <= 8 ? 8 : N <= 16 ? 16 : N <= 32 ? 32 : 64; }      // places of a channel's states
inline int saved_blocks_of(const gdn_scan_t& s) { return (s.D / s.G + fwd_channels(s.N) - 1) / fwd_channels(s.N); }
inline size_t saved_bytes_of(const gdn_scan_t& s)
{
    return ((size_t)(s.rows / kSaveEvery) + s.B + 1) * s.G * saved_blocks_of(s) * fwd_channels(s.N) * state_values(s.N) * 4;
}

cudaError_t launch_norm(const NormArgs& a, cudaStream_t st);
cudaError_t launch_norm_bwd(const NormArgs& a, cudaStream_t st);
cudaError_t launch_conv(const ConvArgs& a, cudaStream_t st);
cudaError_t launch_conv_bwd(const ConvArgs& a, cudaStream_t st);
cudaError_t launch_conv_step(const ConvStepArgs& a, cudaStream_t st);
cudaError_t launch_scan(const ScanArgs& a, cudaStream_t st);
cudaError_t launch_scan_bwd(const ScanArgs& a, cudaStream_t st);
cudaError_t launch_scan_step(const ScanStepArgs& a, cudaStream_t st);

// Launches a kernel as the dependent of the one in front of it, which lets it start as soon as its own blocks have all begun
// (or ended): it waits in cudaGridDependencySynchronize for what that one writes, and every block of it does so before it ends,
// so that what follows in the stream finds both done.
template <typename Args>
cudaError_t launch_after(void (*kernel)(Args), dim3 grid, int threads, size_t smem, cudaStream_t st, const Args& args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args);
}

// Sums over the rows of partial [rows][cols], in a fixed order: the first `a` columns go to out_a, the next `b` to out_b,
// the rest to out_c (NULL: dropped).
struct ColumnSums {
    const float* partial;
    int rows;
    long long cols, a, b;
    float *out_a, *out_b, *out_c;
    const float* decay;       // A_log: out_a's sums are multiplied by -exp of it, at most fp32's largest value (NULL: as they are)
};
cudaError_t launch_column_sums(const ColumnSums& c, cudaStream_t st);

}  // namespace ssm
}  // namespace gdn
