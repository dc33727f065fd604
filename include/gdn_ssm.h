/*
 * gdn_ssm.h -- a selective state-space layer between its projections: the token mixer of hybrids whose layers have a
 * decay for every channel and state, next to gdn.h's recurrence (a matrix state a head) and gdn_mla.h's attention.
 *
 * Three operators, the projections around them being plain matrix products of the caller:
 *
 *   gdn_norm_fwd / gdn_norm_bwd                    addition to the residual stream and RMS norm, the result in the I/O
 *                                                  type or in 8 bits with scales
 *   gdn_conv_fwd / gdn_conv_bwd / gdn_conv_step    short causal convolution of each channel (in front of the scan, or of
 *                                                  the delta rule's v, b, c), whole sequences or new tokens
 *   gdn_scan_fwd / gdn_scan_bwd / gdn_scan_step    the selective scan with step sizes, skip and gate, likewise
 *
 * Conventions are those of gdn.h and gdn_mla.h: the caller owns every buffer and the workspace (device memory, 256-byte
 * aligned); nothing is allocated and nothing synchronises; work goes to the caller's stream; argument errors are
 * reported before anything is enqueued.  The kernels wait on nothing but their own launches, so no status is read back.
 * Calls that may overlap on the GPU need workspaces of their own.
 * io is gdn_dtype_t: GDN_BF16 or GDN_F32; all arithmetic, statistics, sums and states are fp32 and each result is
 * rounded once.  Every pointer to io-typed data, states and weights is 16-byte aligned, every width a multiple of 8, every
 * stride a multiple of 8 elements (bf16) or 4 (f32); int32 arrays are 4-byte aligned.  Outputs must not alias
 * inputs, except where a comment allows it.  Every sum runs in a fixed order: the same call gives the same bits.
 *
 * Sequences of the convolution and the scan: cu NULL: sequence b holds rows b * T .. of the tensors; else int32 [B + 1]
 * row offsets on the device, ascending, with sequences of at most T rows (longer ones are cut there, offsets outside
 * [0, rows] are taken as the nearer bound); T = rows will do where the longest is not known.  Rows of no sequence are
 * neither read into a result nor written.  Values in one sequence never reach another's rows or states, NaN and Inf
 * included; the gradients of weights are sums over all.
 */
#ifndef GDN_SSM_H
#define GDN_SSM_H

#include "gdn_mla.h"      /* gdn_mla_view_t: address, row stride, head stride (ignored for one head) */

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- residual addition and RMS norm
 *
 *   sum[n] = x[n] + res[n]  (rounded to the residual's type),   y[n] = sum[n] / sqrt(mean(sum[n]^2) + eps) * w
 *
 * out = io: y is of the I/O type.  out = GDN_E4M3: y holds 8-bit values and scale one fp32 number for each `group` values
 * of a row (group = 0: for the whole row), y[n, i] ~ value * scale with scale = max(max |y| over the group, 1e-30) / 448
 * and value = y / scale rounded to nearest even.  A NaN in a row gives NaN for its values and scales;
 * a finite row whose sum of squares passes fp32 (values of 1e19 and more) gives zeros.
 * Limits: 0 <= N <= 2^30, 8 <= D <= 16384 a multiple of 8, group 0, 32, 64 or 128 and a divisor of D. */
#define GDN_E4M3 2        /* value of gdn_norm_t.out beside gdn_dtype_t's */

typedef struct {
    int N, D;             /* rows, width                                       */
    int io;               /* gdn_dtype_t of x, dy, dx (and of y, if out == io) */
    int res;              /* gdn_dtype_t of the residual stream: res, sum, dsum, dres; GDN_F32 or io */
    int out;              /* io or GDN_E4M3                                    */
    int group;            /* values a scale covers, 0: a row                   */
    float eps;
} gdn_norm_t;

/* x, res, y, sum: rows of D values at their row strides (elements).  res NULL: nothing is added (sum = x).  sum NULL: not
 * kept; it may be the very same rows as res.  scale [N, D / group] fp32 (NULL iff out == io).  w [D] fp32. */
gdn_status_t gdn_norm_fwd(const gdn_norm_t* shape, const void* x, long long x_tok, const void* res, long long res_tok,
                          const float* w, void* y, long long y_tok, float* scale, void* sum, long long sum_tok,
                          gdn_stream_t stream);

/* Gradients, with the norm taken as if unrounded (an 8-bit out counts as its value): the gradient of sum is the
 * norm's plus dsum (NULL: nothing), written to dx in the I/O type and to dres in the residual's (each may be NULL);
 * dw [D] fp32 is overwritten.  sum is the forward's (of type res).  dres, or dx where io == res, may be the very same
 * rows as dsum. */
size_t gdn_norm_workspace_bytes(const gdn_norm_t* shape);
gdn_status_t gdn_norm_bwd(const gdn_norm_t* shape, const void* sum, long long sum_tok, const float* w, const void* dy,
                          long long dy_tok, const void* dsum, long long dsum_tok, void* dx, long long dx_tok, void* dres,
                          long long dres_tok, float* dw, void* ws, size_t ws_bytes, gdn_stream_t stream);

/* ---------------------------------------------------------------- short causal convolution
 *
 *   pre[t, d] = bias[d] + sum_{k < W} w[d, k] x[t - (W - 1) + k, d],     y = silu ? pre / (1 + exp(-pre)) : pre
 *
 * within each sequence; the rows before its first are those of its state [W - 1, D] (NULL: zeros), and its new state is
 * the last W - 1 rows of state and sequence together.  Limits: 2 <= W <= 4, B >= 1,
 * T >= 1 where rows > 0, B <= 65535, rows <= 2^30, D a multiple of 8 up to 2^24. */
typedef struct {
    int B, T, D, W;       /* sequences, most rows of one, channels, taps       */
    int silu;
    int io;               /* gdn_dtype_t of x, states, y and their gradients   */
    int rows;             /* rows of the tensors (B * T without cu)            */
} gdn_conv_t;

/* x, y [rows, D] views; w [D, W], bias [D] fp32 (NULL: none); s0, sT [B, W - 1, D] (NULL: zeros; not written), which may
 * not overlap. */
gdn_status_t gdn_conv_fwd(const gdn_conv_t* shape, const gdn_mla_view_t* x, const float* w, const float* bias,
                          const int* cu, const void* s0, const gdn_mla_view_t* y, void* sT, gdn_stream_t stream);

/* Gradients from dy and dsT (NULL: zeros): dx, ds0 (NULL: not written), dw, dbias (NULL iff bias is) overwritten. */
size_t gdn_conv_workspace_bytes(const gdn_conv_t* shape);
gdn_status_t gdn_conv_bwd(const gdn_conv_t* shape, const gdn_mla_view_t* x, const float* w, const float* bias,
                          const int* cu, const void* s0, const gdn_mla_view_t* dy, const void* dsT,
                          const gdn_mla_view_t* dx, float* dw, float* dbias, void* ds0, void* ws, size_t ws_bytes,
                          gdn_stream_t stream);

/* T new tokens (1..8) of each of B sequences: rows b * T .. of x and y.  The state of sequence b is read from slot src[b]
 * of state [slots, W - 1, D] and written to slot dst[b] (dst NULL: to src[b]; src NULL: slot b, slots >= B).  A src outside
 * [0, slots) reads zeros (a sequence that begins), a dst outside is not written (a place of the batch without a request).
 * A slot that one sequence writes no other one reads or writes. */
typedef struct {
    int B, T, D, W;
    int silu;
    int io;
    int slots;
} gdn_conv_step_t;
gdn_status_t gdn_conv_step(const gdn_conv_step_t* shape, const gdn_mla_view_t* x, const float* w, const float* bias,
                           void* state, const int* src, const int* dst, const gdn_mla_view_t* y, gdn_stream_t stream);

/* ---------------------------------------------------------------- selective scan
 *
 *   delta[t, d] = softplus(dt[t, d] + dt_bias[d])     (without `softplus`: the sum itself)
 *   h[t, d, n]  = exp(-delta[t, d] exp(A_log[d, n])) h[t - 1, d, n] + delta[t, d] x[t, d] Bm[t, g, n]
 *   y[t, d]     = (sum_n h[t, d, n] Cm[t, g, n] + D[d] x[t, d]) * silu(z[t, d]),        g = d / (D / G)
 *
 * within each sequence, from its state h0 [D, N] (zeros without).  delta is meant to be >= 0 (without softplus a negative
 * one grows the state); an exp(A_log) past fp32 counts as its largest value.  Limits: N a multiple of 8 up to 64, D a
 * multiple of 8 G, B, G >= 1, T >= 1 where rows > 0, B, G <= 65535, rows <= 2^30, B * D * N and D (N + 2) < 2^31. */
typedef struct {
    int B, T, D, N, G;    /* sequences, most rows of one, channels, states a channel, groups that share Bm and Cm */
    int softplus;
    int io;               /* gdn_dtype_t of x, dt, z, Bm, Cm, y and their gradients */
    int rows;             /* rows of the tensors (B * T without cu)            */
} gdn_scan_t;

/* Workspace of gdn_scan_fwd (backward = 0) or gdn_scan_bwd (1); the bytes of `saved`.  0 if the shape is invalid.  The
 * workspace of gdn_scan_bwd serves gdn_scan_fwd of the same shape too.  (Not ascending with the shape: fewer sequences may
 * be split into more segments.)  The gradients' one holds shares of dA_log, dD and ddt_bias, D (N + 2) fp32 for each sequence
 * however short it is: 65535 sequences of 2 rows of 1024 channels with 16 states ask for 5.1 GB, 4096 of 16 rows for 0.44 GB. */
size_t gdn_scan_workspace_bytes(const gdn_scan_t* shape, int backward);
size_t gdn_scan_saved_bytes(const gdn_scan_t* shape);

/* x, dt, z, y [rows, D] views (z NULL: no gate); Bm, Cm [rows, G, N] views; A_log [D, N], D_skip [D] (NULL: none),
 * dt_bias [D] (NULL: none) fp32; h0, hT [B, D, N] fp32 (NULL: zeros; not written), which may not overlap.  saved: the
 * states that gdn_scan_bwd starts its pieces from (256-byte aligned; NULL: not kept). */
gdn_status_t gdn_scan_fwd(const gdn_scan_t* shape, const gdn_mla_view_t* x, const gdn_mla_view_t* dt,
                          const gdn_mla_view_t* z, const gdn_mla_view_t* Bm, const gdn_mla_view_t* Cm,
                          const float* A_log, const float* D_skip, const float* dt_bias, const int* cu,
                          const float* h0, const gdn_mla_view_t* y, float* hT, void* saved, size_t saved_bytes, void* ws,
                          size_t ws_bytes, gdn_stream_t stream);

/* (A sum over channels in dBm or dCm of which a term is infinite is infinite or a NaN; other tokens' sums keep their values.)
 * Gradients from dy, dhT (NULL: zeros) and the forward's saved: dx, ddt, dz (NULL iff z is) views as their inputs, dBm,
 * dCm views; dA_log, dD_skip and ddt_bias (NULL iff theirs are) overwritten; dh0 (NULL: not written). */
gdn_status_t gdn_scan_bwd(const gdn_scan_t* shape, const gdn_mla_view_t* x, const gdn_mla_view_t* dt,
                          const gdn_mla_view_t* z, const gdn_mla_view_t* Bm, const gdn_mla_view_t* Cm,
                          const float* A_log, const float* D_skip, const float* dt_bias, const int* cu,
                          const void* saved, size_t saved_bytes, const gdn_mla_view_t* dy, const float* dhT,
                          const gdn_mla_view_t* dx, const gdn_mla_view_t* ddt, const gdn_mla_view_t* dz,
                          const gdn_mla_view_t* dBm, const gdn_mla_view_t* dCm, float* dA_log, float* dD_skip,
                          float* ddt_bias, float* dh0, void* ws, size_t ws_bytes, gdn_stream_t stream);

/* T new tokens (1..8) of each of B sequences, their states in slots of state [slots, D, N] fp32, as gdn_conv_step. */
typedef struct {
    int B, T, D, N, G;
    int softplus;
    int io;
    int slots;
} gdn_scan_step_t;
gdn_status_t gdn_scan_step(const gdn_scan_step_t* shape, const gdn_mla_view_t* x, const gdn_mla_view_t* dt,
                           const gdn_mla_view_t* z, const gdn_mla_view_t* Bm, const gdn_mla_view_t* Cm,
                           const float* A_log, const float* D_skip, const float* dt_bias, float* state, const int* src,
                           const int* dst, const gdn_mla_view_t* y, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_SSM_H */
