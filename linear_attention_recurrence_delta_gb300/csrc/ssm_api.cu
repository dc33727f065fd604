// ssm_api.cu -- the C ABI of the state-space operators: argument checks, workspace carve-up, dispatch.
#include <algorithm>

#include "ssm_internal.h"

using namespace gdn;
using namespace gdn::ssm;
using mla::aligned;
using mla::io_ok;
using mla::round_up;
using mla::take;

namespace {

// rows of D values at a stride: present, 16-byte aligned, long enough
gdn_status_t rows_ok(const void* p, long long tok, int D, int type)
{
    if (!p) return GDN_ERR_NULL;
    if (tok < D || tok >= (1LL << 38)) return GDN_ERR_SHAPE;
    return aligned(p, 16) && tok % (type == GDN_F32 ? 4 : 8) == 0 ? GDN_OK : GDN_ERR_ALIGN;
}

#define GDN_TRY(call)                          \
    do {                                       \
        const gdn_status_t r_ = (call);        \
        if (r_ != GDN_OK) return r_;           \
    } while (0)

constexpr int kMostRows = 1 << 30;      // so that a row's number and a tile more stay in 32 bits

gdn_status_t norm_check(const gdn_norm_t* s)
{
    if (!s) return GDN_ERR_NULL;
    if (!io_ok(s->io) || (s->res != GDN_F32 && s->res != s->io) || (s->out != s->io && s->out != GDN_E4M3)) return GDN_ERR_MODE;
    if (s->N < 0 || s->N > kMostRows || s->D < 8 || s->D > 16384 || s->D % 8 || !(s->eps >= 0.f)) return GDN_ERR_SHAPE;
    if (s->group != 0 && s->group != 32 && s->group != 64 && s->group != 128) return GDN_ERR_SHAPE;
    return s->group && (s->D % s->group || s->out != GDN_E4M3) ? GDN_ERR_SHAPE : GDN_OK;
}

bool conv_ok(int B, int D, int W) { return B >= 1 && B <= 65535 && D >= 8 && D % 8 == 0 && D <= (1 << 24) && W >= 2 && W <= 4; }
bool scan_ok(int B, int D, int N, int G)
{
    return B >= 1 && B <= 65535 && N >= 8 && N <= 64 && N % 8 == 0 && G >= 1 && G <= 65535 && D >= 8 && D % (8LL * G) == 0 &&
           (double)B * D * N < 2147483648.0 && (double)D * (N + 2) < 2147483648.0;
}

gdn_status_t conv_check(const gdn_conv_t* s)
{
    if (!s) return GDN_ERR_NULL;
    if (!io_ok(s->io)) return GDN_ERR_MODE;
    if (!conv_ok(s->B, s->D, s->W) || s->T < 0 || s->rows < 0 || s->rows > kMostRows || (s->rows > 0 && s->T < 1)) return GDN_ERR_SHAPE;
    return GDN_OK;
}

gdn_status_t scan_check(const gdn_scan_t* s)
{
    if (!s) return GDN_ERR_NULL;
    if (!io_ok(s->io)) return GDN_ERR_MODE;
    if (!scan_ok(s->B, s->D, s->N, s->G) || s->T < 0 || s->rows < 0 || s->rows > kMostRows || (s->rows > 0 && s->T < 1)) return GDN_ERR_SHAPE;
    return GDN_OK;
}

// the sequences' offsets, or B sequences of T rows
gdn_status_t sequences(const int* cu, int B, int* T, int rows)
{
    if (!cu && (long long)B * *T != rows) return GDN_ERR_SHAPE;
    if (!aligned(cu, 4)) return GDN_ERR_ALIGN;
    if (*T > rows) *T = rows;
    return GDN_OK;
}

gdn_status_t weight(const void* p, bool wanted)
{
    if (wanted && !p) return GDN_ERR_NULL;
    return aligned(p, 16) ? GDN_OK : GDN_ERR_ALIGN;
}

gdn_status_t workspace(const void* ws, size_t have, size_t need)
{
    if (!ws || have < need) return GDN_ERR_WORKSPACE;
    return aligned(ws, 256) ? GDN_OK : GDN_ERR_ALIGN;
}

gdn_status_t done(cudaError_t e) { return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }

// the views that both directions of a scan take
gdn_status_t scan_inputs(const gdn_scan_t* s, const gdn_mla_view_t* x, const gdn_mla_view_t* dt, const gdn_mla_view_t* z,
                         const gdn_mla_view_t* Bm, const gdn_mla_view_t* Cm, const float* A_log, const float* D_skip,
                         const float* dt_bias, const int* cu, ScanArgs* a)
{
    GDN_TRY(scan_check(s));
    memset(a, 0, sizeof(*a));
    a->s = *s;
    GDN_TRY(sequences(cu, s->B, &a->s.T, s->rows));
    const bool any = s->rows > 0;
    GDN_TRY(take(x, any, 1, s->io, &a->x));
    GDN_TRY(take(dt, any, 1, s->io, &a->dt));
    GDN_TRY(take(z, any && z, 1, s->io, &a->z));
    GDN_TRY(take(Bm, any, s->G, s->io, &a->Bm));
    GDN_TRY(take(Cm, any, s->G, s->io, &a->Cm));
    GDN_TRY(weight(A_log, true));
    GDN_TRY(weight(D_skip, false));
    GDN_TRY(weight(dt_bias, false));
    a->A_log = A_log; a->D_skip = D_skip; a->dt_bias = dt_bias; a->cu = cu;
    return GDN_OK;
}

void scan_layout(const ScanPlan& p, void* ws, ScanArgs* a)
{
    unsigned char* w = (unsigned char*)ws;
    a->ctas = p.ctas;
    a->blocks = p.blocks;
    a->saved_blocks = saved_blocks_of(a->s);
    a->segments = p.segments;
    a->seg_len = p.seg_len;
    a->shares = p.shares;
    a->sparse = sparse(a->s.B, a->s.T, a->s.rows);
    a->seg_h = (float*)(w + p.h_off);
    a->seg_d = (float*)(w + p.d_off);
    a->wpart = (float*)(w + p.w_off);
    a->bcpart = (float*)(w + p.bc_off);
}

}  // namespace

namespace gdn {
namespace ssm {

ScanPlan scan_plan(const gdn_scan_t& s, int backward)
{
    ScanPlan p;
    const int each = s.D / s.G, ch = backward ? back_channels(s.N) : fwd_channels(s.N), cta = backward ? kBackWarps * ch : ch;
    p.blocks = (each + ch - 1) / ch;
    p.ctas = (each + cta - 1) / cta;
    const long long T = s.T < s.rows ? s.T : s.rows;
    // Segments: as many as keep the SMs in warps, counted by the sequences that run at once on average.  Forwards (up to 16 warps an
    // SM) the first launch takes three fifths of the second: 9 prompts up to 1500 tokens take 213 us whole and 135 in 16
    // segments, which are two rounds of warps (one round, 8: 141; three, 24: 140), 8 x 2048 of 2048 channels 301 and 260 in 9
    // (4, one round five sixths full: 300).  One round where equal sequences fill it and it is of 15 segments or more (us of a call by
    // itself: 16001 tokens of 1536 channels 220 in 50 segments and 233 in 64, 2207 whole; 8 x 2048 of 608 channels 100 in 16 and
    // 105 in 32; 2 x 4096 of 2560 channels 192 in 15 and 194 in 30); of fewer it is slower (4096 tokens of 6208 channels 230 in 12 and 225
    // in 25, of 9376 331 in 8 and 318 in 16; 4 x 2048 of 4864 329 in 4 and 300 in 8).  Backwards (8 warps an SM by their
    // registers) only where few warps would run: 8 x 2048 tokens take 1009 us whole and 1170 in 3 segments, 2 x 333 of 208 channels
    // 145 and 82.
    const double each_round = T > 0 ? 152.0 * 16 * T / ((double)p.blocks * s.G * s.rows) : 1.0;      // segments in a round of 16 warps an SM
    long long seg = (long long)(each_round * (backward ? 0.5 : 2.0));
    if (!backward && (long long)s.B * T == s.rows && each_round >= 15.0 && (long long)each_round >= 0.95 * each_round) seg = (long long)each_round;
    if (seg > T / 32) seg = T / 32;
    if (seg > 64) seg = 64;
    if (seg < (backward ? 3 : 4)) seg = 1;
    p.seg_len = seg > 1 ? (int)(((T + seg - 1) / seg + kSaveEvery - 1) / kSaveEvery * kSaveEvery) : (T > 0 ? (int)((T + 31) / 32 * 32) : 32);
    p.segments = T > 0 ? (int)((T + p.seg_len - 1) / p.seg_len) : 1;
    p.shares = sparse(s.B, s.T, s.rows) ? places(s.B, s.rows, p.seg_len) : p.segments * s.B;
    const size_t kept = p.segments > 1 ? (size_t)places(s.B, s.rows, p.seg_len) * s.G * p.blocks : 0;
    p.h_off = 256;
    p.d_off = p.h_off + round_up(kept * ch * state_values(s.N) * 4, 256);
    p.w_off = p.d_off + round_up(kept * ch * 4, 256);
    p.bc_off = p.w_off + (backward ? round_up((size_t)p.shares * s.D * (s.N + 2) * 4, 256) : 0);
    p.total = p.bc_off + (backward ? round_up((size_t)p.ctas * s.rows * s.G * 2 * s.N * 4, 256) : 0);
    if (backward) p.total = std::max(p.total, scan_plan(s, 0).total);      // one area serves a training step's both calls
    return p;
}

}  // namespace ssm
}  // namespace gdn

extern "C" gdn_status_t gdn_norm_fwd(const gdn_norm_t* s, const void* x, long long x_tok, const void* res, long long res_tok,
                                     const float* w, void* y, long long y_tok, float* scale, void* sum, long long sum_tok,
                                     gdn_stream_t stream)
{
    GDN_TRY(norm_check(s));
    if (s->N == 0) return GDN_OK;
    GDN_TRY(rows_ok(x, x_tok, s->D, s->io));
    if (res) GDN_TRY(rows_ok(res, res_tok, s->D, s->res));
    GDN_TRY(rows_ok(y, y_tok, s->D, s->io));
    if (sum) GDN_TRY(rows_ok(sum, sum_tok, s->D, s->res));
    GDN_TRY(weight(w, true));
    if ((s->out == GDN_E4M3) != (scale != nullptr)) return scale ? GDN_ERR_MODE : GDN_ERR_NULL;
    if (!aligned(scale, 4) || (s->out == GDN_E4M3 && y_tok % 8)) return GDN_ERR_ALIGN;
    GDN_TRY(check_device());
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.s = *s;
    a.x = x; a.x_tok = x_tok; a.res = res; a.res_tok = res_tok; a.w = w; a.y = y; a.y_tok = y_tok;
    a.scale = scale; a.sum = sum; a.sum_tok = sum_tok;
    return done(launch_norm(a, (cudaStream_t)stream));
}

extern "C" size_t gdn_norm_workspace_bytes(const gdn_norm_t* s)
{
    return norm_check(s) != GDN_OK ? 0 : round_up(256 + (size_t)norm_bwd_blocks(*s) * s->D * 4, 256);
}

extern "C" gdn_status_t gdn_norm_bwd(const gdn_norm_t* s, const void* sum, long long sum_tok, const float* w, const void* dy,
                                     long long dy_tok, const void* dsum, long long dsum_tok, void* dx, long long dx_tok,
                                     void* dres, long long dres_tok, float* dw, void* ws, size_t ws_bytes, gdn_stream_t stream)
{
    GDN_TRY(norm_check(s));
    GDN_TRY(weight(w, true));
    if (!dw) return GDN_ERR_NULL;
    if (!aligned(dw, 4)) return GDN_ERR_ALIGN;
    if (s->N > 0) {
        GDN_TRY(rows_ok(sum, sum_tok, s->D, s->res));
        GDN_TRY(rows_ok(dy, dy_tok, s->D, s->io));
        if (dsum) GDN_TRY(rows_ok(dsum, dsum_tok, s->D, s->res));
        if (dx) GDN_TRY(rows_ok(dx, dx_tok, s->D, s->io));
        if (dres) GDN_TRY(rows_ok(dres, dres_tok, s->D, s->res));
    }
    GDN_TRY(workspace(ws, ws_bytes, gdn_norm_workspace_bytes(s)));
    GDN_TRY(check_device());
    NormArgs a;
    memset(&a, 0, sizeof(a));
    a.s = *s;
    a.res = sum; a.res_tok = sum_tok; a.w = w; a.dy = dy; a.dy_tok = dy_tok; a.dsum = dsum; a.dsum_tok = dsum_tok;
    a.dx = dx; a.dx_tok = dx_tok; a.dres = dres; a.dres_tok = dres_tok; a.dw = dw;
    a.partial = (float*)((unsigned char*)ws + 256);
    return done(launch_norm_bwd(a, (cudaStream_t)stream));
}

extern "C" gdn_status_t gdn_conv_fwd(const gdn_conv_t* s, const gdn_mla_view_t* x, const float* w, const float* bias, const int* cu,
                                     const void* s0, const gdn_mla_view_t* y, void* sT, gdn_stream_t stream)
{
    GDN_TRY(conv_check(s));
    ConvArgs a;
    memset(&a, 0, sizeof(a));
    a.s = *s;
    GDN_TRY(sequences(cu, s->B, &a.s.T, s->rows));
    GDN_TRY(take(x, s->rows > 0, 1, s->io, &a.x));
    GDN_TRY(take(y, s->rows > 0, 1, s->io, &a.y));
    GDN_TRY(weight(w, true));
    GDN_TRY(weight(bias, false));
    GDN_TRY(weight(s0, false));
    GDN_TRY(weight(sT, false));
    if (s->rows == 0 && !sT) return GDN_OK;
    GDN_TRY(check_device());
    a.w = w; a.bias = bias; a.cu = cu; a.s0 = s0; a.sT = sT;
    return done(launch_conv(a, (cudaStream_t)stream));
}

extern "C" size_t gdn_conv_workspace_bytes(const gdn_conv_t* s)
{
    return conv_check(s) != GDN_OK ? 0 : round_up(256 + (size_t)conv_bwd_blocks(*s) * s->D * (s->W + 1) * 4, 256);
}

extern "C" gdn_status_t gdn_conv_bwd(const gdn_conv_t* s, const gdn_mla_view_t* x, const float* w, const float* bias, const int* cu,
                                     const void* s0, const gdn_mla_view_t* dy, const void* dsT, const gdn_mla_view_t* dx, float* dw,
                                     float* dbias, void* ds0, void* ws, size_t ws_bytes, gdn_stream_t stream)
{
    GDN_TRY(conv_check(s));
    ConvArgs a;
    memset(&a, 0, sizeof(a));
    a.s = *s;
    GDN_TRY(sequences(cu, s->B, &a.s.T, s->rows));
    GDN_TRY(take(x, s->rows > 0, 1, s->io, &a.x));
    GDN_TRY(take(dy, s->rows > 0, 1, s->io, &a.dy));
    GDN_TRY(take(dx, s->rows > 0, 1, s->io, &a.dx));
    GDN_TRY(weight(w, true));
    GDN_TRY(weight(bias, false));
    GDN_TRY(weight(s0, false));
    GDN_TRY(weight(dsT, false));
    GDN_TRY(weight(ds0, false));
    if (!dw || (bias != nullptr) != (dbias != nullptr)) return GDN_ERR_NULL;
    if (!aligned(dw, 4) || !aligned(dbias, 4)) return GDN_ERR_ALIGN;
    GDN_TRY(workspace(ws, ws_bytes, gdn_conv_workspace_bytes(s)));
    GDN_TRY(check_device());
    a.w = w; a.bias = bias; a.cu = cu; a.s0 = s0; a.dsT = dsT; a.ds0 = ds0; a.dw = dw; a.dbias = dbias;
    a.partial = (float*)((unsigned char*)ws + 256);
    return done(launch_conv_bwd(a, (cudaStream_t)stream));
}

extern "C" gdn_status_t gdn_conv_step(const gdn_conv_step_t* s, const gdn_mla_view_t* x, const float* w, const float* bias, void* state,
                                      const int* src, const int* dst, const gdn_mla_view_t* y, gdn_stream_t stream)
{
    if (!s) return GDN_ERR_NULL;
    if (!io_ok(s->io)) return GDN_ERR_MODE;
    if (!conv_ok(s->B, s->D, s->W) || s->T < 1 || s->T > 8 || s->slots < 1 || (!src && s->slots < s->B)) return GDN_ERR_SHAPE;
    ConvStepArgs a;
    memset(&a, 0, sizeof(a));
    a.s = *s;
    GDN_TRY(take(x, true, 1, s->io, &a.x));
    GDN_TRY(take(y, true, 1, s->io, &a.y));
    GDN_TRY(weight(w, true));
    GDN_TRY(weight(bias, false));
    GDN_TRY(weight(state, true));
    if (!aligned(src, 4) || !aligned(dst, 4)) return GDN_ERR_ALIGN;
    GDN_TRY(check_device());
    a.w = w; a.bias = bias; a.state = state; a.src = src; a.dst = dst;
    return done(launch_conv_step(a, (cudaStream_t)stream));
}

extern "C" size_t gdn_scan_workspace_bytes(const gdn_scan_t* s, int backward)
{
    return scan_check(s) != GDN_OK ? 0 : scan_plan(*s, backward != 0).total;
}

extern "C" size_t gdn_scan_saved_bytes(const gdn_scan_t* s)
{
    return scan_check(s) != GDN_OK ? 0 : saved_bytes_of(*s);
}

extern "C" gdn_status_t gdn_scan_fwd(const gdn_scan_t* s, const gdn_mla_view_t* x, const gdn_mla_view_t* dt, const gdn_mla_view_t* z,
                                     const gdn_mla_view_t* Bm, const gdn_mla_view_t* Cm, const float* A_log, const float* D_skip,
                                     const float* dt_bias, const int* cu, const float* h0, const gdn_mla_view_t* y, float* hT,
                                     void* saved, size_t saved_bytes, void* ws, size_t ws_bytes, gdn_stream_t stream)
{
    ScanArgs a;
    GDN_TRY(scan_inputs(s, x, dt, z, Bm, Cm, A_log, D_skip, dt_bias, cu, &a));
    GDN_TRY(take(y, s->rows > 0, 1, s->io, &a.y));
    GDN_TRY(weight(h0, false));
    GDN_TRY(weight(hT, false));
    if (saved) GDN_TRY(workspace(saved, saved_bytes, gdn_scan_saved_bytes(s)));
    const ScanPlan p = scan_plan(*s, 0);
    GDN_TRY(workspace(ws, ws_bytes, p.total));
    if (s->rows == 0 && !hT) return GDN_OK;
    GDN_TRY(check_device());
    a.h0 = h0; a.hT = hT; a.saved = (float*)saved;
    scan_layout(p, ws, &a);
    return done(launch_scan(a, (cudaStream_t)stream));
}

extern "C" gdn_status_t gdn_scan_bwd(const gdn_scan_t* s, const gdn_mla_view_t* x, const gdn_mla_view_t* dt, const gdn_mla_view_t* z,
                                     const gdn_mla_view_t* Bm, const gdn_mla_view_t* Cm, const float* A_log, const float* D_skip,
                                     const float* dt_bias, const int* cu, const void* saved, size_t saved_bytes,
                                     const gdn_mla_view_t* dy, const float* dhT, const gdn_mla_view_t* dx, const gdn_mla_view_t* ddt,
                                     const gdn_mla_view_t* dz, const gdn_mla_view_t* dBm, const gdn_mla_view_t* dCm, float* dA_log,
                                     float* dD_skip, float* ddt_bias, float* dh0, void* ws, size_t ws_bytes, gdn_stream_t stream)
{
    ScanArgs a;
    GDN_TRY(scan_inputs(s, x, dt, z, Bm, Cm, A_log, D_skip, dt_bias, cu, &a));
    const bool any = s->rows > 0;
    GDN_TRY(take(dy, any, 1, s->io, &a.dy));
    GDN_TRY(take(dx, any, 1, s->io, &a.dx));
    GDN_TRY(take(ddt, any, 1, s->io, &a.ddt));
    GDN_TRY(take(dz, any && z, 1, s->io, &a.dz));
    GDN_TRY(take(dBm, any, s->G, s->io, &a.dBm));
    GDN_TRY(take(dCm, any, s->G, s->io, &a.dCm));
    GDN_TRY(weight(dhT, false));
    GDN_TRY(weight(dh0, false));
    if ((z != nullptr) != (dz != nullptr)) return GDN_ERR_NULL;
    if (!dA_log || (D_skip != nullptr) != (dD_skip != nullptr) || (dt_bias != nullptr) != (ddt_bias != nullptr)) return GDN_ERR_NULL;
    if (!aligned(dA_log, 4) || !aligned(dD_skip, 4) || !aligned(ddt_bias, 4)) return GDN_ERR_ALIGN;
    GDN_TRY(workspace(saved, saved_bytes, gdn_scan_saved_bytes(s)));
    const ScanPlan p = scan_plan(*s, 1);
    GDN_TRY(workspace(ws, ws_bytes, p.total));
    GDN_TRY(check_device());
    a.saved = (float*)const_cast<void*>(saved);
    a.dhT = dhT; a.dA_log = dA_log; a.dD_skip = dD_skip; a.ddt_bias = ddt_bias; a.dh0 = dh0;
    scan_layout(p, ws, &a);
    return done(launch_scan_bwd(a, (cudaStream_t)stream));
}

extern "C" gdn_status_t gdn_scan_step(const gdn_scan_step_t* s, const gdn_mla_view_t* x, const gdn_mla_view_t* dt,
                                      const gdn_mla_view_t* z, const gdn_mla_view_t* Bm, const gdn_mla_view_t* Cm, const float* A_log,
                                      const float* D_skip, const float* dt_bias, float* state, const int* src, const int* dst,
                                      const gdn_mla_view_t* y, gdn_stream_t stream)
{
    if (!s) return GDN_ERR_NULL;
    if (!io_ok(s->io)) return GDN_ERR_MODE;
    if (!scan_ok(s->B, s->D, s->N, s->G) || s->T < 1 || s->T > 8 || s->slots < 1 || (!src && s->slots < s->B)) return GDN_ERR_SHAPE;
    ScanStepArgs a;
    memset(&a, 0, sizeof(a));
    a.s = *s;
    GDN_TRY(take(x, true, 1, s->io, &a.x));
    GDN_TRY(take(dt, true, 1, s->io, &a.dt));
    GDN_TRY(take(z, z != nullptr, 1, s->io, &a.z));
    GDN_TRY(take(Bm, true, s->G, s->io, &a.Bm));
    GDN_TRY(take(Cm, true, s->G, s->io, &a.Cm));
    GDN_TRY(take(y, true, 1, s->io, &a.y));
    GDN_TRY(weight(A_log, true));
    GDN_TRY(weight(D_skip, false));
    GDN_TRY(weight(dt_bias, false));
    GDN_TRY(weight(state, true));
    if (!aligned(src, 4) || !aligned(dst, 4)) return GDN_ERR_ALIGN;
    GDN_TRY(check_device());
    a.A_log = A_log; a.D_skip = D_skip; a.dt_bias = dt_bias; a.state = state; a.src = src; a.dst = dst;
    return done(launch_scan_step(a, (cudaStream_t)stream));
}
