// mla_api.cu -- the C ABI of the latent-attention operators: argument checks, workspace carve-up, dispatch.
#include <string.h>

#include "mla_internal.h"

using namespace gdn;
using namespace gdn::mla;

namespace {

bool prep_ok(const gdn_mla_prep_t& s)
{
    if (s.N < 0 || s.H < 0 || s.H > 65535 || s.npos < 0) return false;
    if (s.N > 0 && s.npos == 0) return false;      // no position would be good, no token written
    if (s.dc < 8 || s.dc > 1024 || s.dc % 8 || s.dr < 0 || s.dr > 128 || s.dr % 16) return false;
    if (!(s.eps >= 0.f)) return false;
    if (s.page < 0) return false;
    if (s.page > 0) {
        if (s.B < 1 || s.npages < 1 || s.maxpages < 1) return false;
        if ((double)s.npages * s.page >= 2147483648.0) return false;
    }
    return (double)s.N * (s.H + 1) < (double)(1LL << 36);   // blocks of a launch stay below 2^31
}

gdn_status_t prep_common(const gdn_mla_prep_t* s, const void* kv, long long kv_tok, const float* w, const float* rot,
                         const int* pos)
{
    if (!s) return GDN_ERR_NULL;
    if (!io_ok(s->io)) return GDN_ERR_MODE;
    if (!prep_ok(*s)) return GDN_ERR_SHAPE;
    if (s->N == 0) return GDN_OK;
    if (!kv || !w || !pos || (s->dr > 0 && !rot)) return GDN_ERR_NULL;
    if (kv_tok < s->dc + s->dr) return GDN_ERR_SHAPE;
    if (!aligned(kv, 16) || kv_tok % (s->io == GDN_BF16 ? 8 : 4) || !aligned(w, 4) || !aligned(rot, 16) || !aligned(pos, 4))
        return GDN_ERR_ALIGN;
    return GDN_OK;
}

bool attn_ok(const gdn_mla_attn_t& s)
{
    if (s.B < 1 || s.B > 65535 || s.H < 1 || s.H > 65535 || s.Hkv < 1 || s.H % s.Hkv) return false;
    if (s.Tq < 0 || s.Tk < 0 || s.Nq < 0 || s.Nk < 0) return false;
    if (s.dn < 8 || s.dn > 128 || s.dn % 8 || s.dr < 0 || s.dr > 64 || s.dr % 8 || s.dv < 8 || s.dv > 128 || s.dv % 8)
        return false;
    // rows with their heads are numbered by 64 bits, launched by 32
    return (double)s.Nq * s.H < 8.0 * 2147483647.0 && (double)s.Nk * s.Hkv < 8.0 * 2147483647.0 && s.scale >= 0.f && s.scale < 1e30f;
}

struct AttnWs {
    size_t delta, dkr, total;
};
AttnWs attn_ws(const gdn_mla_attn_t& s, int backward)
{
    AttnWs w;
    w.delta = 256;
    w.dkr = backward ? round_up(w.delta + (size_t)s.H * s.Nq * 4, 256) : 256;
    w.total = backward ? round_up(w.dkr + (size_t)s.Hkv * s.Nk * s.dr * 4, 256) : 256;
    return w;
}

// what both directions of the expanded attention check and take
gdn_status_t attn_common(const gdn_mla_attn_t* s, const gdn_mla_view_t* qn, const gdn_mla_view_t* qr,
                         const gdn_mla_view_t* kn, const gdn_mla_view_t* kr, const gdn_mla_view_t* v,
                         const int* cu_q, const int* cu_k, void* ws, size_t ws_bytes, int backward, AttnArgs* a)
{
    if (!s) return GDN_ERR_NULL;
    if (!io_ok(s->io)) return GDN_ERR_MODE;
    if (!attn_ok(*s)) return GDN_ERR_SHAPE;
    memset(a, 0, sizeof(*a));
    a->s = *s;
    a->s.Tq = s->Tq < s->Nq ? s->Tq : s->Nq;
    a->s.Tk = s->Tk < s->Nk ? s->Tk : s->Nk;
    const bool q = s->Nq > 0, k = s->Nk > 0;
    GDN_TAKE(qn, q, s->H, s->io, &a->qn);
    GDN_TAKE(qr, q && s->dr > 0, s->H, s->io, &a->qr);
    GDN_TAKE(kn, k, s->Hkv, s->io, &a->kn);
    GDN_TAKE(kr, k && s->dr > 0, 1, s->io, &a->kr);
    GDN_TAKE(v, k, s->Hkv, s->io, &a->v);
    if (!cu_q && (long long)s->B * s->Tq != s->Nq) return GDN_ERR_SHAPE;
    if (!cu_k && (long long)s->B * s->Tk != s->Nk) return GDN_ERR_SHAPE;
    if (!aligned(cu_q, 4) || !aligned(cu_k, 4)) return GDN_ERR_ALIGN;
    if (!ws || ws_bytes < attn_ws(*s, backward).total) return GDN_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return GDN_ERR_ALIGN;
    a->cu_q = cu_q;
    a->cu_k = cu_k;
    a->status = (uint32_t*)ws;
    return GDN_OK;
}

bool cache_ok(const gdn_mla_cache_t& s)
{
    if (s.B < 1 || s.B > 65535 || s.T < 1 || s.T > 8 || s.H < 1 || (long long)s.T * s.H > 1024) return false;
    if (s.dc < 8 || s.dc > 512 || s.dc % 8 || s.dr < 0 || s.dr > 64 || s.dr % 8) return false;
    if (s.page < 8 || s.page % 8 || s.npages < 1 || s.maxpages < 1) return false;
    if ((double)s.npages * s.page >= 2147483648.0 || (double)s.maxpages * s.page >= 2147483648.0) return false;
    // the tiles that the lengths can name are counted in 32 bits
    if ((double)s.B * (((double)s.maxpages * s.page + kDecodeTile - 1) / kDecodeTile + 1) >= 2147483648.0) return false;
    return s.scale >= 0.f && s.scale < 1e30f;
}

}  // namespace

extern "C" gdn_status_t gdn_mla_prep(const gdn_mla_prep_t* s, const void* kv, long long kv_tok, const float* w,
                                     const float* rot, const int* pos, const int* seq, const int* table,
                                     const gdn_mla_view_t* qr, const gdn_mla_view_t* lat, const gdn_mla_view_t* kr,
                                     const gdn_mla_view_t* qr_out, gdn_stream_t stream)
{
    gdn_status_t r = prep_common(s, kv, kv_tok, w, rot, pos);
    if (r != GDN_OK) return r;
    if (s->N == 0) return GDN_OK;
    PrepArgs a;
    memset(&a, 0, sizeof(a));
    a.s = *s;
    a.kv = kv; a.kv_tok = kv_tok; a.w = w; a.rot = rot; a.pos = pos;
    const bool queries = s->H > 0 && s->dr > 0;
    GDN_TAKE(qr, queries, s->H, s->io, &a.qr);
    GDN_TAKE(qr_out, queries, s->H, s->io, &a.qr_out);
    if (s->page > 0) {
        if (!lat || !lat->p || !seq || !table) return GDN_ERR_NULL;
        if (!aligned(lat->p, 16) || !aligned(seq, 4) || !aligned(table, 4)) return GDN_ERR_ALIGN;
        a.lat = *lat;
        a.seq = seq;
        a.table = table;
    } else {
        GDN_TAKE(lat, true, 1, s->io, &a.lat);
        GDN_TAKE(kr, s->dr > 0, 1, s->io, &a.kr);
    }
    if ((r = check_device()) != GDN_OK) return r;
    return launch_prep(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" size_t gdn_mla_prep_workspace_bytes(const gdn_mla_prep_t* s)
{
    if (!s || !io_ok(s->io) || !prep_ok(*s) || s->page > 0) return 0;
    return round_up(256 + (size_t)prep_bwd_blocks(s->N) * s->dc * sizeof(float), 256);
}

extern "C" gdn_status_t gdn_mla_prep_bwd(const gdn_mla_prep_t* s, const void* kv, long long kv_tok, const float* w,
                                         const float* rot, const int* pos, const gdn_mla_view_t* dlat,
                                         const gdn_mla_view_t* dkr, const gdn_mla_view_t* dqr, void* dkv,
                                         long long dkv_tok, float* dw, const gdn_mla_view_t* dqr_out, void* ws,
                                         size_t ws_bytes, gdn_stream_t stream)
{
    gdn_status_t r = prep_common(s, kv, kv_tok, w, rot, pos);
    if (r != GDN_OK) return r;
    if (s->page > 0) return GDN_ERR_MODE;
    if (!dw) return GDN_ERR_NULL;
    if (!aligned(dw, 4)) return GDN_ERR_ALIGN;
    PrepArgs a;
    memset(&a, 0, sizeof(a));
    a.s = *s;
    a.kv = kv; a.kv_tok = kv_tok; a.w = w; a.rot = rot; a.pos = pos;
    const bool tok = s->N > 0, queries = tok && s->H > 0 && s->dr > 0;
    GDN_TAKE(dlat, tok, 1, s->io, &a.dlat);
    GDN_TAKE(dkr, tok && s->dr > 0, 1, s->io, &a.dkr);
    GDN_TAKE(dqr, queries, s->H, s->io, &a.dqr);
    GDN_TAKE(dqr_out, queries, s->H, s->io, &a.dqr_out);
    if (tok) {
        if (!dkv) return GDN_ERR_NULL;
        if (dkv_tok < s->dc + s->dr) return GDN_ERR_SHAPE;
        if (!aligned(dkv, 16) || dkv_tok % (s->io == GDN_BF16 ? 8 : 4)) return GDN_ERR_ALIGN;
    }
    if (!ws || ws_bytes < gdn_mla_prep_workspace_bytes(s)) return GDN_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return GDN_ERR_ALIGN;
    if ((r = check_device()) != GDN_OK) return r;
    a.dkv = dkv; a.dkv_tok = dkv_tok; a.dw = dw;
    a.partial = (float*)((unsigned char*)ws + 256);
    cudaStream_t st = (cudaStream_t)stream;
    if (cudaMemsetAsync(ws, 0, 256, st) != cudaSuccess) return GDN_ERR_CUDA;
    return launch_prep_bwd(a, st) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" size_t gdn_mla_workspace_bytes(const gdn_mla_attn_t* s, int backward)
{
    if (!s || !io_ok(s->io) || !attn_ok(*s)) return 0;
    return attn_ws(*s, backward).total;
}

extern "C" gdn_status_t gdn_mla_fwd(const gdn_mla_attn_t* s, const gdn_mla_view_t* qn, const gdn_mla_view_t* qr,
                                    const gdn_mla_view_t* kn, const gdn_mla_view_t* kr, const gdn_mla_view_t* v,
                                    const int* cu_q, const int* cu_k, void* o, float* lse, void* ws,
                                    size_t ws_bytes, gdn_stream_t stream)
{
    AttnArgs a;
    gdn_status_t r = attn_common(s, qn, qr, kn, kr, v, cu_q, cu_k, ws, ws_bytes, 0, &a);
    if (r != GDN_OK) return r;
    if (s->Nq > 0 && !o) return GDN_ERR_NULL;
    if (!aligned(o, 16) || !aligned(lse, 4)) return GDN_ERR_ALIGN;
    if ((r = check_device()) != GDN_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    if (cudaMemsetAsync(ws, 0, 256, st) != cudaSuccess) return GDN_ERR_CUDA;
    if (s->Nq == 0 || s->Tq == 0) return GDN_OK;
    a.o = o;
    a.lse = lse;
    const cudaError_t e = s->io == GDN_BF16 ? launch_attn_tc(a, st) : launch_attn_f32(a, st);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" gdn_status_t gdn_mla_bwd(const gdn_mla_attn_t* s, const gdn_mla_view_t* qn, const gdn_mla_view_t* qr,
                                    const gdn_mla_view_t* kn, const gdn_mla_view_t* kr, const gdn_mla_view_t* v,
                                    const int* cu_q, const int* cu_k, const void* o, const float* lse,
                                    const void* dO, const gdn_mla_view_t* dqn, const gdn_mla_view_t* dqr,
                                    const gdn_mla_view_t* dkn, const gdn_mla_view_t* dkr, const gdn_mla_view_t* dv,
                                    void* ws, size_t ws_bytes, gdn_stream_t stream)
{
    AttnArgs a;
    gdn_status_t r = attn_common(s, qn, qr, kn, kr, v, cu_q, cu_k, ws, ws_bytes, 1, &a);
    if (r != GDN_OK) return r;
    const bool q = s->Nq > 0, k = s->Nk > 0;
    if (q && (!o || !lse || !dO)) return GDN_ERR_NULL;
    if (!aligned(o, 16) || !aligned(dO, 16) || !aligned(lse, 4)) return GDN_ERR_ALIGN;
    GDN_TAKE(dqn, q, s->H, s->io, &a.dqn);
    GDN_TAKE(dqr, q && s->dr > 0, s->H, s->io, &a.dqr);
    GDN_TAKE(dkn, k, s->Hkv, s->io, &a.dkn);
    GDN_TAKE(dkr, k && s->dr > 0, 1, s->io, &a.dkr);
    GDN_TAKE(dv, k, s->Hkv, s->io, &a.dv);
    if ((r = check_device()) != GDN_OK) return r;
    cudaStream_t st = (cudaStream_t)stream;
    if (cudaMemsetAsync(ws, 0, 256, st) != cudaSuccess) return GDN_ERR_CUDA;
    const AttnWs w = attn_ws(*s, 1);
    a.o = const_cast<void*>(o);
    a.lse = const_cast<float*>(lse);
    a.dO = dO;
    a.delta = (float*)((unsigned char*)ws + w.delta);
    a.dkr_part = (float*)((unsigned char*)ws + w.dkr);
    const cudaError_t e = s->io == GDN_BF16 ? launch_attn_bwd_tc(a, st) : launch_attn_bwd_f32(a, st);
    return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

extern "C" size_t gdn_mla_decode_workspace_bytes(const gdn_mla_cache_t* s)
{
    if (!s || !io_ok(s->io) || !cache_ok(*s)) return 0;
    return decode_plan(*s).total;
}

extern "C" gdn_status_t gdn_mla_decode(const gdn_mla_cache_t* s, const gdn_mla_view_t* qc, const gdn_mla_view_t* qr,
                                       const void* cache, const int* table, const int* len, void* o, float* lse,
                                       void* ws, size_t ws_bytes, gdn_stream_t stream)
{
    if (!s) return GDN_ERR_NULL;
    if (!io_ok(s->io)) return GDN_ERR_MODE;
    if (!cache_ok(*s)) return GDN_ERR_SHAPE;
    DecodeArgs a;
    memset(&a, 0, sizeof(a));
    a.s = *s;
    GDN_TAKE(qc, true, s->H, s->io, &a.qc);
    GDN_TAKE(qr, s->dr > 0, s->H, s->io, &a.qr);
    if (!cache || !table || !len || !o) return GDN_ERR_NULL;
    if (!aligned(cache, 16) || !aligned(table, 4) || !aligned(len, 4) || !aligned(o, 16) || !aligned(lse, 4))
        return GDN_ERR_ALIGN;
    const DecodePlan p = decode_plan(*s);
    if (!ws || ws_bytes < p.total) return GDN_ERR_WORKSPACE;
    if (!aligned(ws, 256)) return GDN_ERR_ALIGN;
    const gdn_status_t r = check_device();
    if (r != GDN_OK) return r;
    unsigned char* w = (unsigned char*)ws;
    a.cache = cache; a.table = table; a.len = len; a.o = o; a.lse = lse;
    a.status = (uint32_t*)w;
    a.cta_err = (uint32_t*)(w + p.err_off);
    a.part_l = (float*)(w + p.l_off);
    a.part_o = (float*)(w + p.o_off);
    a.rows = p.rows; a.groups = p.groups; a.ctas = p.ctas; a.slots = p.slots;
    return launch_decode(a, (cudaStream_t)stream) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
