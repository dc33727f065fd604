/*
 * gdn_mla.h -- latent attention (MLA), the other token mixer of the hybrid that gdn.h's recurrence belongs to.
 *
 * "GDN & MLA Mechanism Deep-Dive" pairs the gated delta rule with full-attention layers whose keys and values come
 * from one low-rank latent a token (MLA: low-rank KV, rotary position on a part of each head, grouped heads, causal).
 * Three operators cover such a layer between its projections, which are plain matrix products of the caller:
 *
 *   gdn_mla_prep / gdn_mla_prep_bwd     the latent's RMS norm, the rotation of the position parts, and the write into
 *                                       a paged cache (or dense rows)
 *   gdn_mla_fwd / gdn_mla_bwd           causal attention over expanded keys and values, with all gradients
 *   gdn_mla_decode                      attention of 1..8 new tokens a sequence over the paged latent cache itself
 *                                       (absorbed form: the up projections sit in the query and behind the output)
 *
 * Conventions are gdn.h's: the caller owns every buffer and the workspace (device memory, 256-byte aligned); nothing
 * is allocated and nothing synchronises; work goes to the caller's stream; argument errors are reported before
 * anything is enqueued; an expired device-side wait is read back with gdn_last_device_status(ws, stream).
 * io is gdn_dtype_t: GDN_BF16 (tensor cores, fp32 accumulation and statistics) or GDN_F32 (CUDA cores, fp32).
 * Every pointer to io-typed data is 16-byte aligned, every width a multiple of 8, every stride a multiple of 8
 * elements (bf16) or 4 (f32); fp32 and int32 arrays are 4-byte aligned unless said otherwise.  Outputs must not
 * alias inputs, except where a comment allows it.
 */
#ifndef GDN_MLA_H
#define GDN_MLA_H

#include "gdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A tensor [rows, heads, width] of which the width is contiguous; tok and head are the distances, in elements,
 * between consecutive rows and heads (positive; head is ignored for one head).  A slice of a projection's output,
 * such as the key part of [rows, heads, d_n + d_v], is such a view. */
typedef struct {
    void* p;
    long long tok, head;
} gdn_mla_view_t;

/* ---------------------------------------------------------------- norm, rotation, cache write
 *
 *   lat[n] = kv[n, :dc] / sqrt(mean(kv[n, :dc]^2) + eps) * w          (statistics in fp32)
 *   kr[n]  = rotate(kv[n, dc:], pos[n]),   qr_out[n, h] = rotate(qr[n, h], pos[n])
 *   rotate(x, p): (x_a, x_b) -> (x_a cos - x_b sin, x_a sin + x_b cos) for the pairs i < dr/2, with
 *   cos = rot[p, i], sin = rot[p, dr/2 + i]; a pair is (x_i, x_{i + dr/2}), or (x_{2i}, x_{2i+1}) if interleaved.
 *
 * page > 0: row n goes to the cache [npages, page, dc + dr] at page table[seq[n], pos[n] / page], place
 * pos[n] % page, latent first.  page = 0: row n of lat and of kr (views of one head).
 * A token whose pos lies outside [0, npos), or whose seq or page lies outside its table, is skipped: its rows
 * (cache; lat, kr, qr_out when the position is bad) are not written.  No two tokens may name the same place.
 * Limits: N, H >= 0, npos >= 1 where N > 0 (without a position part too), 8 <= dc <= 1024, dr a multiple of 16 up to 128
 * (0: no position part). */
typedef struct {
    int N, H;                         /* tokens; query heads (0: no queries)            */
    int dc, dr;                       /* latent width, width of the position part       */
    int io;                           /* gdn_dtype_t                                    */
    int npos;                         /* rows of rot                                    */
    int interleaved;                  /* which two values a rotation turns              */
    int B, page, npages, maxpages;    /* block table [B, maxpages]; page = 0: dense rows */
    float eps;
} gdn_mla_prep_t;

/* kv [N, dc + dr] with row stride kv_tok; w [dc] fp32; rot [npos, dr] fp32, 16-byte aligned; pos, seq [N] int32;
 * table [B, maxpages] int32.  qr, qr_out [N, H, dr] views (NULL iff H = 0 or dr = 0); qr_out may be the very
 * same view as qr.  Paged: lat->p is the cache (lat's strides and kr are ignored). */
gdn_status_t gdn_mla_prep(const gdn_mla_prep_t* shape, const void* kv, long long kv_tok, const float* w,
                          const float* rot, const int* pos, const int* seq, const int* table,
                          const gdn_mla_view_t* qr, const gdn_mla_view_t* lat, const gdn_mla_view_t* kr,
                          const gdn_mla_view_t* qr_out, gdn_stream_t stream);

/* Gradients of the dense form: dkv [N, dc + dr] (row stride dkv_tok), dw [dc] fp32 (overwritten; a fixed-order
 * sum) and dqr_out = the gradient of qr, from dlat, dkr, dqr (dqr_out may be the same view as dqr).  A token whose pos lies
 * outside [0, npos) gets a zero gradient and adds nothing to dw. */
size_t gdn_mla_prep_workspace_bytes(const gdn_mla_prep_t* shape);
gdn_status_t gdn_mla_prep_bwd(const gdn_mla_prep_t* shape, const void* kv, long long kv_tok, const float* w,
                              const float* rot, const int* pos, const gdn_mla_view_t* dlat,
                              const gdn_mla_view_t* dkr, const gdn_mla_view_t* dqr, void* dkv, long long dkv_tok,
                              float* dw, const gdn_mla_view_t* dqr_out, void* ws, size_t ws_bytes,
                              gdn_stream_t stream);

/* ---------------------------------------------------------------- attention over expanded keys and values
 *
 *   s[i, j] = scale (qn[i, h] . kn[j, g] + qr[i, h] . kr[j]),   g = h / (H / Hkv)
 *   o[i, h] = sum_j softmax_j(s[i, j]) v[j, g],                 lse[h, i] = log sum_j exp(s[i, j])
 *
 * over the keys j < n_k that query i sees: all of them, or with causal those j <= i + n_k - n_q (the queries are the
 * sequence's last n_q tokens).  A query that sees no key gets o = 0, lse = -inf and gives no gradient.
 * Sequences: cu_q, cu_k NULL: sequence b holds rows b * Tq .. and b * Tk .. of the tensors; else int32 [B + 1] row
 * offsets on the device, ascending, with sequences of at most Tq and Tk rows (longer ones are cut there, offsets
 * outside [0, Nq] or [0, Nk] are taken as the nearer bound).  Rows of no sequence are neither read into a result nor
 * written.  Values in one sequence never reach another, NaN and Inf included.  Within a sequence a NaN or Inf in a
 * key's v, kn or kr may reach o and the gradients of queries that precede it, by up to 254 positions, and one in a
 * query's qn, qr or dO the gradients of keys that follow it, by up to as many (tiles of 128 meet weights of zero).
 * Limits: H a multiple of Hkv; dn, dv in 8..128, dr in 0..64; B, H <= 65535; Nq, Nk < 2^31, Nq * H and
 * Nk * Hkv < 2^34; scale >= 0. */
typedef struct {
    int B, H, Hkv;
    int Tq, Tk;                       /* most rows of one sequence                      */
    int dn, dr, dv;
    int causal;
    int io;                           /* gdn_dtype_t                                    */
    int Nq, Nk;                       /* rows of the tensors (B * Tq, B * Tk without cu) */
    float scale;
} gdn_mla_attn_t;

/* Workspace of gdn_mla_fwd (backward = 0) or gdn_mla_bwd (1); 0 if the shape is invalid. */
size_t gdn_mla_workspace_bytes(const gdn_mla_attn_t* shape, int backward);

/* qn [Nq, H, dn], qr [Nq, H, dr], kn [Nk, Hkv, dn], kr [Nk, dr], v [Nk, Hkv, dv] views (qr, kr NULL iff dr = 0);
 * o [Nq, H, dv] contiguous; lse [H, Nq] fp32 (NULL: not written). */
gdn_status_t gdn_mla_fwd(const gdn_mla_attn_t* shape, const gdn_mla_view_t* qn, const gdn_mla_view_t* qr,
                         const gdn_mla_view_t* kn, const gdn_mla_view_t* kr, const gdn_mla_view_t* v,
                         const int* cu_q, const int* cu_k, void* o, float* lse, void* ws, size_t ws_bytes,
                         gdn_stream_t stream);

/* Gradients from dO (contiguous as o) with the forward's o and lse.  dqn .. dv are views of their inputs' shapes,
 * with strides of their own.  Every sum runs in a fixed order: the same call gives the same bits. */
gdn_status_t gdn_mla_bwd(const gdn_mla_attn_t* shape, const gdn_mla_view_t* qn, const gdn_mla_view_t* qr,
                         const gdn_mla_view_t* kn, const gdn_mla_view_t* kr, const gdn_mla_view_t* v,
                         const int* cu_q, const int* cu_k, const void* o, const float* lse, const void* dO,
                         const gdn_mla_view_t* dqn, const gdn_mla_view_t* dqr, const gdn_mla_view_t* dkn,
                         const gdn_mla_view_t* dkr, const gdn_mla_view_t* dv, void* ws, size_t ws_bytes,
                         gdn_stream_t stream);

/* ---------------------------------------------------------------- attention over the paged latent cache
 *
 * cache [npages, page, dc + dr]: row j of sequence b is place j % page of page table[b, j / page].
 *   s[t, h, j] = scale (qc[b, t, h] . row_j[:dc] + qr[b, t, h] . row_j[dc:])
 *   o[b, t, h] = sum_j softmax_j(s) row_j[:dc]
 * over the rows j < len[b] - (T - 1 - t): the new tokens' own rows are in the cache already and token t sees its own.
 * lse[b, t, h] = log sum_j exp(s) (fp32, NULL: not written).  A query that sees no row gets o = 0 and lse = -inf.
 * len[b] is taken between 0 and maxpages * page; a page number outside [0, npages) reads as rows of zeros; nothing
 * past len[b] reaches a result, and no sequence another's.  Within a sequence a NaN or Inf in the latent part of one of
 * its last T - 1 rows may reach o of the new tokens that precede that row as well (a weight of zero meets it); their lse
 * it never reaches.  A query that sees a NaN gets one for o and lse.
 * Limits: 1 <= T <= 8, T * H <= 1024, dc in 8..512, dr in 0..64, page a multiple of 8, B <= 65535,
 * npages * page < 2^31, B * (maxpages * page / 64 + 2) < 2^31, scale >= 0. */
typedef struct {
    int B, T, H;
    int dc, dr;
    int page, npages, maxpages;
    int io;                           /* gdn_dtype_t of qc, qr, cache, o                */
    float scale;
} gdn_mla_cache_t;

size_t gdn_mla_decode_workspace_bytes(const gdn_mla_cache_t* shape);

/* qc [B * T, H, dc] and qr [B * T, H, dr] views (qr NULL iff dr = 0); table int32 [B, maxpages]; len int32 [B];
 * o [B, T, H, dc] contiguous. */
gdn_status_t gdn_mla_decode(const gdn_mla_cache_t* shape, const gdn_mla_view_t* qc, const gdn_mla_view_t* qr,
                            const void* cache, const int* table, const int* len, void* o, float* lse, void* ws,
                            size_t ws_bytes, gdn_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_MLA_H */
