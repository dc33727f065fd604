// mla_fwd_tc.cu -- attention over expanded keys and values on the tensor cores (bf16), forward.
//
// A CTA takes two tiles of 128 queries of one head and walks the keys in tiles of 128 with the running maximum and sum
// of a softmax.  Scores S = Q K^T land in TMEM, a thread a row; the weights P go back into TMEM over them, as bf16
// pairs, and are the A operand of O += P V straight from there; O stays in TMEM.  Two query tiles take turns: while
// one's softmax runs, the tensor cores work on the other's products.  The position part is one more 64-column block of
// Q and K (K's is the same for every head).  The maximum that scores are lowered by is raised, and O rescaled, only
// when a score exceeds it by 2^8: P, the sums and O hold that range with the same relative precision.
//
// Shared memory's 128 bytes a cycle and the tensor cores bound a long walk together: a step of two 128 x 128 tiles takes
// 2640 cycles, 2048 of them products (2 x 2048 queries over 8192 keys, 16 heads of 128: 169 us, 1.42 PFLOP/s; 8 x 4096
// tokens: 0.39 ms).  With three 64-column blocks a query tile pair leaves V one stage, and its load shows.
//
// Roles (12 warps): warp 0 loads tiles by TMA, warp 1 issues products, warps 2-3 blank the value rows past a ragged
// end (a weight of zero would still meet a NaN there), warps 4-7 and 8-11 are the two tiles' softmax.
#include "mla_tc.cuh"

namespace gdn {
namespace mla {

namespace {

constexpr int kTile = 128;
constexpr uint32_t kBlock = 16384;      // 128 rows x 64 columns of bf16
constexpr float kSlack = 8.f;           // log2 by which a score may exceed the maximum it is lowered by
constexpr int kMaxStage = 3;
constexpr int kShort = 1024;            // keys

struct Params {
    AttnArgs a;
    CUtensorMap qn, qr, kn, kr, v;
    int nb, vb;                 // 64-column blocks of dn, dv
    int tiles;                  // CTAs that the longest sequence's queries take
    uint32_t v_off;             // V's stages behind K's in shared memory
    int kstages, vstages;
    int starve;                 // failure-path test hook: a key tile that is announced, but never loaded (-1: none)
};

struct Shared {
    uint64_t q_full[2], k_full[kMaxStage], k_empty[kMaxStage], v_full[kMaxStage], v_empty[kMaxStage], v_last, v_fixed, s_full[2],
        p_full[2][2], o_full[2], drain;
    uint32_t tmem, gave_up;
};

// KB: 64-column blocks of a query or key (the position block among them); NT: query tiles, 2 on an SM of its own or 1 on
// half of one
template <int KB, int NT>
__global__ void __launch_bounds__(128 + 128 * NT, 3 - NT) fwd_tc_kernel(const __grid_constant__ Params p)
{
    extern __shared__ unsigned char raw[];
    __shared__ Shared S;
    const AttnArgs& a = p.a;
    const gdn_mla_attn_t& s = a.s;
    const int h = blockIdx.x % s.H, b = blockIdx.y, g = h / (s.H / s.Hkv);
    const int q0 = (p.tiles - 1 - (int)(blockIdx.x / s.H)) * NT * kTile;     // the longest walks first
    const Rows rq = rows_of(a.cu_q, b, s.Tq, s.Nq), rk = rows_of(a.cu_k, b, s.Tk, s.Nk);
    if (q0 >= rq.n) return;
    const int off = rk.n - rq.n;
    // key tiles that each query tile sees
    int nt[2] = {0, 0};
#pragma unroll
    for (int t = 0; t < NT; t++) {
        const int first = q0 + t * kTile;
        const int end = s.causal ? min(rk.n, min(first + kTile, rq.n) + off) : rk.n;
        nt[t] = first < rq.n && end > 0 ? (end + kTile - 1) / kTile : 0;
    }
    const int n = max(nt[0], nt[1]);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    const uint32_t qs = smem_u32(sm), ks = qs + NT * KB * kBlock, vs = qs + p.v_off;

    const bool rope = s.dr > 0;
    const bool ragged = rk.n % kTile != 0 && n == (rk.n + kTile - 1) / kTile;   // the last value tile has rows to blank
    const auto load_q = [&](int t) {
        mbar_arrive_expect_tx(&S.q_full[t], KB * kBlock);
        for (int c = 0; c < p.nb; c++)
            tma_load_3d(qs + (t * KB + c) * kBlock, &p.qn, &S.q_full[t], 64 * c, h, rq.first + q0 + t * kTile);
        if (rope) tma_load_3d(qs + (t * KB + p.nb) * kBlock, &p.qr, &S.q_full[t], 0, h, rq.first + q0 + t * kTile);
    };
    const auto load_k = [&](int j, int st) {
        mbar_arrive_expect_tx(&S.k_full[st], KB * kBlock);
        if (j == p.starve) return;
        const uint32_t d = ks + st * KB * kBlock;
        for (int c = 0; c < p.nb; c++) tma_load_3d(d + c * kBlock, &p.kn, &S.k_full[st], 64 * c, g, rk.first + j * kTile);
        if (rope) tma_load_3d(d + p.nb * kBlock, &p.kr, &S.k_full[st], 0, 0, rk.first + j * kTile);
    };
    const auto load_v = [&](int j, int st) {
        uint64_t* bar = ragged && j == n - 1 ? &S.v_last : &S.v_full[st];   // to the warps that blank rows
        mbar_arrive_expect_tx(bar, p.vb * kBlock);
        for (int c = 0; c < p.vb; c++) tma_load_3d(vs + (st * p.vb + c) * kBlock, &p.v, bar, 64 * c, g, rk.first + j * kTile);
    };
    if (warp == 0) {
        if (elect_one()) {
            for (int i = 0; i < 2; i++) {
                mbar_init(&S.q_full[i], 1);
                mbar_init(&S.s_full[i], 1);
                mbar_init(&S.p_full[i][0], 4);
                mbar_init(&S.p_full[i][1], 4);
                mbar_init(&S.o_full[i], 1);
            }
            for (int i = 0; i < kMaxStage; i++) {
                mbar_init(&S.k_full[i], 1);
                mbar_init(&S.k_empty[i], 1);
                mbar_init(&S.v_full[i], 1);
                mbar_init(&S.v_empty[i], 1);
            }
            mbar_init(&S.v_last, 1);
            mbar_init(&S.v_fixed, 64);
            mbar_init(&S.drain, 1);
            fence_mbar_init();
            S.gave_up = 0;
            if (n > 0) {      // the first tiles come while the other warps set up
                if (nt[0]) load_q(0);
                load_k(0, 0);
                if (nt[1]) load_q(1);
                load_v(0, 0);
            }
        }
    } else if (warp == 1) {
        tmem_alloc(&S.tmem, 256 * NT);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    volatile uint32_t* gave_up = &S.gave_up;
    if (warp < 4) {
        regs_down<NT == 2 ? 88 : 64>();      // of 168 a thread in 384, or 128 in 256
        if (warp == 0) {
            if (elect_one() && n > 0) {
                int klast = 0, vlast = 0, kst = 1 % p.kstages, vst = 1 % p.vstages;
                uint32_t kph = p.kstages == 1, vph = p.vstages == 1;
                for (int j = 1; j < n; j++) {
                    if (!wait_for(&S.k_empty[kst], kph ^ 1, gave_up) || *gave_up) break;
                    load_k(klast = j, kst);
                    if (++kst == p.kstages) kst = 0, kph ^= 1;
                    if (!wait_for(&S.v_empty[vst], vph ^ 1, gave_up) || *gave_up) break;
                    load_v(vlast = j, vst);
                    if (++vst == p.vstages) vst = 0, vph ^= 1;
                }
                if (*gave_up) {   // a wait expired: the loads in flight land before the CTA ends
                    for (int t = 0; t < 2; t++)
                        if (nt[t]) mbar_wait(&S.q_full[t], 0, nullptr, kDrainNs);
                    for (int j = max(0, klast - p.kstages + 1); j <= klast; j++)
                        mbar_wait(&S.k_full[j % p.kstages], (j / p.kstages) & 1, nullptr, kDrainNs);
                    for (int j = max(0, vlast - p.vstages + 1); j <= vlast; j++) {
                        if (ragged && j == n - 1)
                            mbar_wait(&S.v_last, 0, nullptr, kDrainNs);
                        else
                            mbar_wait(&S.v_full[j % p.vstages], (j / p.vstages) & 1, nullptr, kDrainNs);
                    }
                }
            }
        } else if (warp == 1) {
            if (elect_one()) {
                const uint32_t id_s = idesc_bf16(128, 128, false, false);
                const uint32_t id_o = idesc_bf16(128, (s.dv + 15) & ~15, false, true);
                const uint64_t kmajor = sdesc(0, 16u, 1024u), vmajor = sdesc(0, kBlock, 1024u);
                // 16-value steps of each block that hold anything
                int steps[KB];
#pragma unroll
                for (int c = 0; c < KB; c++) steps[c] = c < p.nb ? (min(64, s.dn - 64 * c) + 15) >> 4 : (s.dr + 15) >> 4;
                auto scores = [&](int t, int st) {
                    const uint64_t q = kmajor + at_desc(qs + t * KB * kBlock), k = kmajor + at_desc(ks + st * KB * kBlock);
#pragma unroll
                    for (int c = 0; c < KB; c++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (e < steps[c])
                                mma_bf16(tmem + t * 128, q + c * (kBlock >> 4) + 2 * e, k + c * (kBlock >> 4) + 2 * e, id_s,
                                         (c | e) ? 1u : 0u);
                    mma_commit(&S.s_full[t]);
                };
                int kst = 0, vst = 0;
                uint32_t kph = 0, vph = 0;
                if (n > 0) {
                    wait_for(&S.k_full[0], 0, gave_up);
#pragma unroll
                    for (int t = 0; t < NT; t++)
                        if (nt[t]) {
                            wait_for(&S.q_full[t], 0, gave_up);
                            tc_fence_after();
                            if (!*gave_up) scores(t, 0);
                        }
                    mma_commit(&S.k_empty[0]);
                    if (++kst == p.kstages) kst = 0, kph = 1;
                }
                for (int j = 0; j < n; j++) {
                    if (j == n - 1 && ragged)
                        wait_for(&S.v_fixed, 0, gave_up);
                    else
                        wait_for(&S.v_full[vst], vph, gave_up);
                    bool k_ready = false;
#pragma unroll
                    for (int t = 0; t < NT; t++)
                        if (j < nt[t]) {
                            const uint64_t v = vmajor + at_desc(vs + vst * p.vb * kBlock);
#pragma unroll
                            for (int half = 0; half < 2; half++) {
                                wait_for(&S.p_full[t][half], j & 1, gave_up);
                                tc_fence_after();
                                if (!*gave_up) {
#pragma unroll
                                    for (int e = 4 * half; e < 4 * half + 4; e++)
                                        mma_bf16_ts(tmem + NT * 128 + t * 128, tmem + t * 128 + 8 * e, v + 128 * e, id_o,
                                                    (j | e) ? 1u : 0u);
                                }
                            }
                            if (j + 1 < nt[t]) {
                                if (!k_ready) wait_for(&S.k_full[kst], kph, gave_up);
                                k_ready = true;
                                tc_fence_after();
                                if (!*gave_up) scores(t, kst);
                            } else {
                                mma_commit(&S.o_full[t]);
                            }
                        }
                    mma_commit(&S.v_empty[vst]);
                    if (++vst == p.vstages) vst = 0, vph ^= 1;
                    if (j + 1 < n) {
                        mma_commit(&S.k_empty[kst]);
                        if (++kst == p.kstages) kst = 0, kph ^= 1;
                    }
                }
                if (*gave_up) {   // the products in flight end before TMEM is freed
                    mma_commit(&S.drain);
                    mbar_wait(&S.drain, 0, nullptr, kDrainNs);
                }
            }
        } else if (ragged) {
            const int st = (n - 1) % p.vstages;
            wait_for(&S.v_last, 0, gave_up);
            const int valid = rk.n - (n - 1) * kTile, bad = kTile - valid;
            for (int c = 0; c < p.vb; c++) {
                unsigned char* v = sm + p.v_off + (st * p.vb + c) * kBlock + valid * 128;
                for (int e = tid - 64; e < bad * 8; e += 64) *reinterpret_cast<uint4*>(v + e * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            mbar_arrive(&S.v_fixed);
        }
    } else {
        regs_up<NT == 2 ? 208 : 192>();
        const int t = (warp - 4) >> 2, quad = warp & 3, row = q0 + t * kTile + quad * 32 + lane;
        const uint32_t base = tmem + ((uint32_t)quad << 21), sa = base + t * 128, oa = base + NT * 128 + t * 128;
        // scores times this are exponents of 2; a scale of zero keeps the masked ones' minus infinity
        const float c = fmaxf(s.scale * kLog2e, 1e-37f), slack = kSlack / c;
        const int last = row < rq.n ? (s.causal ? min(rk.n - 1, row + off) : rk.n - 1) : -1;
        const int calm = s.causal ? min(rk.n - 1, q0 + t * kTile + quad * 32 + off) : rk.n - 1;   // the warp's smallest
        float top = -INFINITY;
        uint64_t sum[2] = {0, 0};
        const int steps = t ? nt[1] : nt[0];
        for (int j = 0; j < steps; j++) {
            wait_for(&S.s_full[t], j & 1, gave_up);
            __syncwarp();
            tc_fence_after();
            uint32_t x[128];
            float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            const bool masked = j * kTile + kTile - 1 > calm;
            const int lim = last - j * kTile;
            tmem_ld32(sa, x);
            tmem_ld32(sa + 32, x + 32);
#pragma unroll
            for (int i0 = 0; i0 < 128; i0 += 64) {
                tmem_wait_ld();
                if (i0 == 0) {       // the second half comes while the first one's maximum is taken
                    tmem_ld32(sa + 64, x + 64);
                    tmem_ld32(sa + 96, x + 96);
                }
                if (masked) {
#pragma unroll
                    for (int i = i0; i < i0 + 64; i++) x[i] = i <= lim ? x[i] : 0xff800000u;
                }
#pragma unroll
                for (int i = i0; i < i0 + 64; i += 8)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        m[e] = fmaxf(m[e], fmaxf(__uint_as_float(x[i + 2 * e]), __uint_as_float(x[i + 2 * e + 1])));
            }
            const float most = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
            const bool raise = most > top + slack || top == -INFINITY;
            if (__any_sync(0xffffffffu, raise)) {
                const float now = raise ? fmaxf(most, top) : top;
                const float keep = now == top ? 1.f : fast_exp2((top - now) * c);     // the first time: 0 of nothing
                top = now;
                __syncwarp();
                const uint64_t k2 = pack2(keep, keep);
                sum[0] = mul2(sum[0], k2);
                sum[1] = mul2(sum[1], k2);
                if (j > 0) {     // the scores' commit says that the products into O are done too
#pragma unroll 1
                    for (int i = 0; i < 64 * p.vb; i += 16) {
                        float o[16];
                        tmem_ld16(oa + i, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e++) o[e] *= keep;
                        tmem_st16(oa + i, o);
                    }
                }
            }
            const float lower = top == -INFINITY ? 0.f : -top * c;
            const uint64_t c2 = pack2(c, c), l2 = pack2(lower, lower);
#pragma unroll
            for (int i = 0; i < 128; i += 32) {
                uint32_t y[16];
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    float u, w;
                    unpack2(fma2(pack2(__uint_as_float(x[i + 2 * e]), __uint_as_float(x[i + 2 * e + 1])), c2, l2), u, w);
                    u = fast_exp2(u);
                    w = fast_exp2(w);
                    sum[e & 1] = add2(sum[e & 1], pack2(u, w));
                    y[e] = pack_bf16(u, w);
                }
                tmem_st16u(sa + (i >> 1), y);
                if (i == 32 || i == 96) {     // 64 keys' weights at a time: their products need not wait for the rest
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.p_full[t][i >> 6]);
                    __syncwarp();
                }
            }
        }
        float l = 0.f;
        {
            float u, w;
            unpack2(add2(sum[0], sum[1]), u, w);
            l = u + w;
        }
        const bool mine = row < rq.n;
        if (mine && a.lse) a.lse[(long long)h * s.Nq + rq.first + row] = l == 0.f ? -INFINITY : (top * c + log2f(l)) * kLn2;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (steps > 0) {
            wait_for(&S.o_full[t], 0, gave_up);
            __syncwarp();
            tc_fence_after();
        }
        // rows to global memory by way of this tile's Q, which no product reads any more: a thread holds a row, but a
        // store of the warp is to cover whole lines
        unsigned char* stage = sm + t * KB * kBlock + quad * 32 * 128;
        __nv_bfloat16* out = (__nv_bfloat16*)a.o + ((long long)(rq.first + q0 + t * kTile + quad * 32) * s.H + h) * s.dv;
#pragma unroll 1
        for (int i = 0; i < s.dv; i += 64) {
            __syncwarp();
#pragma unroll
            for (int e = 0; e < 64; e += 16) {
                float o[16];
                if (steps > 0) {
                    tmem_ld16(oa + i + e, o);
                    tmem_wait_ld();
                }
                uint32_t y[8];
#pragma unroll
                for (int f = 0; f < 8; f++) y[f] = steps > 0 ? pack_bf16(o[2 * f] * inv, o[2 * f + 1] * inv) : 0u;
                *reinterpret_cast<uint4*>(stage + sw128(lane, e)) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(stage + sw128(lane, e + 8)) = make_uint4(y[4], y[5], y[6], y[7]);
            }
            __syncwarp();
            const int col = (lane & 7) * 8, rows = rq.n - (q0 + t * kTile + quad * 32);
#pragma unroll
            for (int r = lane >> 3; r < 32; r += 4)
                if (r < rows && i + col < s.dv)
                    *reinterpret_cast<uint4*>(out + (long long)r * s.H * s.dv + i + col) =
                        *reinterpret_cast<const uint4*>(stage + sw128(r, col));
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 256 * NT);
    }
    if (tid == 0 && *gave_up) atomicExch(a.status, kDevTimeout);
}

template <int KB, int NT>
cudaError_t run(Params& p, cudaStream_t st)
{
    const gdn_mla_attn_t& s = p.a.s;
    // of the 228 KB an SM has, 1 KB goes with each CTA
    const uint32_t room = 233472 / (3 - NT) - 1024 - 1024 - (uint32_t)sizeof(Shared) - 64, q = NT * KB * kBlock;
    p.kstages = p.vstages = 1;      // as many stages as fit, keys' first
    const auto total = [&] { return q + (uint32_t)(p.kstages * KB + p.vstages * p.vb) * kBlock; };
    for (int i = 0; i < 2; i++) {
        if (p.kstages < kMaxStage && total() + KB * kBlock <= room) p.kstages++;
        if (p.vstages < kMaxStage && total() + p.vb * kBlock <= room) p.vstages++;
    }
    p.v_off = q + p.kstages * KB * kBlock;
    p.tiles = (s.Tq + NT * kTile - 1) / (NT * kTile);
    const size_t bytes = 1024 + total();
    const cudaError_t e = cudaFuncSetAttribute(fwd_tc_kernel<KB, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    fwd_tc_kernel<KB, NT><<<dim3((unsigned)s.H * p.tiles, s.B), 128 + 128 * NT, bytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_tc(const AttnArgs& a, cudaStream_t st)
{
    const gdn_mla_attn_t& s = a.s;
    Params p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    p.starve = test_starve_chunk();
    p.nb = (s.dn + 63) / 64;
    p.vb = (s.dv + 63) / 64;
    // without keys the maps have nothing to describe and no load is made
    if (!view_map(&p.qn, a.qn, s.Nq, s.H, s.dn, kTile) ||
        (s.dr > 0 && !view_map(&p.qr, a.qr, s.Nq, s.H, s.dr, kTile)) ||
        (s.Nk > 0 && (!view_map(&p.kn, a.kn, s.Nk, s.Hkv, s.dn, kTile) || !view_map(&p.v, a.v, s.Nk, s.Hkv, s.dv, kTile) ||
                      (s.dr > 0 && !view_map(&p.kr, a.kr, s.Nk, 1, s.dr, kTile)))))
        return cudaErrorInvalidValue;
    const int kb = p.nb + (s.dr > 0 ? 1 : 0);
    // One tile and two CTAs an SM for short walks, where a CTA's start and end weigh most and overlap the other's work;
    // two tiles share each load of keys and values, which long walks need.  Two tiles against one, us: 12 x 256 tokens
    // 20.0 / 18.0, 12 x 512 32.8 / 30.9, 8 x 1024 51.4 / 51.7, 6 x 1536 65.1 / 69.3, 2 x 4096 105 / 117.
    const bool single = kb < 3 && s.Tk <= kShort;
    if (kb == 1) return single ? run<1, 1>(p, st) : run<1, 2>(p, st);
    if (kb == 2) return single ? run<2, 1>(p, st) : run<2, 2>(p, st);
    return run<3, 2>(p, st);     // three blocks of Q, K and V's leave no room for a second CTA
}

}  // namespace mla
}  // namespace gdn
