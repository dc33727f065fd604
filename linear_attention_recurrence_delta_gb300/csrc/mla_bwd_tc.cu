// mla_bwd_tc.cu -- gradients of the expanded attention on the tensor cores (bf16).
//
//   P = exp(scale S - lse),  dP = dO V^T,  dS = P (dP - delta),  delta = rowsum(dO O) = rowsum(P dP)
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO
//
// Two kernels, so that every sum has one owner and a fixed order: one holds a tile of queries and walks the keys (dQ),
// one holds a tile of keys and walks its head group's queries (dK, dV, with the scores transposed so that a thread is
// a key).  Both recompute S and dP: 7 products a tile pair instead of the 5 of a kernel that adds dQ up atomically.
// S, dP and the sums live in TMEM.  P and dS go back over S and dP as bf16 pairs and are the A operand of the next
// products from there.  One product's tensor-core time covers the other's elementwise work: while the threads turn
// S(i+1) into P, dK(i) and dP(i+1) run; while they turn dP into dS, dV and the next S run.
//
// 8 x 4096 tokens, 16 query and 4 key heads of 128: 0.71 ms for dQ and 0.72 ms for dK and dV (67 % of the tensor cores'
// cycles; 2400 a step for 2048).  dQ took 0.67 ms (54 %, 2080 a step where the products need 1536, and a start of 6000 a
// CTA that the loads of its first tiles take) before it formed delta itself, which saves a pass over dO and o.
//
// Roles (12 warps): warp 0 loads tiles by TMA, warp 1 issues products, warps 2-3 bring lse and delta and blank the
// rows past a ragged end, warps 4-11 do the elementwise work, half of a tile's columns each.
#include "mla_tc.cuh"

namespace gdn {
namespace mla {

namespace {

constexpr int kThreads = 384, kTile = 128;
constexpr uint32_t kBlock = 16384;      // 128 rows x 64 columns of bf16

struct Params {
    AttnArgs a;
    CUtensorMap qn, qr, dO, kn, kr, v;   // boxes: the held side 128 rows, the walked side as many as a step takes
    int nb, vb;                          // 64-column blocks of dn, dv
    int tiles;                           // tiles of the held side in the longest sequence
    int starve;                          // failure-path test hook: a step whose K (for dQ) or Q is announced, but never loaded
};

// 16-value steps of block c of a query or key
__device__ __forceinline__ int block_steps(const Params& p, int c)
{
    return c < p.nb ? (min(64, p.a.s.dn - 64 * c) + 15) >> 4 : (p.a.s.dr + 15) >> 4;
}
// columns of a product over a query's or key's whole width
__device__ __forceinline__ int width16(const Params& p)
{
    return p.a.s.dr > 0 ? 64 * p.nb + ((p.a.s.dr + 15) & ~15) : (p.a.s.dn + 15) & ~15;
}

// 8 scaled columns of a row of sums as bf16
__device__ __forceinline__ uint4 pack8(const float* x, float f)
{
    return make_uint4(pack_bf16(x[0] * f, x[1] * f), pack_bf16(x[2] * f, x[3] * f), pack_bf16(x[4] * f, x[5] * f),
                      pack_bf16(x[6] * f, x[7] * f));
}

// ================================================================ dQ: a tile of queries walks the keys
//
// dO is an operand from TMEM for the whole walk (products with both operands in shared memory are bound by its 128 bytes
// a cycle); it gets there by way of the third K stage.  Where dQ leaves 64 columns, dS has its own (OWN), so that the next
// tile's dP runs while this one's is turned into dS; else it goes back over dP.
//
// A CTA takes delta = dO . o from the rows of dO that it holds and hands it to the pass over the keys.  That sum carries
// o's rounding, which counts where few keys share a weight of one: dP - delta cancels.
// sum_j P dP is the same number without it.  A tile that walks at most kTwice key tiles takes that sum in a first walk.
// A longer one walks with dO . o: by how much that was off its rows' sums of dS say afterwards, which are zero by the
// exact delta.  The pass over the keys gets the corrected one.  dQ is off by that much times sum_j P K.  dS's own rounding
// to bf16 is off by 2^-9 sum_j |dS| at most; where a tile's rows lack more than that (in squares over the rows), few keys
// take their weight and the tile walks again, by the corrected delta.  The sum of |dS| is twice that over every other key.
// Training steps of 8 x 4096 tokens (6 documents up to 1900) by the standard deviation of the scores, us: 1.5: 1867 (306),
// 3: 1905 (308), 4.5: 1991 (319), 6: 2273 (343), 12: 2521 (359); without the sums and the question 7 (1) less.

constexpr int kTwice = 2;
constexpr float kOff = 0.001953125f;     // 2^-9

// the sum of the products of 8 pairs of bf16
__device__ __forceinline__ float dot8(const uint4& x, const uint4& y)
{
    const uint32_t u[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
    float even = 0.f, odd = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        even += __uint_as_float(u[i] << 16) * __uint_as_float(v[i] << 16);
        odd += __uint_as_float(u[i] & 0xffff0000u) * __uint_as_float(v[i] & 0xffff0000u);
    }
    return even + odd;
}

struct SharedQ {
    uint64_t q_full, a_full, k_full[3], k_empty[3], v_full[2], v_empty[2], k_last[2], k_fixed[2], s_full, s_read, dp_full, dp_read,
        ds_full, ds_empty, dq_full, verdict, drain;
    float part[2][kTile];        // a row's sums from each half of the columns
    uint32_t tmem, gave_up, again;
};

// KB: 64-column blocks of a query or key (the position block among them); KS, VS: stages of K and V.  A key tile is held
// from its scores to its share of dQ, a step later, so K needs three for a load to be ahead
template <int KB, int KS, int VS>
__global__ void __launch_bounds__(kThreads, 1) dq_tc_kernel(const __grid_constant__ Params p)
{
    extern __shared__ unsigned char raw[];
    __shared__ SharedQ S;
    const AttnArgs& a = p.a;
    const gdn_mla_attn_t& s = a.s;
    const int h = blockIdx.x % s.H, b = blockIdx.y, g = h / (s.H / s.Hkv);
    const int q0 = (p.tiles - 1 - (int)(blockIdx.x / s.H)) * kTile;     // the longest walks first
    const Rows rq = rows_of(a.cu_q, b, s.Tq, s.Nq), rk = rows_of(a.cu_k, b, s.Tk, s.Nk);
    cudaTriggerProgrammaticLaunchCompletion();     // the pass over the keys may set up on the SMs that fall free
    if (q0 >= rq.n) return;
    const int off = rk.n - rq.n;
    const int end = s.causal ? min(rk.n, min(q0 + kTile, rq.n) + off) : rk.n;
    const int n = end > 0 ? (end + kTile - 1) / kTile : 0;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    constexpr bool OWN = KB < 3;
    const uint32_t qs = smem_u32(sm), ks = qs + KB * kBlock, vs = ks + KS * KB * kBlock;
    static_assert(KS == 3, "");
    const uint32_t dos = KB == 1 ? vs + VS * p.vb * kBlock : ks + 2 * KB * kBlock;   // one block is too narrow for it

    if (warp == 0) {
        if (elect_one()) {
            for (uint64_t* x : {&S.q_full, &S.k_last[0], &S.k_last[1], &S.s_full, &S.dp_full, &S.ds_empty, &S.dq_full, &S.drain})
                mbar_init(x, 1);
            for (int i = 0; i < KS; i++)
                for (uint64_t* x : {&S.k_full[i], &S.k_empty[i]}) mbar_init(x, 1);
            for (int i = 0; i < VS; i++)
                for (uint64_t* x : {&S.v_full[i], &S.v_empty[i]}) mbar_init(x, 1);
            mbar_init(&S.k_fixed[0], 64);
            mbar_init(&S.k_fixed[1], 64);
            mbar_init(&S.a_full, 8);
            mbar_init(&S.s_read, 8);
            mbar_init(&S.dp_read, 8);
            mbar_init(&S.ds_full, 8);
            mbar_init(&S.verdict, 8);
            fence_mbar_init();
            S.gave_up = S.again = 0;
        }
    } else if (warp == 1) {
        tmem_alloc(&S.tmem, 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    volatile uint32_t* gave_up = &S.gave_up;
    const bool ragged = rk.n % kTile != 0 && n == (rk.n + kTile - 1) / kTile;   // the last key tile has rows to blank
    // Steps are counted through both walks, n each.  `twice`: there are two, and the first forms delta alone.  Else each
    // role asks at the first one's end whether there is a second.
    const bool twice = n <= kTwice;
    const int known = twice ? 2 * n : n;
    const auto again = [&] {
        wait_for(&S.verdict, 0, gave_up);
        return !*gave_up && *(volatile uint32_t*)&S.again;
    };
    // TMEM columns of S, dP, dQ, dO as bf16 pairs, and dS likewise: a half's 32 columns kDsHalf apart
    constexpr uint32_t TS = 0, TP = 128, TQ = 256, TD = 256 + 64 * KB, TE = OWN ? TD + 64 : TP, kDsHalf = OWN ? 32 : 64;
    static_assert(TD + (OWN ? 128 : 64) <= 512, "");

    if (warp == 0) {
        if (elect_one() && n > 0) {
            const bool rope = s.dr > 0;
            mbar_arrive_expect_tx(&S.q_full, (KB + p.vb) * kBlock);
            for (int c = 0; c < p.nb; c++) tma_load_3d(qs + c * kBlock, &p.qn, &S.q_full, 64 * c, h, rq.first + q0);
            if (rope) tma_load_3d(qs + p.nb * kBlock, &p.qr, &S.q_full, 0, h, rq.first + q0);
            for (int c = 0; c < p.vb; c++) tma_load_3d(dos + c * kBlock, &p.dO, &S.q_full, 64 * c, h, rq.first + q0);
            int kdone = 0, vdone = 0;
            for (int j = 0, to = known; j < to; j++) {
                const int ks_ = j % KS, vs_ = j % VS, walk = j >= n, row = rk.first + (walk ? j - n : j) * kTile;
                if (KB > 1 && j == 2) wait_for(&S.a_full, 0, gave_up);      // dO has left the stage
                if (!wait_for(&S.k_empty[ks_], ((j / KS) & 1) ^ 1, gave_up) || *gave_up) break;
                uint64_t* bar = ragged && (j == n - 1 || j == 2 * n - 1) ? &S.k_last[walk] : &S.k_full[ks_];   // to the warps that blank rows
                mbar_arrive_expect_tx(bar, KB * kBlock);
                const uint32_t d = ks + ks_ * KB * kBlock;
                if (j != p.starve) {
                    for (int c = 0; c < p.nb; c++) tma_load_3d(d + c * kBlock, &p.kn, bar, 64 * c, g, row);
                    if (rope) tma_load_3d(d + p.nb * kBlock, &p.kr, bar, 0, 0, row);
                }
                if (bar != &S.k_full[ks_]) mbar_arrive(&S.k_full[ks_]);     // which keeps count of its stage's uses
                kdone = j + 1;
                if (!wait_for(&S.v_empty[vs_], ((j / VS) & 1) ^ 1, gave_up) || *gave_up) break;
                mbar_arrive_expect_tx(&S.v_full[vs_], p.vb * kBlock);
                for (int c = 0; c < p.vb; c++)
                    tma_load_3d(vs + (vs_ * p.vb + c) * kBlock, &p.v, &S.v_full[vs_], 64 * c, g, row);
                vdone = j + 1;
                if (j == n - 1 && !twice && again()) to = 2 * n;
            }
            if (*gave_up) {   // a wait expired: the loads in flight land before the CTA ends
                mbar_wait(&S.q_full, 0, nullptr, kDrainNs);
                for (int j = max(0, kdone - KS); j < kdone; j++) {
                    mbar_wait(&S.k_full[j % KS], (j / KS) & 1, nullptr, kDrainNs);
                    if (ragged && (j == n - 1 || j == 2 * n - 1)) mbar_wait(&S.k_last[j >= n], 0, nullptr, kDrainNs);
                }
                for (int j = max(0, vdone - VS); j < vdone; j++) mbar_wait(&S.v_full[j % VS], (j / VS) & 1, nullptr, kDrainNs);
            }
        }
    } else if (warp == 1) {
        if (elect_one() && n > 0) {
            const uint32_t id_s = idesc_bf16(128, 128, false, false), id_q = idesc_bf16(128, width16(p), false, true);
            const uint64_t kmajor = sdesc(0, 16u, 1024u), nmajor = sdesc(0, kBlock, 1024u);
            int steps[KB];
#pragma unroll
            for (int c = 0; c < KB; c++) steps[c] = block_steps(p, c);
            const int vsteps = (s.dv + 15) >> 4;
            auto scores = [&](int j) {
                wait_for(&S.k_full[j % KS], (j / KS) & 1, gave_up);
                if (ragged && (j == n - 1 || j == 2 * n - 1)) wait_for(&S.k_fixed[j >= n], 0, gave_up);
                tc_fence_after();
                if (!*gave_up) {
                    const uint64_t q = kmajor + at_desc(qs), k = kmajor + at_desc(ks + (j % KS) * KB * kBlock);
#pragma unroll
                    for (int c = 0; c < KB; c++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (e < steps[c])
                                mma_bf16(tmem + TS, q + c * (kBlock >> 4) + 2 * e, k + c * (kBlock >> 4) + 2 * e, id_s,
                                         (c | e) ? 1u : 0u);
                }
                mma_commit(&S.s_full);
            };
            auto dprobs = [&](int j) {
                wait_for(&S.v_full[j % VS], (j / VS) & 1, gave_up);
                tc_fence_after();
                if (!*gave_up) {
                    const uint64_t v = kmajor + at_desc(vs + (j % VS) * p.vb * kBlock);
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (e < vsteps)
                            mma_bf16_ts(tmem + TP, tmem + TD + 8 * e, v + (e >> 2) * (kBlock >> 4) + 2 * (e & 3), id_s, e ? 1u : 0u);
                }
                mma_commit(&S.dp_full);
                mma_commit(&S.v_empty[j % VS]);
            };
            wait_for(&S.q_full, 0, gave_up);
            wait_for(&S.a_full, 0, gave_up);
            tc_fence_after();
            scores(0);
            dprobs(0);
            for (int j = 0, to = known, start = twice ? n : 0; j < to; j++) {     // start: of the walk that forms dQ
                wait_for(&S.s_read, j & 1, gave_up);
                if (j + 1 < to) scores(j + 1);
                if (OWN) {
                    wait_for(&S.dp_read, j & 1, gave_up);
                    if (j + 1 < to) dprobs(j + 1);
                }
                wait_for(&S.ds_full, j & 1, gave_up);
                tc_fence_after();
                if (j >= start && !*gave_up) {
                    const uint64_t k = nmajor + at_desc(ks + (j % KS) * KB * kBlock);
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        mma_bf16_ts(tmem + TQ, tmem + TE + (e >> 2) * kDsHalf + 8 * (e & 3), k + 128 * e, id_q, (j > start || e) ? 1u : 0u);
                }
                mma_commit(&S.k_empty[j % KS]);
                if (OWN) mma_commit(&S.ds_empty);
                if (!OWN && j + 1 < to) dprobs(j + 1);
                if (j == n - 1 && !twice && again()) {
                    to = 2 * n;
                    start = n;
                    scores(n);
                    dprobs(n);
                }
            }
            mma_commit(&S.dq_full);
            if (*gave_up) {   // the products in flight end before TMEM is freed
                mma_commit(&S.drain);
                mbar_wait(&S.drain, 0, nullptr, kDrainNs);
            }
        }
    } else if (warp < 4) {
        if (ragged)
            for (int walk = 0; walk < 2; walk++) {
                if (walk && !twice && !again()) break;
                const int j = walk * n + n - 1, valid = rk.n - (n - 1) * kTile, bad = kTile - valid;
                wait_for(&S.k_last[walk], 0, gave_up);
                for (int c = 0; c < KB; c++) {
                    unsigned char* k = sm + (ks - qs) + ((j % KS) * KB + c) * kBlock + valid * 128;
                    for (int e = tid - 64; e < bad * 8; e += 64) *reinterpret_cast<uint4*>(k + e * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                mbar_arrive(&S.k_fixed[walk]);
            }
    } else {
        const int half = (warp - 4) >> 2, quad = warp & 3, row = q0 + quad * 32 + lane;
        const uint32_t base = tmem + ((uint32_t)quad << 21);
        const bool mine = row < rq.n;
        const long long at = (long long)h * s.Nq + rq.first + (mine ? row : 0);
        const float c = s.scale * kLog2e;
        const float lse = mine ? a.lse[at] : -INFINITY;
        float delta = 0.f;
        if (n > 0) {     // this half's 64 columns of the row of dO into TMEM, and their share of dO . o
            uint4 o[8];
#pragma unroll
            for (int e = 0; e < 8; e++) o[e] = make_uint4(0, 0, 0, 0);
            if (mine && !twice) {
                const __nv_bfloat16* y = (const __nv_bfloat16*)a.o + ((long long)(rq.first + row) * s.H + h) * s.dv + 64 * half;
#pragma unroll
                for (int e = 0; e < 8; e++)
                    if (64 * half + 8 * e < s.dv) o[e] = __ldg(reinterpret_cast<const uint4*>(y + 8 * e));
            }
            wait_for(&S.q_full, 0, gave_up);
            __syncwarp();
            if (half < p.vb) {
                uint32_t x[32];
#pragma unroll
                for (int e = 0; e < 8; e++) {
                    const uint4 v = *reinterpret_cast<const uint4*>(sm + (dos - qs) + half * kBlock + sw128(quad * 32 + lane, 8 * e));
                    x[4 * e] = v.x;
                    x[4 * e + 1] = v.y;
                    x[4 * e + 2] = v.z;
                    x[4 * e + 3] = v.w;
                    delta += dot8(v, o[e]);
                }
                __syncwarp();
                tmem_st32(base + TD + 32 * half, x);
            }
            if (!twice) {
                S.part[half][quad * 32 + lane] = mine ? delta : 0.f;    // another's dO, or none
                group_sync(1, 256);
                delta = S.part[0][quad * 32 + lane] + S.part[1][quad * 32 + lane];
                group_sync(1, 256);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.a_full);
        }
        const float lower = lse == -INFINITY ? -INFINITY : -lse * kLog2e;       // a row without keys: weights of zero
        // a query that sees one key has a constant weight: no gradient, not the difference of two roundings
        int last = !mine ? -1 : s.causal ? min(rk.n - 1, row + off) : rk.n - 1;
        if (last == 0) last = -1;
        const int calm = min(rk.n - 1, s.causal ? q0 + quad * 32 + off : rk.n - 1);
        const uint64_t c2 = pack2(c, c), l2 = pack2(lower, lower);
        uint64_t d2 = pack2(twice ? 0.f : -delta, twice ? 0.f : -delta), sum2[2] = {0, 0};
        float size = 0.f;     // of the dS that sum2 adds up: every other one's
        // this row's sum over both halves' columns
        const auto row_total = [&](float x) {
            S.part[half][quad * 32 + lane] = x;
            group_sync(1, 256);
            const float t = S.part[0][quad * 32 + lane] + S.part[1][quad * 32 + lane];
            group_sync(1, 256);
            return t;
        };
        for (int j = 0, to = known; j < to; j++) {
            uint32_t x[64];
            wait_for(&S.s_full, j & 1, gave_up);
            __syncwarp();
            tc_fence_after();
            tmem_ld32(base + TS + 64 * half, x);
            tmem_ld32(base + TS + 64 * half + 32, x + 32);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.s_read);
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
                float u, w;
                unpack2(fma2(pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2, l2), u, w);
                x[i] = __float_as_uint(fast_exp2(u));
                x[i + 1] = __float_as_uint(fast_exp2(w));
            }
            const int j0 = (j < n ? j : j - n) * kTile + 64 * half;
            const bool masked = j0 + 63 > calm || calm <= 0;
            wait_for(&S.dp_full, j & 1, gave_up);
            __syncwarp();
            tc_fence_after();
            uint32_t y[64];
            tmem_ld32(base + TP + 64 * half, y);
            tmem_ld32(base + TP + 64 * half + 32, y + 32);
            tmem_wait_ld();
            if (OWN) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.dp_read);
                __syncwarp();
                if (j > 0) {     // the last tile's dS has been used
                    wait_for(&S.ds_empty, (j - 1) & 1, gave_up);
                    __syncwarp();
                    tc_fence_after();
                }
            }
#pragma unroll
            for (int i0 = 0; i0 < 64; i0 += 32) {
                uint32_t z[16];
#pragma unroll
                for (int i = i0; i < i0 + 32; i += 2) {
                    // P (dP - delta), or P dP in the first walk
                    uint64_t t = mul2(pack2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                      add2(pack2(__uint_as_float(y[i]), __uint_as_float(y[i + 1])), d2));
                    if (masked) {
                        float u, w;
                        unpack2(t, u, w);
                        t = pack2(j0 + i <= last ? u : 0.f, j0 + i + 1 <= last ? w : 0.f);
                    }
                    sum2[(i >> 1) & 1] = add2(sum2[(i >> 1) & 1], t);
                    float u, w;
                    unpack2(t, u, w);
                    size += fabsf(u);
                    z[(i - i0) >> 1] = pack_bf16(u, w);
                }
                if (!twice || j >= n) tmem_st16u(base + TE + kDsHalf * half + (i0 >> 1), z);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.ds_full);
            if (j == n - 1) {     // the sum of P dP is delta; that of dS is what delta lacks, as P's rows add up to one
                float even, odd;
                unpack2(add2(sum2[0], sum2[1]), even, odd);
                const float lacks = row_total(even + odd);
                delta = twice ? lacks : delta + lacks;
                d2 = pack2(-delta, -delta);
                if (!twice) {
                    const float all = row_total(2.f * size), off = lacks / kOff;
                    float over = mine ? off * off - all * all : 0.f;     // over the tile's rows
                    if (!(fabsf(over) < INFINITY)) over = 0.f;           // a row of NaN has no say
#pragma unroll
                    for (int m = 16; m; m >>= 1) over += __shfl_xor_sync(0xffffffffu, over, m);
                    S.part[half][quad * 32 + lane] = over;
                    group_sync(1, 256);
                    const bool more = S.part[0][0] + S.part[0][32] + S.part[0][64] + S.part[0][96] > 0.f;
                    if (more) to = 2 * n;
                    if (tid == 128) S.again = more;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.verdict);
                }
            }
        }
        if (n > 0) {
            wait_for(&S.dq_full, 0, gave_up);
            __syncwarp();
            tc_fence_after();
        }
        if (mine && half == 0) a.delta[at] = delta;     // for the pass over the keys
        __nv_bfloat16* on = (__nv_bfloat16*)a.dqn.p + (long long)(rq.first + row) * a.dqn.tok + (long long)h * a.dqn.head;
        __nv_bfloat16* op = (__nv_bfloat16*)a.dqr.p + (long long)(rq.first + row) * a.dqr.tok + (long long)h * a.dqr.head;
#pragma unroll 1
        for (int i = 16 * half; i < 64 * KB; i += 32) {     // the two halves take 16 columns in turn
            float o[16];
            __syncwarp();
            if (n > 0) {
                tmem_ld16(base + TQ + i, o);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 16; e++) o[e] = 0.f;
            }
            if (!mine) continue;
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
                const int col = i + e, rcol = col - 64 * p.nb;
                if (rcol < 0) {
                    if (col < s.dn) *reinterpret_cast<uint4*>(on + col) = pack8(o + e, s.scale);
                } else if (rcol < s.dr) {
                    *reinterpret_cast<uint4*>(op + rcol) = pack8(o + e, s.scale);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && *gave_up) atomicExch(a.status, kDevTimeout);
}

// ================================================================ dK, dV: a tile of keys walks the queries

template <int NQ>
struct SharedK {
    uint64_t kv_full, q_full[3], q_empty[3], do_full[2], do_empty[2], st_full[2], st_empty[2], s_full, p_full, dp_full, ds_full,
        acc_full, drain;
    alignas(16) float lower[2][NQ];     // -lse log2(e), minus infinity for a row that adds nothing
    alignas(16) float delta[2][NQ];     // -delta
    uint32_t tmem, gave_up;
};

// NQ: queries a step; TMEM holds two NQ columns of scores, dV and dK.  QS: stages of Q, held from the scores to dK; dO and
// the statistics have two
template <int KB, int NQ, int QS>
__global__ void __launch_bounds__(kThreads, 1) dkv_tc_kernel(const __grid_constant__ Params p)
{
    extern __shared__ unsigned char raw[];      // tiles (1024-byte aligned), then the shared state
    const AttnArgs& a = p.a;
    const gdn_mla_attn_t& s = a.s;
    const int g = blockIdx.x % s.Hkv, b = blockIdx.y, G = s.H / s.Hkv;
    const int k0 = (int)(blockIdx.x / s.Hkv) * kTile;       // under the causal mask the first keys have most queries
    const Rows rq = rows_of(a.cu_q, b, s.Tq, s.Nq), rk = rows_of(a.cu_k, b, s.Tk, s.Nk);
    cudaTriggerProgrammaticLaunchCompletion();     // the sum over the heads follows likewise
    // launched as a dependent of dQ's kernel, of which it reads delta alone; a CTA waits for it even if it reads none, so that
    // its end is the end of both
    if (k0 >= rk.n) {
        cudaGridDependencySynchronize();
        return;
    }
    if (smem_u32(raw) & 1023) {     // never so without static shared memory; the tiles below would not fit otherwise
        if (threadIdx.x == 0) atomicExch(a.status, kDevLayout);
        cudaGridDependencySynchronize();
        return;
    }
    const int off = rk.n - rq.n;
    const int first = s.causal ? max(0, k0 - off) / NQ : 0;                // the first step whose queries see key k0
    const int per = max(0, (rq.n + NQ - 1) / NQ - first), n = per * G;     // steps a head, in all
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    unsigned char* sm = raw;
    constexpr uint32_t kStep = NQ * 128;                                   // bytes of a 64-column block of a step
    SharedK<NQ>& S = *reinterpret_cast<SharedK<NQ>*>(sm + (KB + p.vb) * kBlock + (QS * KB + 2 * p.vb) * kStep);
    const uint32_t ks = smem_u32(sm), vs = ks + KB * kBlock, qs = vs + p.vb * kBlock, dos = qs + QS * KB * kStep;

    if (warp == 0) {
        if (elect_one()) {
            for (uint64_t* x : {&S.kv_full, &S.s_full, &S.dp_full, &S.acc_full, &S.drain}) mbar_init(x, 1);
            for (int i = 0; i < QS; i++)
                for (uint64_t* x : {&S.q_full[i], &S.q_empty[i]}) mbar_init(x, 1);
            for (int i = 0; i < 2; i++) {
                for (uint64_t* x : {&S.do_full[i], &S.do_empty[i]}) mbar_init(x, 1);
                mbar_init(&S.st_full[i], 64);
                mbar_init(&S.st_empty[i], 8);
            }
            mbar_init(&S.p_full, 8);
            mbar_init(&S.ds_full, 8);
            fence_mbar_init();
            S.gave_up = 0;
        }
    } else if (warp == 1) {
        tmem_alloc(&S.tmem, 512);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    volatile uint32_t* gave_up = &S.gave_up;
    constexpr uint32_t TS = 0, TP = NQ, TV = 2 * NQ, TK = 2 * NQ + 128;    // TMEM columns of S, dP, dV, dK
    constexpr int HC = NQ / 2, KS = NQ / 16;                               // columns a half, 16-query steps

    if (warp == 0) {
        if (elect_one() && n > 0) {
            const bool rope = s.dr > 0;
            mbar_arrive_expect_tx(&S.kv_full, (KB + p.vb) * kBlock);
            for (int c = 0; c < p.nb; c++) tma_load_3d(ks + c * kBlock, &p.kn, &S.kv_full, 64 * c, g, rk.first + k0);
            if (rope) tma_load_3d(ks + p.nb * kBlock, &p.kr, &S.kv_full, 0, 0, rk.first + k0);
            for (int c = 0; c < p.vb; c++) tma_load_3d(vs + c * kBlock, &p.v, &S.kv_full, 64 * c, g, rk.first + k0);
            int qdone = 0, ddone = 0;
            for (int i = 0, h = g * G, t = first; i < n; i++) {
                const int st = i & 1, qst = i % QS;
                const int row = rq.first + t * NQ;
                if (!wait_for(&S.q_empty[qst], ((i / QS) & 1) ^ 1, gave_up) || *gave_up) break;
                mbar_arrive_expect_tx(&S.q_full[qst], KB * kStep);
                const uint32_t q = qs + qst * KB * kStep, d = dos + st * p.vb * kStep;
                if (i != p.starve) {
                    for (int c = 0; c < p.nb; c++) tma_load_3d(q + c * kStep, &p.qn, &S.q_full[qst], 64 * c, h, row);
                    if (rope) tma_load_3d(q + p.nb * kStep, &p.qr, &S.q_full[qst], 0, h, row);
                }
                qdone = i + 1;
                if (!wait_for(&S.do_empty[st], ((i >> 1) & 1) ^ 1, gave_up) || *gave_up) break;
                mbar_arrive_expect_tx(&S.do_full[st], p.vb * kStep);
                for (int c = 0; c < p.vb; c++) tma_load_3d(d + c * kStep, &p.dO, &S.do_full[st], 64 * c, h, row);
                ddone = i + 1;
                if (++t == first + per) {
                    t = first;
                    h++;
                }
            }
            if (*gave_up) {   // a wait expired: the loads in flight land before the CTA ends
                mbar_wait(&S.kv_full, 0, nullptr, kDrainNs);
                for (int i = max(0, qdone - QS); i < qdone; i++) mbar_wait(&S.q_full[i % QS], (i / QS) & 1, nullptr, kDrainNs);
                for (int i = max(0, ddone - 2); i < ddone; i++) mbar_wait(&S.do_full[i & 1], (i >> 1) & 1, nullptr, kDrainNs);
            }
        }
    } else if (warp == 1) {
        if (elect_one() && n > 0) {
            const uint32_t id_s = idesc_bf16(128, NQ, false, false);
            const uint32_t id_v = idesc_bf16(128, (s.dv + 15) & ~15, false, true), id_k = idesc_bf16(128, width16(p), false, true);
            const uint64_t kmajor = sdesc(0, 16u, 1024u), nmajor = sdesc(0, kStep, 1024u);
            int steps[KB];
#pragma unroll
            for (int c = 0; c < KB; c++) steps[c] = block_steps(p, c);
            const int vsteps = (s.dv + 15) >> 4;
            const bool ragged = rq.n % NQ != 0;
            auto scores = [&](int i) {
                wait_for(&S.q_full[i % QS], (i / QS) & 1, gave_up);
                if (ragged && i % per == per - 1) wait_for(&S.st_full[i & 1], (i >> 1) & 1, gave_up);   // rows past the end blanked
                tc_fence_after();
                if (!*gave_up) {
                    const uint64_t k = kmajor + at_desc(ks), q = kmajor + at_desc(qs + (i % QS) * KB * kStep);
#pragma unroll
                    for (int c = 0; c < KB; c++)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (e < steps[c])
                                mma_bf16(tmem + TS, k + c * (kBlock >> 4) + 2 * e, q + c * (kStep >> 4) + 2 * e, id_s,
                                         (c | e) ? 1u : 0u);
                }
                mma_commit(&S.s_full);
            };
            auto dprobs = [&](int i) {
                wait_for(&S.do_full[i & 1], (i >> 1) & 1, gave_up);
                tc_fence_after();
                if (!*gave_up) {
                    const uint64_t v = kmajor + at_desc(vs), d = kmajor + at_desc(dos + (i & 1) * p.vb * kStep);
#pragma unroll
                    for (int e = 0; e < 8; e++)
                        if (e < vsteps)
                            mma_bf16(tmem + TP, v + (e >> 2) * (kBlock >> 4) + 2 * (e & 3), d + (e >> 2) * (kStep >> 4) + 2 * (e & 3),
                                     id_s, e ? 1u : 0u);
                }
                mma_commit(&S.dp_full);
            };
            wait_for(&S.kv_full, 0, gave_up);
            scores(0);
            dprobs(0);
            for (int i = 0; i < n; i++) {
                wait_for(&S.p_full, i & 1, gave_up);
                tc_fence_after();
                if (!*gave_up) {
                    const uint64_t d = nmajor + at_desc(dos + (i & 1) * p.vb * kStep);
#pragma unroll
                    for (int e = 0; e < KS; e++)     // P: the first quarter of S's columns and the third
                        mma_bf16_ts(tmem + TV, tmem + TS + (e >= KS / 2 ? HC + 8 * (e - KS / 2) : 8 * e), d + 128 * e, id_v,
                                    (i | e) ? 1u : 0u);
                }
                mma_commit(&S.do_empty[i & 1]);
                if (i + 1 < n) scores(i + 1);
                wait_for(&S.ds_full, i & 1, gave_up);
                tc_fence_after();
                if (!*gave_up) {
                    const uint64_t q = nmajor + at_desc(qs + (i % QS) * KB * kStep);
#pragma unroll
                    for (int e = 0; e < KS; e++)
                        mma_bf16_ts(tmem + TK, tmem + TP + (e >= KS / 2 ? HC + 8 * (e - KS / 2) : 8 * e), q + 128 * e, id_k,
                                    (i | e) ? 1u : 0u);
                }
                mma_commit(&S.q_empty[i % QS]);
                if (i + 1 < n) dprobs(i + 1);
            }
            mma_commit(&S.acc_full);
            if (*gave_up) {   // the products in flight end before TMEM is freed
                mma_commit(&S.drain);
                mbar_wait(&S.drain, 0, nullptr, kDrainNs);
            }
        }
    } else if (warp < 4) {
        const int t0 = tid - 64;
        cudaGridDependencySynchronize();
        for (int i = 0, h = g * G, t = first; i < n; i++) {
            const int st = i & 1;
            wait_for(&S.st_empty[st], ((i >> 1) & 1) ^ 1, gave_up);
            const long long at = (long long)h * s.Nq + rq.first;
            for (int e = t0; e < NQ; e += 64) {
                const int row = t * NQ + e;
                const float lse = row < rq.n ? a.lse[at + row] : -INFINITY;
                S.lower[st][e] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
                S.delta[st][e] = row < rq.n ? -a.delta[at + row] : 0.f;
            }
            const int valid = rq.n - t * NQ;
            if (valid < NQ) {      // rows past the end hold anything: weights of zero would still meet a NaN
                wait_for(&S.q_full[i % QS], (i / QS) & 1, gave_up);
                wait_for(&S.do_full[st], (i >> 1) & 1, gave_up);
                for (int c = 0; c < KB + p.vb; c++) {
                    const uint32_t from = c < KB ? qs - ks + ((i % QS) * KB + c) * kStep : dos - ks + (st * p.vb + c - KB) * kStep;
                    unsigned char* x = sm + from + valid * 128;
                    for (int e = t0; e < (NQ - valid) * 8; e += 64) *reinterpret_cast<uint4*>(x + e * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
            }
            mbar_arrive(&S.st_full[st]);
            if (++t == first + per) {
                t = first;
                h++;
            }
        }
    } else {
        const int half = (warp - 4) >> 2, quad = warp & 3, key = k0 + quad * 32 + lane;
        const uint32_t base = tmem + ((uint32_t)quad << 21);
        const float c = s.scale * kLog2e;
        const uint64_t c2 = pack2(c, c);
        for (int i = 0, t = first; i < n; i++) {
            const int st = i & 1, q0 = t * NQ + HC * half;
            // column e is seen from q0 + e on; a query that sees one key has a constant weight, and no gradient of it
            const bool masked = s.causal ? q0 + off < k0 + kTile - 1 || q0 + off <= 0 : rk.n == 1;
            const int from = s.causal ? key - off - q0 : 0;
            const int from_s = rk.n == 1 ? NQ : s.causal ? max(from, 1 - off - q0) : 0;
            float x[HC];
            wait_for(&S.st_full[st], (i >> 1) & 1, gave_up);
            wait_for(&S.s_full, i & 1, gave_up);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < HC; e += 16) tmem_ld16(base + TS + HC * half + e, *reinterpret_cast<float(*)[16]>(&x[e]));
            tmem_wait_ld();
#pragma unroll
            for (int e0 = 0; e0 < HC; e0 += 16) {
                uint32_t y[8];
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(&S.lower[st][HC * half + e0 + e]);
                    float* v = &x[e0 + e];
                    unpack2(fma2(pack2(v[0], v[1]), c2, l.x), v[0], v[1]);
                    unpack2(fma2(pack2(v[2], v[3]), c2, l.y), v[2], v[3]);
#pragma unroll
                    for (int f = 0; f < 4; f++) {
                        v[f] = fast_exp2(v[f]);
                        if (masked) v[f] = e0 + e + f >= from ? v[f] : 0.f;
                    }
                    y[e >> 1] = pack_bf16(v[0], v[1]);
                    y[(e >> 1) + 1] = pack_bf16(v[2], v[3]);
                }
                asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(base + TS + HC * half +
                                                                                                         (e0 >> 1)),
                             "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                             : "memory");
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_full);
            wait_for(&S.dp_full, i & 1, gave_up);
            __syncwarp();
            tc_fence_after();
#pragma unroll
            for (int e0 = 0; e0 < HC; e0 += 16) {
                float d[16];
                uint32_t y[8];
                tmem_ld16(base + TP + HC * half + e0, d);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; e += 4) {
                    const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(&S.delta[st][HC * half + e0 + e]);
                    float v[4];
                    unpack2(mul2(pack2(x[e0 + e], x[e0 + e + 1]), add2(pack2(d[e], d[e + 1]), l.x)), v[0], v[1]);
                    unpack2(mul2(pack2(x[e0 + e + 2], x[e0 + e + 3]), add2(pack2(d[e + 2], d[e + 3]), l.y)), v[2], v[3]);
                    if (masked) {
#pragma unroll
                        for (int f = 0; f < 4; f++) v[f] = e0 + e + f >= from_s ? v[f] : 0.f;
                    }
                    y[e >> 1] = pack_bf16(v[0], v[1]);
                    y[(e >> 1) + 1] = pack_bf16(v[2], v[3]);
                }
                asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(base + TP + HC * half +
                                                                                                         (e0 >> 1)),
                             "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                             : "memory");
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&S.ds_full);
                mbar_arrive(&S.st_empty[st]);
            }
            if (++t == first + per) t = first;
        }
        if (n > 0) {
            wait_for(&S.acc_full, 0, gave_up);
            __syncwarp();
            tc_fence_after();
        }
        const bool mine = key < rk.n;
        __nv_bfloat16* ov = (__nv_bfloat16*)a.dv.p + (long long)(rk.first + key) * a.dv.tok + (long long)g * a.dv.head;
        __nv_bfloat16* on = (__nv_bfloat16*)a.dkn.p + (long long)(rk.first + key) * a.dkn.tok + (long long)g * a.dkn.head;
        float* op = a.dkr_part + ((long long)g * s.Nk + rk.first + key) * s.dr;
#pragma unroll 1
        for (int i = 16 * half; i < 128 + 64 * KB; i += 32) {     // the two halves take 16 columns in turn
            float o[16];
            __syncwarp();
            if (n > 0) {
                tmem_ld16(base + TV + i, o);
                tmem_wait_ld();
            } else {
#pragma unroll
                for (int e = 0; e < 16; e++) o[e] = 0.f;
            }
            if (!mine) continue;
#pragma unroll
            for (int e = 0; e < 16; e += 8) {
                const int vcol = i + e, col = vcol - 128, rcol = col - 64 * p.nb;
                if (col < 0) {
                    if (vcol < s.dv) *reinterpret_cast<uint4*>(ov + vcol) = pack8(o + e, 1.f);
                } else if (rcol < 0) {
                    if (col < s.dn) *reinterpret_cast<uint4*>(on + col) = pack8(o + e, s.scale);
                } else if (rcol < s.dr) {
                    *reinterpret_cast<float4*>(op + rcol) =
                        make_float4(o[e] * s.scale, o[e + 1] * s.scale, o[e + 2] * s.scale, o[e + 3] * s.scale);
                    *reinterpret_cast<float4*>(op + rcol + 4) =
                        make_float4(o[e + 4] * s.scale, o[e + 5] * s.scale, o[e + 6] * s.scale, o[e + 7] * s.scale);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if (tid == 0 && *gave_up) atomicExch(a.status, kDevTimeout);
}

bool maps(Params& p, int q_rows, int k_rows)
{
    const AttnArgs& a = p.a;
    const gdn_mla_attn_t& s = a.s;
    const gdn_mla_view_t dO = {const_cast<void*>(a.dO), (long long)s.H * s.dv, s.dv};
    // a side without rows is never loaded
    if (s.Nq > 0 && (!view_map(&p.qn, a.qn, s.Nq, s.H, s.dn, q_rows) || !view_map(&p.dO, dO, s.Nq, s.H, s.dv, q_rows) ||
                     (s.dr > 0 && !view_map(&p.qr, a.qr, s.Nq, s.H, s.dr, q_rows))))
        return false;
    return s.Nk == 0 || (view_map(&p.kn, a.kn, s.Nk, s.Hkv, s.dn, k_rows) && view_map(&p.v, a.v, s.Nk, s.Hkv, s.dv, k_rows) &&
                         (s.dr == 0 || view_map(&p.kr, a.kr, s.Nk, 1, s.dr, k_rows)));
}

template <int KB, int KS, int VS>
cudaError_t run_dq(Params& p, cudaStream_t st)
{
    if (!maps(p, kTile, kTile)) return cudaErrorInvalidValue;
    p.tiles = (p.a.s.Tq + kTile - 1) / kTile;
    const size_t bytes = 1024 + (size_t)(KB + KS * KB + VS * p.vb + (KB == 1 ? p.vb : 0)) * kBlock;
    const cudaError_t e = cudaFuncSetAttribute(dq_tc_kernel<KB, KS, VS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    dq_tc_kernel<KB, KS, VS><<<dim3((unsigned)p.a.s.H * p.tiles, p.a.s.B), kThreads, bytes, st>>>(p);
    return cudaGetLastError();
}

template <int KB, int NQ, int QS>
cudaError_t run_dkv(Params& p, cudaStream_t st)
{
    if (!maps(p, NQ, kTile)) return cudaErrorInvalidValue;
    p.tiles = (p.a.s.Tk + kTile - 1) / kTile;
    // (without static shared memory the dynamic part begins 1024-byte aligned)
    const size_t bytes = (size_t)(KB + p.vb) * kBlock + (size_t)(QS * KB + 2 * p.vb) * NQ * 128 + sizeof(SharedK<NQ>);
    const cudaError_t e = cudaFuncSetAttribute(dkv_tc_kernel<KB, NQ, QS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.a.s.Hkv * p.tiles, p.a.s.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.a.s.Tq > 0 ? 1 : 0;      // after dQ's kernel
    return cudaLaunchKernelEx(&cfg, dkv_tc_kernel<KB, NQ, QS>, p);
}

}  // namespace

cudaError_t launch_attn_bwd_tc(const AttnArgs& a, cudaStream_t st)
{
    const gdn_mla_attn_t& s = a.s;
    Params p;
    memset(&p, 0, sizeof(p));
    p.a = a;
    p.starve = test_starve_chunk();
    p.nb = (s.dn + 63) / 64;
    p.vb = (s.dv + 63) / 64;
    const int kb = p.nb + (s.dr > 0 ? 1 : 0);
    cudaError_t e = cudaSuccess;
    if (s.Tq > 0) e = kb == 1 ? run_dq<1, 3, 2>(p, st) : kb == 2 ? run_dq<2, 3, 2>(p, st) : run_dq<3, 3, 1>(p, st);
    if (e == cudaSuccess && s.Tk > 0) {
        // dV and 192 columns of dK leave 192 for S and dP
        e = kb == 1 ? run_dkv<1, 128, 3>(p, st) : kb == 2 ? run_dkv<2, 128, 3>(p, st) : run_dkv<3, 96, 2>(p, st);
        if (e == cudaSuccess && s.dr > 0) e = launch_dkr(a, st);
    }
    return e;
}

}  // namespace mla
}  // namespace gdn
