// mla_decode_tc.cu -- the decode worker on the tensor cores (bf16).
//
// Scores and outputs are formed transposed, S^T = K Q^T and O^T = V^T P^T, so that the cache's rows are the tall side
// of every product (M = 64 rows, M = 128 latent columns) and the few query rows its narrow one (N = 16..80): with 16
// heads nothing is padded.  The same shared-memory tile serves both products, as a K-major operand of the first and,
// its columns read as rows, as an MN-major operand of the second: each cache byte crosses HBM once.
//
// Roles of a CTA (one per SM, 12 warps): warp 0 streams the cache by TMA through a ring of 64 rows x 128 columns
// pieces (page by page: a page's rows are one box); warp 1 issues the scores' products and warp 2 the outputs', each
// waiting for its own operands only, so that the next tiles' scores run ahead of this tile's outputs; warp 3 lays the
// queries out; warps 4-11 do the softmax.  The softmax keeps a running maximum of each query row but lowers scores by an
// old one until a score exceeds it by 2^16: exp2 and fp32 hold that range, P's bf16 rounding is relative, and the outputs
// in TMEM are rescaled only then (rarely after a sequence's first tile).
//
// HBM bounds it while the query rows fit one group: 8 x 32768 rows of 512 + 64 values under 16 heads take 57 us
// (302 MB, 5.3 TB/s; 3250 cycles a 64-row tile are 22.7 bytes a cycle and SM, the card's rate, the rest start and end).
// A call of 160 rows in two groups takes 88 us where the bytes alone need 20: less than two tiles fit beside 92 KB
// of queries, so a tile's load waits for the products of the one before it.
#include "mla_decode_common.cuh"
#include "mla_tc.cuh"

namespace gdn {
namespace mla {

namespace {

constexpr int kThreads = 384, kSoft = 256;   // kSoft of them do the softmax
constexpr int kMaxPairs = 16, kMaxRope = 4, kMaxCols = kDecodeRows;
constexpr uint32_t kPairBytes = 16384, kBlockBytes = 8192;
// buffers of weights: with 80 query rows a second one would take the room of half a pair of cache blocks
template <int NC> constexpr int kWeights = NC > 64 ? 1 : 2;
constexpr float kSlack = 16.f;          // log2 by which a score may exceed the maximum it is lowered by

struct Params {
    DecodeArgs a;
    CUtensorMap map, qc, qr;     // the cache; the queries as rows (b, t, h), where their strides allow that
    int q_tma;
    int nb, np;                  // 64-column blocks of the latent, pairs of them
    int npair, nrope;            // ring sizes
    int box;                     // rows of a TMA box: divides the page and the tile
    int total_rows;              // rows of the cache; a box that starts there reads as zeros
    int starve;                  // failure-path test hook: a worker's tile that is announced, but never loaded (-1: none)
    uint32_t rope_off, q_off, p_off;   // shared memory, from the pair ring's start
};

struct Shared {
    uint64_t pair_full[kMaxPairs], pair_empty[kMaxPairs], rope_full[kMaxRope], rope_empty[kMaxRope];
    uint64_t q_full, q_empty, s_full[2], p_full[2], p_empty[2], o_full, drain[2];
    alignas(16) float top[kMaxCols];   // read four at a time
    float keep[kMaxCols], up[kMaxCols], red[4][kMaxCols], back[kMaxCols];
    uint32_t tmem, gave_up;
    int b, tile, total;
};

// the worker's run of tiles: sequence b's tiles [tile, to), then the next sequence's
struct Run {
    const Deal& d;
    int b, tile, to, n, tiles, left;

    __device__ __forceinline__ Run(const Deal& deal, int b0, int tile0, int count) : d(deal), b(b0), tile(tile0), left(count)
    {
        load();
    }
    __device__ __forceinline__ void load()
    {
        n = tiles = to = 0;
        while (left > 0 && b < d.B) {
            n = d.rows(b);
            tiles = (n + kDecodeTile - 1) / kDecodeTile;
            if (tiles > tile) break;
            b++;
            tile = 0;
        }
        to = min(tiles, tile + left);
    }
    // to the next tile; true if that begins another piece
    __device__ __forceinline__ bool step()
    {
        left--;
        if (++tile < to) return false;
        b++;
        tile = 0;
        load();
        return true;
    }
};

__device__ __forceinline__ uint32_t lane_base(uint32_t tmem, int quad) { return tmem + ((uint32_t)quad << 21); }

__device__ __forceinline__ void tmem_ld4(uint32_t addr, float (&v)[4])
{
    uint32_t* r = reinterpret_cast<uint32_t*>(v);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
template <int NC>
__device__ __forceinline__ void load_cols(uint32_t addr, float (&v)[NC])
{
#pragma unroll
    for (int c = 0; c + 16 <= NC; c += 16) tmem_ld16(addr + c, *reinterpret_cast<float(*)[16]>(&v[c]));
#pragma unroll
    for (int c = NC / 16 * 16; c < NC; c += 4) tmem_ld4(addr + c, *reinterpret_cast<float(*)[4]>(&v[c]));
    tmem_wait_ld();
}

// 16 bytes to shared memory, zeros if `in` is false
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in)
{
    const uint32_t bytes = in ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

template <int NC>
__global__ void __launch_bounds__(kThreads, 1) decode_tc_kernel(const __grid_constant__ Params p)
{
    extern __shared__ unsigned char raw[];
    __shared__ Shared S;
    unsigned char* sm = (unsigned char*)(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    const DecodeArgs& a = p.a;
    const gdn_mla_cache_t& s = a.s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x, group = blockIdx.y;
    const int row0 = group * a.rows, rows = min(a.rows, s.T * s.H - row0);
    const Deal deal{a.len, s.B, s.maxpages * s.page};
    const bool rope = s.dr > 0;
    constexpr uint32_t kCols = NC <= 16 ? 128 : NC <= 32 ? 256 : 512;   // 2 score buffers + 4 output blocks

    if (warp == 0) {
        const int all = deal_tiles(deal), share = deal_share(all, a.ctas);
        const int start = min((long long)share * cta, (long long)all);
        int b, tile;
        deal_find(deal, start, b, tile);
        if (lane == 0) {
            S.b = b;
            S.tile = tile;
            S.total = min(share, all - start);
        }
    } else if (warp == 1) {
        tmem_alloc(&S.tmem, kCols);
    } else if (warp == 3) {
        if (elect_one()) {
            tma_prefetch_desc(&p.map);
            if (p.q_tma) {
                tma_prefetch_desc(&p.qc);
                if (rope) tma_prefetch_desc(&p.qr);
            }
        }
    } else if (tid == 64) {
        for (int i = 0; i < kMaxPairs; i++) {
            mbar_init(&S.pair_full[i], 1);
            mbar_init(&S.pair_empty[i], 1);
        }
        for (int i = 0; i < kMaxRope; i++) {
            mbar_init(&S.rope_full[i], 1);
            mbar_init(&S.rope_empty[i], 1);
        }
        mbar_init(&S.q_full, p.q_tma ? 1 : 32);
        mbar_init(&S.q_empty, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(&S.s_full[i], 1);
            mbar_init(&S.p_full[i], kSoft / 32);
            mbar_init(&S.p_empty[i], 1);
        }
        mbar_init(&S.o_full, 1);
        mbar_init(&S.drain[0], 1);
        mbar_init(&S.drain[1], 1);
        fence_mbar_init();
        S.gave_up = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cudaTriggerProgrammaticLaunchCompletion();   // the join's blocks may take their places
    const uint32_t tmem = S.tmem;
    const uint32_t pairs = smem_u32(sm), ropes = pairs + p.rope_off, qs = pairs + p.q_off, ps = pairs + p.p_off;
    const int total = S.total;
    volatile uint32_t* gave_up = &S.gave_up;

    if (warp == 0) {
        // ------------------------------------------------------------ the cache, tile by tile
        Run r(deal, S.b, S.tile, total);
        const int subs = kDecodeTile / p.box, sub = lane & (subs - 1), blk = lane / subs;   // subs: 1, 2, 4 or 8
        uint32_t slot = 0, phase = 0, rslot = 0, rphase = 0;
        int issued = 0, rissued = 0;
        for (int i = 0; i < total; i++) {
            int at = p.total_rows;
            const int j = r.tile * kDecodeTile + sub * p.box;
            if (blk < 2 && j < r.n) {
                const int in = j / s.page, page = a.table[(long long)r.b * s.maxpages + in];
                if (page >= 0 && page < s.npages) at = page * s.page + (j - in * s.page);
            }
            if (rope) {
                wait_for(&S.rope_empty[rslot], rphase ^ 1, gave_up);
                __syncwarp();
                if (!__any_sync(0xffffffffu, *gave_up != 0)) {
                    uint64_t* bar = &S.rope_full[rslot];
                    if (elect_one()) mbar_arrive_expect_tx(bar, kBlockBytes);
                    __syncwarp();
                    const uint32_t dst = ropes + rslot * kBlockBytes + sub * p.box * 128;
                    if (lane < subs) tma_load_2d(dst, &p.map, bar, s.dc, at);
                    rissued++;
                }
                if (++rslot == (uint32_t)p.nrope) {
                    rslot = 0;
                    rphase ^= 1;
                }
            }
            for (int k = 0; k < p.np; k++) {
                wait_for(&S.pair_empty[slot], phase ^ 1, gave_up);
                __syncwarp();
                if (!__any_sync(0xffffffffu, *gave_up != 0)) {
                    const int blocks = min(2, p.nb - 2 * k);
                    uint64_t* bar = &S.pair_full[slot];
                    if (elect_one()) mbar_arrive_expect_tx(bar, blocks * kBlockBytes);
                    __syncwarp();
                    if (lane < blocks * subs && i != p.starve)   // a lane a box
                        tma_load_2d(pairs + slot * kPairBytes + blk * kBlockBytes + sub * p.box * 128, &p.map, bar, 128 * k + 64 * blk, at);
                    issued++;
                }
                if (++slot == (uint32_t)p.npair) {
                    slot = 0;
                    phase ^= 1;
                }
            }
            r.step();
        }
        if (*gave_up) {   // a wait expired: the copies in flight land before the CTA ends
            for (int i = 0; i < p.npair; i++) {
                const int n = (issued - i + p.npair - 1) / p.npair;
                if (n > 0) mbar_wait(&S.pair_full[i], (uint32_t)(n - 1) & 1, nullptr, kDrainNs);
            }
            for (int i = 0; i < p.nrope; i++) {
                const int n = (rissued - i + p.nrope - 1) / p.nrope;
                if (n > 0) mbar_wait(&S.rope_full[i], (uint32_t)(n - 1) & 1, nullptr, kDrainNs);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ the scores' products
        if (elect_one()) {
            const uint32_t id = idesc_bf16(64, NC, false, false);
            constexpr uint32_t kQBlock = NC * 128;
            const uint64_t base = sdesc(0, 16u, 1024u);
            Run r(deal, S.b, S.tile, total);
            uint32_t slot = 0, phase = 0, rslot = 0, rphase = 0, piece = 0;
            bool first = true;
            for (int i = 0; i < total; i++) {
                const uint32_t d = tmem + (uint32_t)(i & 1) * NC;
                if (first) wait_for(&S.q_full, piece++ & 1, gave_up);
                if (i >= 2) wait_for(&S.p_full[i & 1], (uint32_t)((i - 2) >> 1) & 1, gave_up);   // the buffer's last scores are read
                uint64_t q = base + at_desc(qs);
                if (rope) {      // first: a tile's last latent columns come in late where the ring holds less than two tiles
                    wait_for(&S.rope_full[rslot], rphase, gave_up);
                    tc_fence_after();
                    if (!*gave_up) {
                        const uint64_t kt = base + at_desc(ropes + rslot * kBlockBytes), qt = base + at_desc(qs + p.nb * kQBlock);
#pragma unroll
                        for (int ks = 0; ks < 4; ks++) mma_bf16(d, kt + 2 * ks, qt + 2 * ks, id, ks ? 1u : 0u);
                    }
                    mma_commit(&S.rope_empty[rslot]);
                    if (++rslot == (uint32_t)p.nrope) {
                        rslot = 0;
                        rphase ^= 1;
                    }
                }
                for (int k = 0; k < p.np; k++) {
                    wait_for(&S.pair_full[slot], phase, gave_up);
                    tc_fence_after();
                    if (!*gave_up) {
                        const uint64_t kt = base + at_desc(pairs + slot * kPairBytes);
#pragma unroll
                        for (int ks = 0; ks < 4; ks++) mma_bf16(d, kt + 2 * ks, q + 2 * ks, id, (rope || (k | ks)) ? 1u : 0u);
                        if (2 * k + 1 < p.nb) {
#pragma unroll
                            for (int ks = 0; ks < 4; ks++)
                                mma_bf16(d, kt + (kBlockBytes >> 4) + 2 * ks, q + (kQBlock >> 4) + 2 * ks, id, 1u);
                        }
                    }
                    q += 2 * (kQBlock >> 4);
                    if (++slot == (uint32_t)p.npair) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                mma_commit(&S.s_full[i & 1]);
                first = r.step();
                if (first) mma_commit(&S.q_empty);
            }
            if (*gave_up) {   // the products in flight end before TMEM is freed
                mma_commit(&S.drain[0]);
                mbar_wait(&S.drain[0], 0, nullptr, kDrainNs);
            }
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ the outputs' products
        if (elect_one()) {
            const uint32_t id = idesc_bf16(128, NC, true, false);
            const uint64_t vbase = sdesc(0, kBlockBytes, 1024u), pbase = sdesc(0, 16u, 1024u);
            Run r(deal, S.b, S.tile, total);
            uint32_t slot = 0;
            bool first = true;
            for (int i = 0; i < total; i++) {
                wait_for(&S.p_full[i & 1], (uint32_t)(i >> 1) & 1, gave_up);
                tc_fence_after();
                const bool go = !*gave_up;
                const uint64_t pt = pbase + at_desc(ps + (uint32_t)(i & (kWeights<NC> - 1)) * (NC * 128));
                for (int m = 0; m < p.np; m++) {
                    const uint64_t v = vbase + at_desc(pairs + slot * kPairBytes);
                    if (go) {
#pragma unroll
                        for (int ks = 0; ks < 4; ks++)
                            mma_bf16(tmem + (2 + m) * NC, v + 128 * ks, pt + 2 * ks, id, (first && ks == 0) ? 0u : 1u);
                    }
                    mma_commit(&S.pair_empty[slot]);
                    if (++slot == (uint32_t)p.npair) slot = 0;
                }
                mma_commit(&S.p_empty[i & 1]);
                first = r.step();
                if (first) mma_commit(&S.o_full);
            }
            if (*gave_up) {
                mma_commit(&S.drain[1]);
                mbar_wait(&S.drain[1], 0, nullptr, kDrainNs);
            }
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax, outputs
        // Two warpgroups take half of the query rows' columns each (against one, when a load served two groups, us: 160 rows
        // 92.3 to 90.1, 128 rows 92.3 to 88.2, 16 rows unchanged, 160 rows over 256 + 64 53.3 to 55.3).  An M = 64 product
        // fills the first 16 lanes of each warp's 32 in TMEM: lanes 16..31 take over the second half of these rows' columns.
        constexpr int HC = NC / 4;
        const int quad = warp & 3, half = (warp - 4) >> 2, t = tid - 128, key = quad * 16 + (lane & 15);
        const int col0 = 2 * HC * half + (lane < 16 ? 0 : HC);
        const float c = s.scale * kLog2e;
        float l[HC];
        Run r(deal, S.b, S.tile, total);
        uint32_t piece = 0, pslot = 0;
        if (t < NC) S.back[t] = (float)(s.T - 1 - (row0 + min(t, rows - 1)) / s.H);
        int from = r.tile;
        bool first = true;
        for (int i = 0; i < total; i++) {
            const uint32_t buf = (uint32_t)i & 1, phase = (uint32_t)(i >> 1) & 1;
            if (first) {
                from = r.tile;
                if (t < NC) S.top[t] = t < rows ? 0.f : INFINITY;   // a column of another's queries never asks to raise
#pragma unroll
                for (int n = 0; n < HC; n++) l[n] = 0.f;
                group_sync(1, kSoft);
            }
            wait_for(&S.s_full[buf], phase, gave_up);
            __syncwarp();
            tc_fence_after();
            float x[HC];
            {
                float y[2 * HC];
                load_cols<2 * HC>(lane_base(tmem, quad) + buf * NC + 2 * HC * half, y);
#pragma unroll
                for (int n = 0; n < HC; n++) {
                    const float other = __shfl_sync(0xffffffffu, y[n + HC], lane & 15);
                    x[n] = lane < 16 ? y[n] : other;
                }
            }
            const int j = r.tile * kDecodeTile + key, end = (r.tile + 1) * kDecodeTile;
            if (end > r.n - (s.T - 1)) {
#pragma unroll
                for (int n = 0; n < HC; n++) x[n] = j < r.n - (int)S.back[col0 + n] ? x[n] * c : -INFINITY;
            } else {
#pragma unroll
                for (int n = 0; n < HC; n++) x[n] *= c;
            }
            // the first tile of a piece sets the maximum; a query that sees none of it sees none of the later ones either
            bool over = first;
#pragma unroll
            for (int n = 0; n < HC; n += 4) {
                const float4 m = *reinterpret_cast<const float4*>(&S.top[col0 + n]);
                x[n] -= m.x;       // lowered by the maximum so far
                x[n + 1] -= m.y;
                x[n + 2] -= m.z;
                x[n + 3] -= m.w;
                over |= fmaxf(fmaxf(x[n], x[n + 1]), fmaxf(x[n + 2], x[n + 3])) > kSlack;
            }
            if (end > r.n) {   // rows past the length hold anything: weights of zero would still meet a NaN
                const int valid = r.n - r.tile * kDecodeTile, bad = kDecodeTile - valid;
                for (int k = 0; k < p.nb; k++) {
                    uint32_t slot = pslot + (k >> 1);
                    if (slot >= (uint32_t)p.npair) slot -= p.npair;
                    unsigned char* v = sm + slot * kPairBytes + (k & 1) * kBlockBytes + valid * 128;
                    for (int e = t; e < bad * 8; e += kSoft) *reinterpret_cast<uint4*>(v + e * 16) = make_uint4(0, 0, 0, 0);
                }
            }
            if (bar_any(1, kSoft, over)) {
#pragma unroll
                for (int n = 0; n < HC; n++) {
                    float m = x[n];
#pragma unroll
                    for (int k = 8; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
                    if ((lane & 15) == 0) S.red[quad][col0 + n] = m;
                }
                group_sync(1, kSoft);
                if (t < NC) {
                    const float m = fmaxf(fmaxf(S.red[0][t], S.red[1][t]), fmaxf(S.red[2][t], S.red[3][t]));
                    const float up = first ? (m == -INFINITY ? 0.f : m) : fmaxf(m, 0.f);   // what the maximum rises by
                    S.up[t] = up;
                    S.top[t] += up;
                    S.keep[t] = first ? 1.f : fast_exp2(-up);
                }
                group_sync(1, kSoft);
#pragma unroll
                for (int n = 0; n < HC; n++) {
                    l[n] *= S.keep[col0 + n];
                    x[n] -= S.up[col0 + n];
                }
                if (!first) {   // the outputs so far, by the same factors
                    wait_for(&S.p_empty[buf ^ 1], (uint32_t)((i - 1) >> 1) & 1, gave_up);
                    __syncwarp();
                    tc_fence_after();
#pragma unroll 1
                    for (int n0 = 0; n0 < NC; n0 += 16) {
                        float f[16];
#pragma unroll
                        for (int n = 0; n < 16; n++) f[n] = S.keep[n0 + n];
#pragma unroll 1
                        for (int m = half; m < p.np; m += 2) {
                            const uint32_t addr = lane_base(tmem, quad) + (2 + m) * NC + n0;
                            float o[16];
                            tmem_ld16(addr, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int n = 0; n < 16; n++) o[n] *= f[n];
                            tmem_st16(addr, o);
                        }
                    }
                    tmem_wait_st();
                }
            }
            // the buffer's last weights are read
            if (i >= kWeights<NC>) wait_for(&S.p_empty[(i - kWeights<NC>) & 1], (uint32_t)((i - kWeights<NC>) >> 1) & 1, gave_up);
            unsigned char* P = sm + p.p_off + (i & (kWeights<NC> - 1)) * (NC * 128);
#pragma unroll
            for (int n = 0; n < HC; n++) {
                const float y = fast_exp2(x[n]);
                l[n] += y;
                *reinterpret_cast<__nv_bfloat16*>(P + sw128(col0 + n, key)) = __float2bfloat16_rn(y);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.p_full[buf]);
            pslot += p.np;
            while (pslot >= (uint32_t)p.npair) pslot -= p.npair;
            const int b = r.b, to = r.to, tiles = r.tiles;
            first = r.step();
            if (!first) continue;
            // ---- the piece's end: sums of the 64 rows' threads, outputs out of TMEM
#pragma unroll
            for (int n = 0; n < HC; n++) {
                float m = l[n];
#pragma unroll
                for (int k = 8; k; k >>= 1) m += __shfl_xor_sync(0xffffffffu, m, k);
                if ((lane & 15) == 0) S.red[quad][col0 + n] = m;
            }
            group_sync(1, kSoft);
            const bool whole = from == 0 && to == tiles;
            const long long slot = ((long long)group * a.slots + cta + b) * a.rows;
            const long long out = (long long)b * s.T * s.H + row0;
            if (t < NC) {
                const float sum = S.red[0][t] + S.red[1][t] + S.red[2][t] + S.red[3][t];
                S.keep[t] = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;   // a NaN stays one
                const float l2 = sum == 0.f ? -INFINITY : S.top[t] + log2f(sum);
                if (t < rows) {
                    if (!whole)
                        a.part_l[slot + t] = l2;
                    else if (a.lse)
                        a.lse[out + t] = l2 * kLn2;
                }
            }
            group_sync(1, kSoft);
            wait_for(&S.o_full, piece & 1, gave_up);
            __syncwarp();
            piece++;
            tc_fence_after();
#pragma unroll 1
            for (int n0 = 0; n0 < rows; n0 += 16) {
                float f[16];
#pragma unroll
                for (int n = 0; n < 16; n++) f[n] = S.keep[n0 + n];
                const int here = rows - n0;
#pragma unroll 1
                for (int m = half; m < p.np; m += 2) {
                    const int d = 128 * m + 32 * quad + lane;
                    float o[16];
                    __syncwarp();
                    tmem_ld16(lane_base(tmem, quad) + (2 + m) * NC + n0, o);
                    tmem_wait_ld();
                    if (d >= s.dc) continue;
                    if (whole) {
                        __nv_bfloat16* y = (__nv_bfloat16*)a.o + (out + n0) * s.dc + d;
#pragma unroll
                        for (int n = 0; n < 16; n++, y += s.dc)
                            if (n < here) *y = __float2bfloat16_rn(o[n] * f[n]);
                    } else {
                        float* y = a.part_o + (slot + n0) * s.dc + d;
#pragma unroll
                        for (int n = 0; n < 16; n++, y += s.dc)
                            if (n < here) *y = o[n] * f[n];
                    }
                }
            }
            tc_fence_before();
            group_sync(1, kSoft);   // the sums' words are free for the next piece
        }
    } else {
        // ------------------------------------------------------------ queries: [query rows][64 columns] blocks
        const int col = (lane & 7) * 8;
        Run r(deal, S.b, S.tile, total);
        uint32_t piece = 0, loaded = ~0u;
        for (int i = 0; i < total;) {
            if (piece > 0) wait_for(&S.q_empty, (piece - 1) & 1, gave_up);
            if (p.q_tma) {
                // rows past the group's are another's: their scores and outputs are columns that nobody reads
                __syncwarp();
                if (elect_one() && !*gave_up) {
                    const int from = r.b * s.T * s.H + row0;
                    mbar_arrive_expect_tx(&S.q_full, (p.nb + (rope ? 1 : 0)) * NC * 128);
                    for (int k = 0; k < p.nb; k++) tma_load_2d(qs + k * NC * 128, &p.qc, &S.q_full, 64 * k, from);
                    if (rope) tma_load_2d(qs + p.nb * NC * 128, &p.qr, &S.q_full, 0, from);
                    loaded = piece;
                }
                piece++;
                do i++;
                while (!r.step() && i < total);
                continue;
            }
            for (int n = lane >> 3; n < NC; n += 4) {    // past the rows or the width: zeros
                const bool row = n < rows;
                const int tt = row ? (row0 + n) / s.H : 0, h = row ? row0 + n - tt * s.H : 0;
                const long long tok = (long long)r.b * s.T + tt;
                const __nv_bfloat16* c = (const __nv_bfloat16*)a.qc.p + tok * a.qc.tok + h * a.qc.head;
                uint32_t dst = qs + sw128(n, col);
                for (int k = 0; k < p.nb; k++, dst += NC * 128) {
                    const bool in = row && 64 * k + col < s.dc;
                    copy16(dst, c + (in ? 64 * k + col : 0), in);
                }
                if (rope) {
                    const __nv_bfloat16* x = (const __nv_bfloat16*)a.qr.p + tok * a.qr.tok + h * a.qr.head;
                    const bool in = row && col < s.dr;
                    copy16(dst, x + (in ? col : 0), in);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            fence_proxy_async_smem();
            mbar_arrive(&S.q_full);
            piece++;
            do i++;
            while (!r.step() && i < total);
        }
        if (loaded != ~0u && *gave_up) mbar_wait(&S.q_full, loaded & 1, nullptr, kDrainNs);   // the copy in flight lands
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
    if (tid == 0) a.cta_err[group * a.ctas + cta] = S.gave_up;
}

template <int NC>
cudaError_t run(Params& p, cudaStream_t st)
{
    const int blocks = p.nb + (p.a.s.dr > 0 ? 1 : 0);
    const uint32_t q = blocks * NC * 128, pp = kWeights<NC> * NC * 128;
    const uint32_t room = 232448 - 1024 - (uint32_t)sizeof(Shared) - (NC > 64 ? 2048 : 4096);   // a join block beside the worker
    p.nrope = p.a.s.dr == 0 ? 0 : p.np >= 3 ? (NC > 64 ? 1 : 2) : 4;
    const uint32_t fixed = q + pp + p.nrope * kBlockBytes;
    p.npair = (int)((room - fixed) / kPairBytes);
    if (p.npair > kMaxPairs) p.npair = kMaxPairs;
    if (p.npair < p.np) return cudaErrorInvalidValue;
    p.rope_off = p.npair * kPairBytes;
    p.q_off = p.rope_off + p.nrope * kBlockBytes;
    p.p_off = p.q_off + q;
    const size_t bytes = 1024 + p.p_off + pp;
    const cudaError_t e = cudaFuncSetAttribute(decode_tc_kernel<NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    decode_tc_kernel<NC><<<dim3(p.a.ctas, p.a.groups), kThreads, bytes, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

// Workers on the tensor cores: bf16 query rows in groups of at most 80.
cudaError_t launch_decode_tc(const DecodeArgs& a, cudaStream_t st)
{
    const gdn_mla_cache_t& s = a.s;
    Params p;
    p.a = a;
    p.nb = (s.dc + 63) / 64;
    p.np = (p.nb + 1) / 2;
    p.box = 8;
    while (p.box < kDecodeTile && s.page % (2 * p.box) == 0) p.box *= 2;
    p.total_rows = s.npages * s.page;
    p.starve = test_starve_chunk();
    const int W = s.dc + s.dr;
    p.q_tma = a.qc.tok == (long long)s.H * a.qc.head && (s.dr == 0 || a.qr.tok == (long long)s.H * a.qr.head) &&
              (long long)s.B * s.T * s.H < 0x7fffffffLL;
    const int nc = a.rows <= 16 ? 16 : a.rows <= 32 ? 32 : a.rows <= 48 ? 48 : a.rows <= 64 ? 64 : 80;
    if (!row_map(&p.map, a.cache, (long long)W, p.total_rows, W, p.box) ||
        (p.q_tma && (!row_map(&p.qc, a.qc.p, a.qc.head, (long long)s.B * s.T * s.H, s.dc, nc) ||
                     (s.dr > 0 && !row_map(&p.qr, a.qr.p, a.qr.head, (long long)s.B * s.T * s.H, s.dr, nc)))))
        return cudaErrorInvalidValue;
    return nc == 16   ? run<16>(p, st)
           : nc == 32 ? run<32>(p, st)
           : nc == 48 ? run<48>(p, st)
           : nc == 64 ? run<64>(p, st)
                      : run<80>(p, st);
}

}  // namespace mla
}  // namespace gdn
