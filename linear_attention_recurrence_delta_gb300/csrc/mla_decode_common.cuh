// mla_decode_common.cuh -- how the cache rows of a batch are dealt out to decode workers.
//
// A worker's share is a run of kDecodeTile-row tiles in the order of all sequences' tiles laid end to end, so every
// worker has the same work whatever the lengths: a long sequence is cut over many workers, short ones share one.
// The lengths are on the device only; each worker finds its own run from them.  A worker's stretch of one sequence
// is a piece; piece (worker c, sequence b) has slot c + b of the workspace, which no other piece of the group has,
// since a step along the pieces moves c or b on by one.
#pragma once

#include "mla_internal.h"

namespace gdn {
namespace mla {

struct Deal {
    const int* len;
    int B, most;       // most: rows a block table can name

    __device__ __forceinline__ int rows(int b) const { return min(max(len[b], 0), most); }
    __device__ __forceinline__ int tiles(int b) const { return (rows(b) + kDecodeTile - 1) / kDecodeTile; }
};

// by all lanes of one warp: tiles of all sequences (the entry point bounds their number by 2^31)
__device__ __forceinline__ int deal_tiles(const Deal& d)
{
    int t = 0;
    for (int b = threadIdx.x & 31; b < d.B; b += 32) t += d.tiles(b);
    return __reduce_add_sync(0xffffffffu, t);
}

// a worker's share of them
__device__ __forceinline__ int deal_share(int tiles, int ctas) { return tiles / ctas + (tiles % ctas != 0); }

// by all lanes of one warp: the sequence that holds the tile `at` of the whole row, and the tile's place in it
// (b = B: past the end)
__device__ __forceinline__ void deal_find(const Deal& d, int at, int& b, int& tile)
{
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int b0 = 0; b0 < d.B; b0 += 32) {
        const int n = b0 + lane < d.B ? d.tiles(b0 + lane) : 0;
        int to = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, to, m);
            if (lane >= m) to += x;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + to > at);
        if (past) {
            const int l = __ffs(past) - 1;
            b = b0 + l;
            tile = (int)(at - base - __shfl_sync(0xffffffffu, to - n, l));
            return;
        }
        base += __shfl_sync(0xffffffffu, to, 31);
    }
    b = d.B;
    tile = 0;
}

// by all lanes of one warp: tiles before sequence b
__device__ __forceinline__ int deal_before(const Deal& d, int b)
{
    int t = 0;
    for (int i = threadIdx.x & 31; i < b; i += 32) t += d.tiles(i);
    return __reduce_add_sync(0xffffffffu, t);
}

}  // namespace mla
}  // namespace gdn
