// mla_tc.cuh -- what the tensor-core latent-attention kernels share: bounded waits that all roles of a CTA wind down
// on, tensor maps of strided row/head views, products with a TMEM operand.
#pragma once

#include <cuda.h>

#include "fwd_tc_common.cuh"
#include "mla_internal.h"
#include "tc_ptx.cuh"

namespace gdn {
namespace mla {

using fwdtc::fast_exp2;
using fwdtc::kLog2e;
using fwdtc::kWaitNs;
using namespace tc;

constexpr float kLn2 = 0.6931471805599453f;

// A wait on a phase of `bar`.  After one wait of the CTA has expired, `gave_up` is set and every wait returns at once:
// the roles then run through their loops without touching data, so that none is left at a barrier.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile uint32_t* gave_up)
{
    if (mbar_try_wait(bar, parity)) return true;
    if (*gave_up) return false;
    if (mbar_wait(bar, parity, nullptr, kWaitNs)) return true;
    *gave_up = 1;
    return false;
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// True in one lane of a converged warp.  Products and TMA loads are issued under it: the compiler then knows that one
// thread runs them and keeps their operands in uniform registers (a test of the lane number instead costs about 190
// cycles a product).
__device__ __forceinline__ bool elect_one()
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

// 2-D and 3-D tiled loads global -> shared, completion counted on `bar`
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, uint64_t* bar, int c0, int c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

// barrier of `threads` threads that also tells whether any of them said yes
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t threads, bool yes)
{
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"((uint32_t)yes)
        : "memory");
    return r != 0;
}

// ---------------------------------------------------------------- host side

// rows [n, heads, d] with strides in elements -> 3-D map (d, heads, rows), box 64 x 1 x box_rows, 128-byte swizzle;
// columns past d and rows past n read as zeros
inline bool view_map(CUtensorMap* m, const gdn_mla_view_t& v, long long n, int heads, int d, int box_rows)
{
    const fwdtc::EncodeTiledFn enc = fwdtc::get_encode();
    if (!enc) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)v.head * 2, (cuuint64_t)v.tok * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_rows}, one[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, v.p, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

}  // namespace mla
}  // namespace gdn
