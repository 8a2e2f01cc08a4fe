// tensor.cuh - pieces shared by the attention kernels whose products run on
// tcgen05: descriptors, issue and commit, tensor-memory fences, two-part f16 splits.
#pragma once

#include "cache.h"
#include "common.cuh"
#include "ring.cuh"

namespace luce {

// The driver's encoder of tiled tensor maps; nullptr when there is none.
PFN_cuTensorMapEncodeTiled_v12000 tree_map_encoder();

__device__ __forceinline__ uint64_t tree_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    // 128-byte swizzle; start address, leading and stride byte offsets in units of 16
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// D[128][N] (+)= A (tensor memory, f16) * B (shared memory), one 16-wide step, N
// from idesc, by the lane whose `elected` is set.  The whole warp comes here: issued
// from a branch of one thread, each product of the attention of draft trees (N = 128)
// cost 152 cycles (its descriptor goes through registers that only a converged warp has
// at hand) against 64.
__device__ __forceinline__ void tree_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate,
                                         uint32_t elected)
{
    asm volatile("{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
                 " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"(elected));
}

__device__ __forceinline__ void tree_commit_mma(uint64_t* bar, uint32_t elected)
{
    asm volatile("{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
                 " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_addr(bar)),
                 "r"(elected)
                 : "memory");
}

// One arrival for the warp, behind what all of its threads have done to tensor
// memory (32 arrivals of their own would queue at the barrier's word).
__device__ __forceinline__ void warp_arrive(uint64_t* bar)
{
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ uint32_t elect_one()
{
    uint32_t e;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(e));
    return e;
}
__device__ __forceinline__ void tm_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this warp's 32 lanes, written.
__device__ __forceinline__ void tm_st32(uint32_t addr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
        "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
        : "memory");
}
// The same of 16.
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]), "r"(r[1]),
        "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
        "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float tree_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of fp32 values: two sums or fused multiply-adds per instruction.
__device__ __forceinline__ uint64_t pair(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// Two fp32 values as f16 pairs, x = hi + lo; the first in the low half.
__device__ __forceinline__ void tree_split(float x0, float x1, uint32_t& hi, uint32_t& lo)
{
    float l0, l1;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x1), "f"(x0));
    asm("{\n .reg .f16 a, b, n;\n mov.b32 {a, b}, %2;\n mov.b16 n, 0xBC00;\n"  // x - hi, exactly
        " fma.rn.f32.f16 %0, a, n, %3;\n fma.rn.f32.f16 %1, b, n, %4;\n}"
        : "=f"(l0), "=f"(l1)
        : "r"(hi), "f"(x0), "f"(x1));
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(l1), "f"(l0));
}

// A box of the (d, key, head, page) map.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, int x, int y, int z, int w, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_addr(dst)),
        "l"(m), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ float4 half4(uint2 x)
{
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&x.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void axpy4(float4& o, float4 x, float a)
{
    o.x = __fmaf_rn(x.x, a, o.x);
    o.y = __fmaf_rn(x.y, a, o.y);
    o.z = __fmaf_rn(x.z, a, o.z);
    o.w = __fmaf_rn(x.w, a, o.w);
}

}  // namespace luce
