// q8kv_seal.cu - whole blocks of a slot's f16 tail become 8-bit codes.
//
// A block is 32 tokens of one layer and KV head: d = max |x| / 127 over its 32 x 128
// finite values, code = x / d rounded to the nearest integer (fp32 division,
// halves away from zero), K as [key][dim], V transposed, [dim][key], so that
// attention finds both operands of its products with the summed axis in a row.
// A block is quantised once, when all of its tokens are there: its codes
// follow from the tokens alone, not from the steps that brought them.
//
// Bound by memory: 16 KB read and 8 KB written a block.  One CTA of 256 threads
// a block, all its loads under way at once.  The division would take longer
// than the bytes (25 instructions a value with it, 9 without): x * (1 / d) is
// within 2^-22 of the quotient's 32-bit value relatively, 3e-5 in all, so its
// rounding is the quotient's wherever it lies further than 1e-4 from a half;
// eight values with one nearer go through the division.
#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"
#include "q8kv.h"

namespace luce {

constexpr int kSealThreads = 256;
constexpr int kSealPitch = 33;  // words from key to key of V's codes on their way: the reads of a warp in 32 banks

// The largest finite |x| of eight values.
__device__ __forceinline__ float seal_top(const uint4& x)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t lo = w[e] & 0x7fffu, hi = w[e] >> 16 & 0x7fffu;  // (magnitudes order as integers)
        if (lo < 0x7c00u) top = max(top, lo);
        if (hi < 0x7c00u) top = max(top, hi);
    }
    return __half2float(__ushort_as_half((unsigned short)top));
}

// Eight values' codes, in order.
__device__ __forceinline__ uint2 seal_codes(const uint4& x, float d, float inv)
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8];
    uint32_t n[8];
    bool sure = true;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
        v[2 * e] = f.x;
        v[2 * e + 1] = f.y;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = __fmul_rn(v[e], inv), m = __fadd_rn(t, 12582912.0f);  // 1.5 * 2^23: the nearest integer in the low bits
        n[e] = __float_as_uint(m);
        sure = sure && fabsf(__fsub_rn(t, __fsub_rn(m, 12582912.0f))) < 0.4999f;  // (false for a NaN)
    }
    if (!sure) {
#pragma unroll
        for (int e = 0; e < 8; ++e) n[e] = (uint32_t)q8_code(v[e], d);
    }
    const uint32_t a = __byte_perm(n[0], n[1], 0x0040), b = __byte_perm(n[2], n[3], 0x0040);
    const uint32_t c = __byte_perm(n[4], n[5], 0x0040), e = __byte_perm(n[6], n[7], 0x0040);
    return make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(c, e, 0x5410));
}

__global__ void __launch_bounds__(kSealThreads)
q8kv_seal_kernel(const __grid_constant__ Q8SealBatch b, int64_t heads)
{
    __shared__ float tops[2][kSealThreads / 32];
    __shared__ uint32_t vt[kQ8Block * kSealPitch];
    pdl_trigger();
    int unit = blockIdx.y, sl = 0;
    while (sl + 1 < b.n_slot && unit >= b.slot[sl].n / kQ8Block) unit -= b.slot[sl++].n / kQ8Block;
    const Q8SealSlot& s = b.slot[sl];
    const int64_t lh = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    __half* k = s.k + lh * s.cap * kHeadDim;
    __half* v = s.v + lh * s.cap * kHeadDim;
    const int block = s.sealed / kQ8Block + unit, quarter = block & 3;
    pdl_wait();
    const int page = s.table ? ld_placed_i(s.table + (block >> 2)) : block >> 2;
    // 16 threads a row, 16 bytes each: rows tid / 16 and tid / 16 + 16
    const int64_t at = ((int64_t)unit * kQ8Block + (tid >> 4)) * kHeadDim + 8 * (tid & 15);
    uint4 x[2][2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        x[0][e] = ld_placed_cs_u4(k + at + 16 * e * kHeadDim);
        x[1][e] = ld_placed_cs_u4(v + at + 16 * e * kHeadDim);
    }
    // the rows behind the last whole block move to the front, by the first block's CTA
    const int whole = s.n / kQ8Block * kQ8Block, rest = unit == 0 ? (s.n - whole) * 16 : 0;
    uint4 y[2][2];
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (tid + e * kSealThreads < rest) {
            const int64_t from = (int64_t)whole * kHeadDim + 8 * (tid + e * kSealThreads);
            y[0][e] = ld_placed_cs_u4(k + from);
            y[1][e] = ld_placed_cs_u4(v + from);
        }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const float top = warp_max(fmaxf(seal_top(x[w][0]), seal_top(x[w][1])));
        if (lane == 0) tops[w][warp] = top;
    }
    __syncthreads();  // (every row of the block has been read, too)
    float d[2], inv[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float top = tops[w][0];
#pragma unroll
        for (int e = 1; e < kSealThreads / 32; ++e) top = fmaxf(top, tops[w][e]);
        d[w] = __fdiv_rn(top, 127.0f);
        inv[w] = __fdiv_rn(1.0f, d[w]);
    }
    const bool in = page >= 0 && page < s.n_pages;
    const int64_t place = (int64_t)page * heads + lh;
    if (in && tid < 2) s.scales[place * kQ8PageScales + 4 * tid + quarter] = d[tid];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const int key = (tid >> 4) + 16 * e;
        const uint2 kc = seal_codes(x[0][e], d[0], inv[0]), vc = seal_codes(x[1][e], d[1], inv[1]);
        if (in)
            *reinterpret_cast<uint2*>(s.k_codes + place * kQ8PageBytes + (quarter * kQ8Block + key) * kHeadDim + 8 * (tid & 15)) = kc;
        vt[key * kSealPitch + 2 * (tid & 15)] = vc.x;
        vt[key * kSealPitch + 2 * (tid & 15) + 1] = vc.y;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
        if (tid + e * kSealThreads < rest) {
            *reinterpret_cast<uint4*>(k + 8 * (tid + e * kSealThreads)) = y[0][e];
            *reinterpret_cast<uint4*>(v + 8 * (tid + e * kSealThreads)) = y[1][e];
        }
    __syncthreads();
    // four keys by four dims a thread, turned
    const int kg = tid & 7, dg = tid >> 3;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = vt[(4 * kg + e) * kSealPitch + dg];
    const uint32_t a0 = __byte_perm(w[0], w[1], 0x5140), a1 = __byte_perm(w[0], w[1], 0x7362);  // dims 0, 1 and 2, 3 of keys 0, 1
    const uint32_t b0 = __byte_perm(w[2], w[3], 0x5140), b1 = __byte_perm(w[2], w[3], 0x7362);
    const uint32_t o[4] = {__byte_perm(a0, b0, 0x5410), __byte_perm(a0, b0, 0x7632), __byte_perm(a1, b1, 0x5410),
                           __byte_perm(a1, b1, 0x7632)};
    if (in) {
        int8_t* to = s.v_codes + place * kQ8PageBytes + 4 * dg * kQ8Page + quarter * kQ8Block + 4 * kg;
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(to + e * kQ8Page) = o[e];
    }
}

cudaError_t launch_q8kv_seal(const Q8SealBatch& b, int n_layers, int Hkv, cudaStream_t s)
{
    int units = 0;
    for (int i = 0; i < b.n_slot; ++i) units += b.slot[i].n / kQ8Block;
    const int64_t heads = (int64_t)n_layers * Hkv;
    const cudaError_t e = launch_pdl(q8kv_seal_kernel, dim3((unsigned)heads, (unsigned)units), dim3(kSealThreads), s, b, heads);
    count_launches(1);
    return e;
}

}  // namespace luce
