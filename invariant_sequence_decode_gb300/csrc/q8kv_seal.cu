// q8kv_seal.cu - whole blocks of a slot's f16 tail become 8-bit codes.
//
// A block is 32 tokens of one layer and KV head: d = max |x| / 127 over its 32 x 128
// finite values, code = x / d rounded to the nearest integer (fp32 division,
// halves away from zero), K as [key][dim], V transposed, [dim][key], so that
// attention finds both operands of its products with the summed axis in a row.
// A block is quantised once, when all of its tokens are there: its codes
// follow from the tokens alone, not from the steps that brought them.
//
// Bound by memory: 16 KB read and 8 KB written a block.  One CTA of 256 threads a
// block, eight CTAs a multiprocessor, all loads of a CTA under way at once.  A division
// for every code takes longer than the bytes: x * (1 / d), with a reciprocal within 2^-23
// of 1 / d, is within 2^-21 of the quotient's 32-bit value relatively, 7e-5 in all, so
// its rounding is the quotient's wherever it lies further than 1e-4 from a half; four
// values with one nearer go through the division.  The codes are formed in pairs, and
// maxima found on packed magnitudes: 85 % of the issue slots were taken before that.
// 32,736 keys of 32 heads take 125 us, 6.45 TB/s, 0.95 of a copy's rate (147 in single
// values, 225 with divisions; six CTAs a multiprocessor 128); a block of each of 2,048 heads,
// four slots of 512, 13.8 us.
#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"
#include "q8kv.h"
#include "tensor.cuh"

namespace luce {

constexpr int kSealThreads = 256;
constexpr int kSealPitch = 33;  // words from key to key of V's codes on their way: the reads of a warp in 32 banks

// 32 bytes, read once.
__device__ __forceinline__ void seal_load(const __half* p, uint32_t (&v)[8])
{
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p)
                 : "memory");
}

// The largest finite |x| of sixteen values.  Magnitudes order as integers, two a
// word; what is not finite is the largest of all, and only then looked for.
__device__ __forceinline__ float seal_top(const uint32_t (&w)[8])
{
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    if (top >= 0x7c00u) {
        top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t lo = w[e] & 0x7fffu, hi = w[e] >> 16 & 0x7fffu;
            top = max(top, max(lo < 0x7c00u ? lo : 0u, hi < 0x7c00u ? hi : 0u));
        }
    }
    return __half2float(__ushort_as_half((unsigned short)top));
}

// Four values' codes, in order.
__device__ __forceinline__ uint32_t seal_codes(uint32_t a, uint32_t b, float d, float inv)
{
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&a)), y = __half22float2(*reinterpret_cast<const __half2*>(&b));
    // 1.5 * 2^23 and the product in one: the nearest integer in the low bits; then the
    // product's distance from it
    const uint64_t up = pair(12582912.0f, 12582912.0f), inv2 = pair(inv, inv), less = pair(-1.0f, -1.0f);
    const uint64_t x2 = pair(x.x, x.y), y2 = pair(y.x, y.y), m = fma2(x2, inv2, up), n = fma2(y2, inv2, up);
    const float2 p = unpair(fma2(x2, inv2, fma2(m, less, up))), q = unpair(fma2(y2, inv2, fma2(n, less, up)));
    float far;  // the furthest from its nearest integer
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(far) : "f"(p.x), "f"(p.y), "f"(q.x));
    asm("max.NaN.abs.f32 %0, %1, %2, %2;" : "=f"(far) : "f"(far), "f"(q.y));
    const float2 mf = unpair(m), nf = unpair(n);
    uint32_t c[4] = {__float_as_uint(mf.x), __float_as_uint(mf.y), __float_as_uint(nf.x), __float_as_uint(nf.y)};
    if (!(far < 0.4999f)) {  // (or a NaN, which the maximum keeps)
        const float v[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) c[e] = (uint32_t)q8_code(v[e], d);
    }
    return __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
}

__global__ void __launch_bounds__(kSealThreads, 8)
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
    // eight threads a row, 32 bytes each
    const int key = tid >> 3, piece = tid & 7;
    const int64_t at = ((int64_t)unit * kQ8Block + key) * kHeadDim + 16 * piece;
    uint32_t x[2][8];
    seal_load(k + at, x[0]);
    seal_load(v + at, x[1]);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const float top = warp_max(seal_top(x[w]));
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
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv[w]) : "f"(d[w]));
    }
    const bool in = page >= 0 && page < s.n_pages;
    const int64_t place = (int64_t)page * heads + lh;
    if (in && tid < 2) s.scales[place * kQ8PageScales + 4 * tid + quarter] = d[tid];
    uint4 kc;
    kc.x = seal_codes(x[0][0], x[0][1], d[0], inv[0]);
    kc.y = seal_codes(x[0][2], x[0][3], d[0], inv[0]);
    kc.z = seal_codes(x[0][4], x[0][5], d[0], inv[0]);
    kc.w = seal_codes(x[0][6], x[0][7], d[0], inv[0]);
    if (in) *reinterpret_cast<uint4*>(s.k_codes + place * kQ8PageBytes + (quarter * kQ8Block + key) * kHeadDim + 16 * piece) = kc;
#pragma unroll
    for (int e = 0; e < 4; ++e) vt[key * kSealPitch + 4 * piece + e] = seal_codes(x[1][2 * e], x[1][2 * e + 1], d[1], inv[1]);
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
    // the rows behind the last whole block move to the front, by the first block's CTA
    // (which has read what lay there)
    const int whole = s.n / kQ8Block * kQ8Block, rest = unit == 0 ? (s.n - whole) * 16 : 0;
    for (int e = tid; e < rest; e += kSealThreads) {
        const uint4 a = ld_placed_cs_u4(k + (int64_t)whole * kHeadDim + 8 * e), c = ld_placed_cs_u4(v + (int64_t)whole * kHeadDim + 8 * e);
        *reinterpret_cast<uint4*>(k + 8 * e) = a;
        *reinterpret_cast<uint4*>(v + 8 * e) = c;
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
