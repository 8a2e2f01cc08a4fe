// rope_kv.cu - pos-vector RoPE and the per-sequence K/V append.
//
// "antirez/ds4 pull 604", Commit walkthrough: decode tokens of different
// sequences sit at arbitrary positions, so RoPE takes a position per row and
// its per-element math is that of a single-token launch at that position;
// section 2: KV append runs per sequence with the single-token helpers.
//
// Pairing: dims (i, i + 64) of a 128-dim head rotate by pos * theta^(-i/64).
// theta^(-i/64) is evaluated in double on the host; the angle is formed and
// reduced in double on the device and only the reduced angle goes through
// fp32 sincosf (see rope_cs), so even position 32767 carries no fp32 angle
// error.  The rotation is fp32 with explicit rounding.  One CTA of 64 threads
// per (row, head): thread i owns pair i.  The decode step applies the same
// rotation and append in the epilogue of its q|k|v projection (matvec.cu).
#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"
#include "q8kv.h"

namespace luce {

__global__ void __launch_bounds__(64)
rope_posvec_kernel(float* __restrict__ x, int64_t ldx, const int32_t* __restrict__ pos, RopeFreq f)
{
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x, h = blockIdx.y, i = threadIdx.x;
    const float2 cs = rope_cs(pos[t], f.inv[i]);
    float* p = x + (size_t)t * ldx + (size_t)h * kHeadDim + i;
    float x0 = p[0], x1 = p[kHeadDim / 2];
    rope_rotate(x0, x1, cs.x, cs.y);
    p[0] = x0;
    p[kHeadDim / 2] = x1;
}

cudaError_t launch_rope_posvec(float* x, int T, int n_heads, int64_t ldx, const int32_t* pos,
                               const RopeFreq& f, cudaStream_t s)
{
    const cudaError_t e = launch_pdl(rope_posvec_kernel, dim3(T, n_heads), dim3(64), s, x, ldx, pos, f);
    count_launches(1);
    return e;
}

// RoPE and the K/V append of the decode step from a q|k|v projection already
// in memory (the wide-verify path, where the projection runs on the tensor
// cores without an epilogue): one 64-thread CTA per (row t, head h of the
// q|k|v output), thread i owning the pair (i, i + 64).  q and k heads rotate
// by the row's position, q heads go to q_rot [T][Hq][128], k and v heads are
// rounded to binary16 at the row's K/V destination.  These are the rotation
// and conversion of the fused q|k|v epilogue (rope_cs, rope_rotate, round to
// nearest), so either path gives the same bits; cos/sin are formed before the
// wait on the projection.
__global__ void __launch_bounds__(64)
qkv_rope_kv_kernel(const float* __restrict__ qkv, int Hq, int Hkv, RowPos pos, RopeFreq f, float* __restrict__ q_rot,
                   KvRows kv)
{
    pdl_trigger();
    const int t = blockIdx.x, h = blockIdx.y, i = threadIdx.x;
    const bool rot = h < Hq + Hkv;
    const float2 cs = rot ? rope_cs(pos.pos[t], f.inv[i]) : make_float2(1.0f, 0.0f);
    pdl_wait();
    const float* src = qkv + (size_t)t * (Hq + 2 * Hkv) * kHeadDim + (size_t)h * kHeadDim;
    float x0 = src[i], x1 = src[i + kHeadDim / 2];
    if (rot) rope_rotate(x0, x1, cs.x, cs.y);
    if (h < Hq) {
        float* dst = q_rot + ((size_t)t * Hq + h) * kHeadDim;
        dst[i] = x0;
        dst[i + kHeadDim / 2] = x1;
    } else {
        const KvRow r = kv.row[t];
        __half* dst = rot ? r.k + (h - Hq) * r.head_stride : r.v + (h - Hq - Hkv) * r.head_stride;
        dst[i] = __float2half_rn(x0);
        dst[i + kHeadDim / 2] = __float2half_rn(x1);
    }
}

cudaError_t launch_qkv_rope_kv(const float* qkv, int T, int Hq, int Hkv, const RowPos& pos, const RopeFreq& f,
                               float* q_rot, const KvRows& kv, cudaStream_t s)
{
    const cudaError_t e =
        launch_pdl(qkv_rope_kv_kernel, dim3(T, Hq + 2 * Hkv), dim3(kHeadDim / 2), s, qkv, Hq, Hkv, pos, f, q_rot, kv);
    count_launches(1);
    return e;
}

// Standalone K/V append: one CTA per row; fp32 -> binary16 round-to-nearest.
__global__ void __launch_bounds__(256)
kv_append_kernel(const float* __restrict__ k, const float* __restrict__ v, int64_t ld, int Hkv, KvRows rows)
{
    pdl_trigger();
    pdl_wait();
    const int t = blockIdx.x;
    const KvRow r = rows.row[t];
    for (int idx = threadIdx.x; idx < Hkv * kHeadDim; idx += blockDim.x) {
        const int g = idx >> 7, dd = idx & 127;
        r.k[g * r.head_stride + dd] = __float2half_rn(k[(size_t)t * ld + idx]);
        r.v[g * r.head_stride + dd] = __float2half_rn(v[(size_t)t * ld + idx]);
    }
}

cudaError_t launch_kv_append(const float* k, const float* v, int64_t ld, int Hkv, const KvRows& rows,
                             cudaStream_t s)
{
    const cudaError_t e = launch_pdl(kv_append_kernel, dim3(rows.n_rows), dim3(256), s, k, v, ld, Hkv, rows);
    count_launches(1);
    return e;
}

// Norms of q and k per head, rotation, and append of a projection's rows in one
// pass.  Head x of row t becomes y = x / sqrt(mean(x^2) + eps) * gamma (as it is
// without a gamma), and the pair (y_i, y_(i+64)) rotates by the row's position on
// the pair's axis times theta^(-i/64); v heads are only rounded.
// Bound by memory (read once, written once), so what is shared is kept small:
// a row's 64 cosines and sines and the gammas go once per CTA into shared memory, and
// 16 lanes take a head, four pairs each as two 16-byte loads, kProjectAhead heads at a
// time.  All loads of the first are under way before the angles (formed in 64-bit
// arithmetic) and the sums are.  8,192 rows of 40 + 2 x 8 heads take 67.0 us, 6.5 TB/s,
// 0.96 of a copy's rate; with four heads at a time 70.7, three 73.4, one 75.5, eight CTAs a
// multiprocessor instead of six 74.1.  One row takes 2.1 us in a graph, latency; its call
// 4.6 to 5.0, the host's.  Sums of squares: a lane's eight in order, then lanes by an xor butterfly,
// so a row's bits do not depend on the other rows or the grid; without
// gammas and with one axis they are those of rope_posvec_kernel and kv_append_kernel.
constexpr int kProjectAhead = 2;

__global__ void __launch_bounds__(256, 6)
qk_norm_rope_kernel(const float* qkv, int64_t ld, int Hq, int Hkv, const __grid_constant__ AppendViews views,
                    const float* q_gamma, const float* k_gamma, float eps, const int32_t* pos, int T, PairAxes axes,
                    const __grid_constant__ RopeFreq f, float* __restrict__ q)
{
    __shared__ __align__(16) float cs[2][kHeadDim / 2];
    __shared__ __align__(16) float gammas[2][kHeadDim];
    pdl_trigger();
    const int t = blockIdx.x, tid = threadIdx.x, part = tid & 15, heads = Hq + 2 * Hkv;
    const int step = 16 * gridDim.y;
    int v = 0;
    while (v + 1 < views.n_view && (t < views.view[v].row0 || t >= views.view[v].row0 + views.view[v].n)) ++v;
    const AppendView& to = views.view[v];
    const int64_t at = (int64_t)(to.at0 + t - to.row0) * to.tok_stride;
    const float* row = qkv + (int64_t)t * ld + 4 * part;
    pdl_wait();
    bool turned = false;
    for (int h0 = blockIdx.y * 16 + (tid >> 4); h0 - (tid >> 4) < heads; h0 += kProjectAhead * step) {
        float4 a[kProjectAhead], b[kProjectAhead];
#pragma unroll
        for (int e = 0; e < kProjectAhead; ++e) {
            const int h = h0 + e * step;
            a[e] = b[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (h < heads) {
                a[e] = ld_placed_cs_f4(row + (int64_t)h * kHeadDim);
                b[e] = ld_placed_cs_f4(row + (int64_t)h * kHeadDim + kHeadDim / 2);
            }
        }
        if (!turned) {
            if (tid < kHeadDim / 2) {
                const int axis = axes.bits[tid >> 4] >> (2 * (tid & 15)) & 3;
                const float2 x = rope_cs(ld_placed_i(pos + (int64_t)axis * T + t), f.inv[tid]);
                cs[0][tid] = x.x;
                cs[1][tid] = x.y;
            } else if (tid < kHeadDim / 2 + 2 * kHeadDim / 4) {
                const int i = tid - kHeadDim / 2, at4 = 4 * (i & (kHeadDim / 4 - 1));
                const float* gamma = i < kHeadDim / 4 ? q_gamma : k_gamma;
                if (gamma) *reinterpret_cast<float4*>(&gammas[i / (kHeadDim / 4)][at4]) = ld_placed_f4(gamma + at4);
            }
        }
        float inv[kProjectAhead];
#pragma unroll
        for (int e = 0; e < kProjectAhead; ++e) {
            const float4 x = a[e], y = b[e];
            float sq = __fmul_rn(x.x, x.x);
            sq = __fmaf_rn(x.y, x.y, sq);
            sq = __fmaf_rn(x.z, x.z, sq);
            sq = __fmaf_rn(x.w, x.w, sq);
            sq = __fmaf_rn(y.x, y.x, sq);
            sq = __fmaf_rn(y.y, y.y, sq);
            sq = __fmaf_rn(y.z, y.z, sq);
            sq = __fmaf_rn(y.w, y.w, sq);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) sq = __fadd_rn(sq, __shfl_xor_sync(0xffffffffu, sq, o));
            inv[e] = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(sq, 1.0f / kHeadDim), eps)));
        }
        if (!turned) __syncthreads();
        turned = true;
        const float4 c = *reinterpret_cast<const float4*>(&cs[0][4 * part]);
        const float4 s = *reinterpret_cast<const float4*>(&cs[1][4 * part]);
#pragma unroll
        for (int e = 0; e < kProjectAhead; ++e) {
            const int h = h0 + e * step;
            if (h >= heads) break;
            float4 x = a[e], y = b[e];
            const float* gamma = h < Hq ? q_gamma : h < Hq + Hkv ? k_gamma : nullptr;
            if (gamma) {
                const float* gs = gammas[h >= Hq];
                const float4 g0 = *reinterpret_cast<const float4*>(gs + 4 * part), g1 = *reinterpret_cast<const float4*>(gs + kHeadDim / 2 + 4 * part);
                x.x = __fmul_rn(__fmul_rn(x.x, inv[e]), g0.x);
                x.y = __fmul_rn(__fmul_rn(x.y, inv[e]), g0.y);
                x.z = __fmul_rn(__fmul_rn(x.z, inv[e]), g0.z);
                x.w = __fmul_rn(__fmul_rn(x.w, inv[e]), g0.w);
                y.x = __fmul_rn(__fmul_rn(y.x, inv[e]), g1.x);
                y.y = __fmul_rn(__fmul_rn(y.y, inv[e]), g1.y);
                y.z = __fmul_rn(__fmul_rn(y.z, inv[e]), g1.z);
                y.w = __fmul_rn(__fmul_rn(y.w, inv[e]), g1.w);
            }
            if (h < Hq + Hkv) {
                rope_rotate(x.x, y.x, c.x, s.x);
                rope_rotate(x.y, y.y, c.y, s.y);
                rope_rotate(x.z, y.z, c.z, s.z);
                rope_rotate(x.w, y.w, c.w, s.w);
            }
            if (h < Hq) {
                float* o = q + ((int64_t)t * Hq + h) * kHeadDim + 4 * part;
                *reinterpret_cast<float4*>(o) = x;
                *reinterpret_cast<float4*>(o + kHeadDim / 2) = y;
            } else {
                __half* o = h < Hq + Hkv ? to.k + (h - Hq) * to.head_stride : to.v + (h - Hq - Hkv) * to.head_stride;
                o += at + 4 * part;
                __half2 w[4] = {__floats2half2_rn(x.x, x.y), __floats2half2_rn(x.z, x.w), __floats2half2_rn(y.x, y.y),
                                __floats2half2_rn(y.z, y.w)};
                *reinterpret_cast<uint2*>(o) = *reinterpret_cast<uint2*>(&w[0]);
                *reinterpret_cast<uint2*>(o + kHeadDim / 2) = *reinterpret_cast<uint2*>(&w[2]);
            }
        }
    }
}

cudaError_t launch_qk_norm_rope(const float* qkv, int64_t ld, int T, int Hq, int Hkv, const AppendViews& views,
                                const float* q_gamma, const float* k_gamma, float eps, const int32_t* pos,
                                const PairAxes& axes, const RopeFreq& f, float* q, cudaStream_t s)
{
    // few rows: 16 heads a CTA, so that a row's heads go at once (40 + 2 x 8 heads, with the
    // launch: 6.8 us for 8.9 up to 40 rows, 8.9 for 10.9 at 152, no difference up to 456); many: a
    // row a CTA, its angles formed once (608 rows 13.0 us for 15.0, 8,192 67 for 98)
    const int groups = T < 152 ? std::min((Hq + 2 * Hkv + 15) / 16, 65535) : 1;
    const cudaError_t e = launch_pdl(qk_norm_rope_kernel, dim3(T, groups), dim3(256), s, qkv, ld, Hq, Hkv, views, q_gamma,
                                     k_gamma, eps, pos, T, axes, f, q);
    count_launches(1);
    return e;
}

}  // namespace luce
