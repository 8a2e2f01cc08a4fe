// q8kv.cu - attention over a slot's cache in 8 bits, its tail and a draft tree.
//
// A slot's prefix is `sealed` keys in blocks of 32 that share a scale for K and
// one for V, and `tail` f16 keys behind them; then come the nodes of its draft
// tree.  Row r of node j at position p = sealed + tail + (ancestors of j) sees the
// keys i of the prefix and of its own path with i < sinks or p - i < window (all
// of them without a window).  For query head h
//   out = sum_i e^(s_i - m) v_i / l,  s_i = scale q.k_i,  m = max s_i,  l = sum e^(s_i - m),
// where a sealed key is its codes times its block's scale.  The sealed keys are cut
// into chunks of 128-key tiles; each chunk yields (m, l, sum e^(s - m) v) per row, and
// the merge adds the chunks in order, then the tail's keys and the path's.  A
// node's bits follow from its prefix and its path alone.
#include <algorithm>
#include <cmath>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"
#include "q8kv.h"
#include "ring.cuh"

namespace luce {

constexpr int kQ8MaxChunks = 160;

// A chunk's weights, and so its sums, are 2^15 e^(s - m): the tree attention's
// reason, f16 has no digits below 2^-24.
constexpr float kQ8Up = 15.0f, kQ8Down = 1.0f / 32768.0f;

// Scores in powers of two: e^(s - m) = 2^(log2 dot - max).  The scale's sign goes
// into q.
struct Q8Scale {
    float sign, log2;
};

int q8kv_max_chunks(int max_sealed, int Hkv) { return max_sealed > 0 ? tree_max_chunks(std::max(max_sealed, kQ8Page), Hkv) : 0; }

size_t q8kv_part_bytes(int64_t n_part) { return (size_t)n_part * (kHeadDim + 2) * sizeof(float); }

int64_t q8kv_chunks(Q8Batch& b, int Hq, int Hkv)
{
    int64_t part = 0;
    for (int i = 0; i < b.n_view; ++i) {
        Q8View& v = b.view[i];
        const int all = (v.sealed + kQ8Page - 1) / kQ8Page;
        v.front = all;
        v.back = all;
        if (v.window > 0) {
            // the earliest key that a node without ancestors sees through the window
            const int first = v.sealed + v.tail - v.window + 1;
            v.back = first >= v.sealed ? all : std::max(0, first) / kQ8Page;
            v.front = std::min(v.back, (std::min(v.sinks, v.sealed) + kQ8Page - 1) / kQ8Page);
            if (v.front >= v.back) v.front = v.back = all;
        }
        v.n_tile = v.front + all - v.back;
        v.chunk = v.n_tile ? tree_chunk_keys(v.n_tile * kQ8Page, Hkv) / kQ8Page : 1;
        v.n_chunk = (v.n_tile + v.chunk - 1) / v.chunk;
        v.part0 = part;
        part += (int64_t)v.n_chunk * v.n_nodes * Hq;
    }
    return part;
}

// The key that tile t of a view's starts with.
__device__ __forceinline__ int q8_tile_key(const Q8View& v, int t) { return (t < v.front ? t : t - v.front + v.back) * kQ8Page; }

__device__ __forceinline__ float q8_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---------------------------------------------------------------- chunks

// One CTA of 128 threads a chunk and KV head; rows in groups of 32.  Scores: a key
// a thread.  Sums: a dim a thread.
constexpr int kQ8Rows = 32;

__global__ void __launch_bounds__(128)
q8kv_chunk_kernel(const float* q, const __grid_constant__ Q8Batch b, int Hq, int Hkv, Q8Scale scale,
                  float* __restrict__ part_o, float* __restrict__ part_ml)
{
    __shared__ __align__(16) float qs[kQ8Rows][kHeadDim];
    __shared__ float ps[kQ8Rows][kQ8Page];
    __shared__ float ms[kQ8Rows], ls[kQ8Rows], al[kQ8Rows];
    pdl_trigger();
    int u = blockIdx.x, vi = 0;
    while (vi + 1 < b.n_view && u >= Hkv * b.view[vi].n_chunk) u -= Hkv * b.view[vi++].n_chunk;
    const Q8View& v = b.view[vi];
    const int c = u / Hkv, g = u % Hkv, GQ = Hq / Hkv, R = v.n_nodes * GQ, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int t0 = c * v.chunk, t1 = min(t0 + v.chunk, v.n_tile), total = v.sealed + v.tail;
    const int64_t pr = v.part0 + ((int64_t)c * Hkv + g) * R;
    pdl_wait();
    for (int r0 = 0; r0 < R; r0 += kQ8Rows) {
        const int n = min(kQ8Rows, R - r0);
        __syncthreads();
        for (int r = 0; r < n; ++r) {
            const int i = r0 + r;
            qs[r][tid] = __fmul_rn(ld_placed_f(q + ((int64_t)(v.row0 + i / GQ) * Hq + g * GQ + i % GQ) * kHeadDim + tid), scale.sign);
        }
        if (tid < kQ8Rows) {
            ms[tid] = -INFINITY;
            ls[tid] = 0.0f;
        }
        float o[kQ8Rows];
#pragma unroll
        for (int r = 0; r < kQ8Rows; ++r) o[r] = 0.0f;
        for (int t = t0; t < t1; ++t) {
            const int key0 = q8_tile_key(v, t), page = v.table ? ld_placed_i(v.table + key0 / kQ8Page) : key0 / kQ8Page;
            const bool in = page >= 0 && page < v.n_pages;
            const int64_t at = (int64_t)page * v.page_stride + (int64_t)g * kQ8PageBytes + tid * 128;
            const float* sc = v.scales + (int64_t)page * v.scale_stride + g * kQ8PageScales;
            __syncthreads();
            {
                uint4 x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = in ? ld_placed_u4(v.k_codes + at + 16 * e) : make_uint4(0, 0, 0, 0);
                const int key = key0 + tid;
                const float ks = in && key < v.sealed ? __fmul_rn(ld_placed_f(sc + warp), scale.log2) : 0.0f;
                for (int r = 0; r < n; ++r) {
                    float dot = 0.0f;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint32_t w = reinterpret_cast<const uint32_t*>(x)[e];
                        const float4 y = *reinterpret_cast<const float4*>(&qs[r][4 * e]);
                        dot = __fmaf_rn(y.x, (float)(int8_t)w, dot);
                        dot = __fmaf_rn(y.y, (float)(int8_t)(w >> 8), dot);
                        dot = __fmaf_rn(y.z, (float)(int8_t)(w >> 16), dot);
                        dot = __fmaf_rn(y.w, (float)(int8_t)(w >> 24), dot);
                    }
                    const int p = total + b.row[v.row0 + (r0 + r) / GQ].n_path - 1;
                    const bool seen = key < v.sealed && (v.window == 0 || key < v.sinks || p - key < v.window);
                    ps[r][tid] = seen ? __fmul_rn(dot, ks) : -INFINITY;
                }
            }
            __syncthreads();
            for (int r = warp; r < n; r += 4) {
                float x[4], top = ms[r];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = ps[r][lane + 32 * e];
                    top = fmaxf(top, x[e]);
                }
                top = warp_max(top);
                const float ref = top == -INFINITY ? 0.0f : top;
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[e] = q8_exp2(__fadd_rn(__fsub_rn(x[e], ref), kQ8Up));
                    ps[r][lane + 32 * e] = x[e];
                    sum = __fadd_rn(sum, x[e]);
                }
                sum = warp_sum_butterfly(sum);
                __syncwarp();
                if (lane == 0) {
                    al[r] = q8_exp2(__fsub_rn(ms[r], ref));
                    ls[r] = __fmaf_rn(ls[r], al[r], sum);
                    ms[r] = top;
                }
            }
            __syncthreads();
            uint4 x[8];
            float vs[4];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = in ? ld_placed_u4(v.v_codes + at + 16 * e) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) vs[e] = in && key0 + 32 * e < v.sealed ? ld_placed_f(sc + 4 + e) : 0.0f;
#pragma unroll
            for (int r = 0; r < kQ8Rows; ++r) {
                if (r >= n) break;
                o[r] = __fmul_rn(o[r], al[r]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t w = reinterpret_cast<const uint32_t*>(x)[8 * e + i];
                        const float* p = &ps[r][32 * e + 4 * i];
                        sum = __fmaf_rn(p[0], (float)(int8_t)w, sum);
                        sum = __fmaf_rn(p[1], (float)(int8_t)(w >> 8), sum);
                        sum = __fmaf_rn(p[2], (float)(int8_t)(w >> 16), sum);
                        sum = __fmaf_rn(p[3], (float)(int8_t)(w >> 24), sum);
                    }
                    o[r] = __fmaf_rn(sum, vs[e], o[r]);
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kQ8Rows; ++r)
            if (r < n) part_o[(pr + r0 + r) * kHeadDim + tid] = o[r];
        if (tid < n) *reinterpret_cast<float2*>(part_ml + 2 * (pr + r0 + tid)) = make_float2(ms[tid], ls[tid]);
    }
}

// ---------------------------------------------------------------- merge

// Merge of one (row, query head): the chunks' results, the tail's keys and the
// path's.  One CTA of 4 warps.  Scores of the f16 keys: eight lanes a key, 16 dims
// each, key 16 i + 4 warp + lane / 8 in step i.  Sums: four dims a lane, warp w takes
// chunks w, w + 4, .. in order, then f16 keys w, w + 4, .. in order; the four are added
// in order.  Bound by latency: K and V of the first 48 f16 keys (a tail that is
// sealed at every step and the longest path), statistics and chunk sums are all
// asked for before anything is used.
constexpr int kQ8Ahead = 8;       // chunk sums in flight per warp
constexpr int kQ8Keys = 48;       // f16 keys in flight
constexpr int kQ8MaxKeys = kQ8MaxTail + kMaxTree;

__device__ __forceinline__ float4 q8_half4(uint2 x)
{
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&x.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&x.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void q8_axpy(float4& o, float4 x, float a)
{
    o.x = __fmaf_rn(x.x, a, o.x);
    o.y = __fmaf_rn(x.y, a, o.y);
    o.z = __fmaf_rn(x.z, a, o.z);
    o.w = __fmaf_rn(x.w, a, o.w);
}

__global__ void __launch_bounds__(kHeadDim)
q8kv_merge_kernel(const float* q, const __grid_constant__ Q8Batch b, int Hq, int Hkv, Q8Scale scale, const float* part_o,
                  const float* part_ml, float* __restrict__ out, int8_t* __restrict__ out_q, float* __restrict__ out_d)
{
    __shared__ float ps[kQ8MaxKeys];          // the f16 keys' products
    __shared__ float4 os[4][kHeadDim / 4];    // the warps' sums
    pdl_trigger();
    const int h = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const TreeRow& row = b.row[r];
    const Q8View& v = b.view[row.view];
    const int GQ = Hq / Hkv, g = h / GQ, R = v.n_nodes * GQ, nch = v.n_chunk, n = v.tail + row.n_path, total = v.sealed + v.tail;
    const int64_t pr0 = v.part0 + (int64_t)g * R + row.node * GQ + h % GQ, pstep = (int64_t)Hkv * R;
    const size_t rh = (size_t)r * Hq + h;
    const int pos = total + row.n_path - 1;
    // f16 key a: the tail's, then the path's; its row in the tail
    auto place = [&](int a) { return a < v.tail ? a : v.tail + row.path[a - v.tail]; };
    auto seen = [&](int a) { return a < n && (v.window == 0 || v.sealed + a < v.sinks || pos - (v.sealed + a) < v.window); };
    pdl_wait();
    const int part = lane & 7;
    float4 qv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) qv[e] = ld_placed_f4(q + rh * kHeadDim + 16 * part + 4 * e);
    uint4 kx[kQ8Keys / 16][2];
    uint2 vx[kQ8Keys / 4];
    auto load_k = [&](int base) {
#pragma unroll
        for (int i = 0; i < kQ8Keys / 16; ++i) {
            const int a = base + 16 * i + 4 * warp + (lane >> 3);
            kx[i][0] = kx[i][1] = make_uint4(0, 0, 0, 0);
            if (seen(a)) {
                const __half* p = v.k + g * v.head_stride + place(a) * v.tok_stride + 16 * part;
                kx[i][0] = ld_placed_u4(p);
                kx[i][1] = ld_placed_u4(p + 8);
            }
        }
    };
    auto load_v = [&](int base) {
#pragma unroll
        for (int i = 0; i < kQ8Keys / 4; ++i) {
            const int a = base + 4 * i + warp;
            vx[i] = make_uint2(0, 0);
            if (seen(a)) vx[i] = ld_placed_u2(v.v + g * v.head_stride + place(a) * v.tok_stride + 4 * lane);
        }
    };
    load_k(0);
    load_v(0);
    constexpr int kStats = kQ8MaxChunks / 32;
    float w[kStats], ls[kStats], L = 0.0f, M = -INFINITY;  // every warp has all chunks': chunk lane + 32 j in its lane
#pragma unroll
    for (int j = 0; j < kStats; ++j) {
        const int c = lane + 32 * j;
        w[j] = -INFINITY;
        ls[j] = 0.0f;
        if (c < nch) {
            const float2 ml = ld_placed_f2(part_ml + 2 * (pr0 + c * pstep));
            w[j] = ml.x;
            ls[j] = ml.y;
        }
    }
    float4 ov[kQ8Ahead];
    auto load_o = [&](int j) {
#pragma unroll
        for (int e = 0; e < kQ8Ahead; ++e) {
            const int c = 4 * (j + e) + warp;
            if (c < nch) ov[e] = ld_placed_cg_f4(part_o + (pr0 + c * pstep) * kHeadDim + 4 * lane);
        }
    };
    load_o(0);
    for (int base = 0; base < n; base += kQ8Keys) {
        if (base > 0) load_k(base);
#pragma unroll
        for (int i = 0; i < kQ8Keys / 16; ++i) {
            const int a = base + 16 * i + 4 * warp + (lane >> 3);
            float dot = 0.0f;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint4 x = kx[i][e >> 1];
                const float4 k = q8_half4(e & 1 ? make_uint2(x.z, x.w) : make_uint2(x.x, x.y));
                dot = __fmaf_rn(qv[e].w, k.w, __fmaf_rn(qv[e].z, k.z, __fmaf_rn(qv[e].y, k.y, __fmaf_rn(qv[e].x, k.x, dot))));
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) dot = __fadd_rn(dot, __shfl_xor_sync(0xffffffffu, dot, o));
            if (part == 0 && a < n) ps[a] = seen(a) ? __fmul_rn(__fmul_rn(dot, scale.sign), scale.log2) : -INFINITY;
        }
    }
    __syncthreads();
    constexpr int kKeyStats = kQ8MaxKeys / 32;
    float p[kKeyStats];  // key lane + 32 j
#pragma unroll
    for (int j = 0; j < kKeyStats; ++j) {
        p[j] = lane + 32 * j < n ? ps[lane + 32 * j] : -INFINITY;
        M = fmaxf(M, p[j]);
    }
#pragma unroll
    for (int j = 0; j < kStats; ++j) M = fmaxf(M, w[j]);
    M = warp_max(M);  // (a row sees itself: there is one)
#pragma unroll
    for (int j = 0; j < kStats; ++j) {
        w[j] = __fmul_rn(q8_exp2(__fsub_rn(w[j], M)), kQ8Down);
        L = __fmaf_rn(ls[j], w[j], L);
    }
#pragma unroll
    for (int j = 0; j < kKeyStats; ++j) {
        p[j] = q8_exp2(__fsub_rn(p[j], M));
        L = __fadd_rn(L, p[j]);
    }
    L = warp_sum_butterfly(L);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < kQ8MaxChunks / 4; ++j) {  // chunk 4 j + warp: its weight is in lane (4 j + warp) & 31's w[j >> 3]
        const int c = 4 * j + warp;
        if ((j & (kQ8Ahead - 1)) == 0 && j > 0) {
            if (4 * j >= nch) break;
            load_o(j);
        }
        const float f = __shfl_sync(0xffffffffu, w[j >> 3], c & 31);
        if (c < nch) q8_axpy(o, ov[j & (kQ8Ahead - 1)], f);
    }
    for (int base = 0; base < n; base += kQ8Keys) {
        if (base > 0) load_v(base);
#pragma unroll
        for (int i = 0; i < kQ8Keys / 4; ++i) {
            const int a = base + 4 * i + warp;  // (its weight: recomputed from ps, the same in every lane)
            if (a < n) q8_axpy(o, q8_half4(vx[i]), q8_exp2(__fsub_rn(ps[a], M)));
        }
    }
    os[warp][lane] = o;
    __syncthreads();
    const float* of = &os[0][0].x;
    const float O = __fadd_rn(__fadd_rn(of[tid], of[kHeadDim + tid]), __fadd_rn(of[2 * kHeadDim + tid], of[3 * kHeadDim + tid]));
    const float val = __fdiv_rn(O, L);
    out[rh * kHeadDim + tid] = val;
    if (out_q) {
        float dd;
        const int code = q8_quantize_lane(val, &dd);
        out_q[rh * kHeadDim + tid] = (int8_t)code;
        if (lane == 0) out_d[(rh * kHeadDim + tid) / 32] = dd;
    }
}

cudaError_t launch_q8kv_attention(const float* q, const Q8Batch& b, int Hq, int Hkv, float scale, void* part, float* out,
                                  int8_t* out_q, float* out_d, cudaStream_t s)
{
    int64_t units = 0, n_part = 0;
    for (int i = 0; i < b.n_view; ++i) {
        units += (int64_t)b.view[i].n_chunk * Hkv;
        n_part += (int64_t)b.view[i].n_chunk * b.view[i].n_nodes * Hq;
    }
    float* part_o = (float*)part;
    float* part_ml = part_o + n_part * kHeadDim;
    const Q8Scale sc = {scale < 0 ? -1.0f : 1.0f, (float)(std::fabs((double)scale) * 1.4426950408889634)};
    if (units > 0) {
        const cudaError_t e = launch_pdl(q8kv_chunk_kernel, dim3((unsigned)units), dim3(128), s, q, b, Hq, Hkv, sc, part_o, part_ml);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    const cudaError_t e = launch_pdl(q8kv_merge_kernel, dim3(Hq, b.n_row), dim3(kHeadDim), s, q, b, Hq, Hkv, sc,
                                     (const float*)part_o, (const float*)part_ml, out, out_q, out_d);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return cudaSuccess;
}

}  // namespace luce
