// tree.cu - attention of the nodes of draft trees over slots' caches.
//
// A slot verifies a tree of drafted tokens: node j sees the cache's prefix
// (keys 0 .. len-1), its ancestors and itself, whose K/V rows sit behind the
// prefix at len + node.  For row r of node j and query head h
//   out = sum_i e^(s_i - m) v_i / l,  s_i = scale q.k_i,  m = max s_i,  l = sum e^(s_i - m).
// The prefix, which every node of the tree sees, is cut into chunks of
// tree_chunk_keys(len) keys; each chunk yields (m, l, sum e^(s - m) v) per row
// and the merge adds the chunks in order, then the node's own path, key by key
// from the prefix down to the node.  A node's bits so follow from its prefix
// and its path alone: the other branches of its tree, which lie between its
// ancestors in the cache, take no part in any of its sums.
#include <math.h>

#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"

namespace luce {

// Prefixes up to kTreeShort keys take 128-key chunks, up to kTreeMid 512, longer ones 1,024.
constexpr int kTreeShort = 8192, kTreeMid = 32768;

int tree_chunk_keys(int len) { return len <= kTreeShort ? 128 : (len <= kTreeMid ? 512 : 1024); }

int tree_max_chunks(int max_len)
{
    int most = 0;
    for (int len : {std::min(max_len, kTreeShort), std::min(max_len, kTreeMid), max_len})
        most = std::max(most, (len + tree_chunk_keys(len) - 1) / tree_chunk_keys(len));
    return most;
}

constexpr int kMaxTreeChunkKeys = 1024;
constexpr int kMaxTreeChunks = 128;

// A view chunk's partial results: part_o [row][128] and part_ml [row][2] with
// row = part0 + (chunk * Hkv + g) * R + i, i = node * GQ + head of the group.
size_t tree_part_bytes(int64_t n_part) { return (size_t)n_part * (kHeadDim + 2) * sizeof(float); }

__device__ __forceinline__ const __half* tree_key(const TreeView& v, const __half* base, int g, int key)
{
    if (!v.pages) return base + (int64_t)g * v.head_stride + (int64_t)key * v.tok_stride;
    const int p = __ldg(v.pages + (key >> 7));
    if (p < 0 || p >= v.n_pages) return nullptr;
    return base + (int64_t)p * v.page_stride + (int64_t)g * v.head_stride + (int64_t)(key & 127) * v.tok_stride;
}

__global__ void __launch_bounds__(128)
tree_chunk_kernel(const float* __restrict__ q, TreeBatch b, int Hq, int Hkv, float scale, float* __restrict__ part_o,
                  float* __restrict__ part_ml, float* __restrict__ scores, int64_t lds)
{
    __shared__ float s[kMaxTreeChunkKeys];
    __shared__ float qs[kHeadDim];
    __shared__ float red[4];
    pdl_trigger();
    const int g = blockIdx.y, tid = threadIdx.x, GQ = Hq / Hkv;
    int c = blockIdx.x, vi = 0;
    while (vi + 1 < b.n_view && c >= b.view[vi].n_chunk) c -= b.view[vi++].n_chunk;
    const TreeView& v = b.view[vi];
    const int key0 = c * v.chunk, n = min(v.chunk, v.len - key0), R = v.n_nodes * GQ;
    pdl_wait();
    for (int i = 0; i < R; ++i) {
        const int row = v.row0 + i / GQ, h = g * GQ + i % GQ;
        qs[tid] = q[((size_t)row * Hq + h) * kHeadDim + tid];
        __syncthreads();
        float m = -INFINITY;
        for (int j = tid; j < n; j += 128) {
            const __half* k = tree_key(v, v.k, g, key0 + j);
            float acc = 0.0f;
            for (int d = 0; k && d < kHeadDim; ++d) acc = __fmaf_rn(qs[d], __half2float(k[d]), acc);
            const float x = __fmul_rn(acc, scale);
            s[j] = x;
            m = fmaxf(m, x);
            if (scores) scores[((size_t)row * Hq + h) * lds + key0 + j] = x;
        }
        m = warp_max(m);
        if ((tid & 31) == 0) red[tid >> 5] = m;
        __syncthreads();
        m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
        const float ref = m == -INFINITY ? 0.0f : m;
        __syncthreads();
        float l = 0.0f;
        for (int j = tid; j < n; j += 128) {
            const float p = expf(__fsub_rn(s[j], ref));
            s[j] = p;
            l = __fadd_rn(l, p);
        }
        l = warp_sum_butterfly(l);
        if ((tid & 31) == 0) red[tid >> 5] = l;
        __syncthreads();
        const int64_t pr = v.part0 + ((int64_t)c * Hkv + g) * R + i;
        float o = 0.0f;
        for (int j = 0; j < n; ++j) {
            const __half* x = tree_key(v, v.v, g, key0 + j);
            if (x) o = __fmaf_rn(s[j], __half2float(x[tid]), o);
        }
        part_o[pr * kHeadDim + tid] = o;
        if (tid == 0) {
            part_ml[2 * pr] = m;
            part_ml[2 * pr + 1] = __fadd_rn(__fadd_rn(red[0], red[1]), __fadd_rn(red[2], red[3]));
        }
        __syncthreads();
    }
}

// Merge of one (row, query head): the prefix's chunks in order, then the
// node's path from the prefix down.  One thread per dim.
__global__ void __launch_bounds__(kHeadDim)
tree_merge_kernel(const float* __restrict__ q, TreeBatch b, int Hq, int Hkv, float scale,
                  const float* __restrict__ part_o, const float* __restrict__ part_ml, float* __restrict__ out,
                  float* __restrict__ scores, int64_t lds, float* __restrict__ stats, int8_t* __restrict__ out_q,
                  float* __restrict__ out_d)
{
    __shared__ float w[kMaxTreeChunks];
    __shared__ float ps[kMaxTree];
    __shared__ float Ls;
    pdl_trigger();
    const int h = blockIdx.x, r = blockIdx.y, d = threadIdx.x, lane = d & 31, warp = d >> 5;
    const TreeRow& row = b.row[r];
    const TreeView& v = b.view[row.view];
    const int GQ = Hq / Hkv, g = h / GQ, R = v.n_nodes * GQ, np = row.n_path, nch = v.n_chunk;
    const int64_t pr0 = v.part0 + (int64_t)g * R + row.node * GQ + h % GQ, pstep = (int64_t)Hkv * R;
    pdl_wait();
    const float* qr = q + ((size_t)r * Hq + h) * kHeadDim;
    const float4 qv = *reinterpret_cast<const float4*>(qr + 4 * lane);
    for (int a = warp; a < np; a += 4) {
        const __half* k = tree_key(v, v.k, g, v.len + row.path[a]);
        float acc = 0.0f;
        if (k) {
            const uint2 kv = *reinterpret_cast<const uint2*>(k + 4 * lane);
            const float2 k0 = __half22float2(*reinterpret_cast<const __half2*>(&kv.x));
            const float2 k1 = __half22float2(*reinterpret_cast<const __half2*>(&kv.y));
            acc = __fmaf_rn(qv.w, k1.y, __fmaf_rn(qv.z, k1.x, __fmaf_rn(qv.y, k0.y, __fmul_rn(qv.x, k0.x))));
        }
        acc = warp_sum_butterfly(acc);
        if (lane == 0) ps[a] = __fmul_rn(acc, scale);
    }
    __syncthreads();
    float* sc = scores ? scores + ((size_t)r * Hq + h) * lds + v.len : nullptr;
    if (sc && d < v.n_nodes) {
        float x = -INFINITY;
        for (int a = 0; a < np; ++a)
            if (row.path[a] == d) x = ps[a];
        sc[d] = x;
    }
    __syncthreads();  // the scores are read before the path's become weights
    if (warp == 0) {
        float M = -INFINITY;
        for (int c = lane; c < nch; c += 32) {
            const float m = __ldcg(part_ml + 2 * (pr0 + c * pstep));
            w[c] = m;
            M = fmaxf(M, m);
        }
        const float mine = lane < np ? ps[lane] : -INFINITY;
        M = warp_max(fmaxf(M, mine));
        const float ref = M == -INFINITY ? 0.0f : M;
        float L = 0.0f;
        for (int c = lane; c < nch; c += 32) {
            const float f = expf(__fsub_rn(w[c], ref));
            w[c] = f;
            L = __fmaf_rn(__ldcg(part_ml + 2 * (pr0 + c * pstep) + 1), f, L);
        }
        L = warp_sum_butterfly(L);
        __syncwarp();
        if (lane < np) ps[lane] = expf(__fsub_rn(mine, ref));
        __syncwarp();
        for (int a = 0; a < np; ++a) L = __fadd_rn(L, ps[a]);
        if (lane == 0) {
            Ls = L;
            if (stats) {
                stats[2 * ((size_t)r * Hq + h)] = M;
                stats[2 * ((size_t)r * Hq + h) + 1] = L;
            }
        }
    }
    __syncthreads();
    float O = 0.0f;
    for (int c = 0; c < nch; ++c) O = __fmaf_rn(__ldcg(part_o + (pr0 + c * pstep) * kHeadDim + d), w[c], O);
    for (int a = 0; a < np; ++a) {
        const __half* x = tree_key(v, v.v, g, v.len + row.path[a]);
        if (x) O = __fmaf_rn(ps[a], __half2float(x[d]), O);
    }
    const float val = __fdiv_rn(O, Ls);
    const size_t oi = ((size_t)r * Hq + h) * kHeadDim + d;
    out[oi] = val;
    if (out_q) {
        float dd;
        const int code = q8_quantize_lane(val, &dd);
        out_q[oi] = (int8_t)code;
        if (lane == 0) out_d[oi / 32] = dd;
    }
}

cudaError_t launch_tree_attention(const float* q, const TreeBatch& b, int Hq, int Hkv, float scale, void* part,
                                  float* out, float* scores, int64_t lds, float* stats, int8_t* out_q, float* out_d,
                                  cudaStream_t s)
{
    int chunks = 0;
    int64_t n_part = 0;
    for (int i = 0; i < b.n_view; ++i) {
        chunks += b.view[i].n_chunk;
        n_part += (int64_t)b.view[i].n_chunk * b.view[i].n_nodes * Hq;
    }
    float* part_o = (float*)part;
    float* part_ml = part_o + n_part * kHeadDim;
    if (chunks > 0) {
        const cudaError_t e = launch_pdl(tree_chunk_kernel, dim3(chunks, Hkv), dim3(128), s, q, b, Hq, Hkv, scale,
                                         part_o, part_ml, scores, lds);
        count_launches(1);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e =
        launch_pdl(tree_merge_kernel, dim3(Hq, b.n_row), dim3(kHeadDim), s, q, b, Hq, Hkv, scale,
                   (const float*)part_o, (const float*)part_ml, out, scores, lds, stats, out_q, out_d);
    count_launches(1);
    return e;
}

}  // namespace luce
