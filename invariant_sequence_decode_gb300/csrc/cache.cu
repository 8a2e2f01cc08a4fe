// cache.cu - what happens to a slot's cache between steps: the commit of a
// verified tree's accepted path, and eviction by accumulated attention weight.
#include <math.h>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"

namespace luce {

// ---------------------------------------------------------------- commit
//
// Rows: one warp per (slot, layer, KV head), lanes 0..15 the 16-byte pieces of
// K's rows, lanes 16..31 of V's.  A piece is moved by one thread, so its rows
// are all read before any is written and a path may move onto itself.
//
// Weights: acc_j += sum over accepted rows r and the group's heads h of
// e^(s_rhj - m_rh) / l_rh; a stream over the scores (4 A GQ bytes per key
// against 8 of acc), four keys per thread.
constexpr int kCommitThreads = 256;
constexpr int kCommitKeys = 4 * kCommitThreads;

__device__ __forceinline__ float commit_weight(const float* __restrict__ sc, int64_t lds, int64_t col, const float2* ml,
                                               int n)
{
    float w = 0.0f;
    for (int i = 0; i < n; ++i) w = __fmaf_rn(expf(__fsub_rn(sc[i * lds + col], ml[i].x)), ml[i].y, w);
    return w;
}

__global__ void __launch_bounds__(kCommitThreads)
tree_commit_kernel(CommitBatch b, int n_layers, int Hq, int Hkv, const float* __restrict__ scores, int n_rows,
                   int64_t lds, const float* __restrict__ stats, int move_ctas)
{
    __shared__ float2 ml[kMaxTree * 8];  // (m, 1 / l) of the accepted rows' heads
    pdl_trigger();
    const CommitSlot& sl = b.slot[blockIdx.y];
    const int tid = threadIdx.x, A = sl.n_path, heads = n_layers * Hkv;
    if ((int)blockIdx.x < move_ctas) {
        const int lane = tid & 31, lh = blockIdx.x * (kCommitThreads / 32) + (tid >> 5);
        pdl_wait();
        if (lh >= heads || A == 0) return;
        uint4* p = reinterpret_cast<uint4*>(lane < 16 ? sl.k : sl.v) + ((int64_t)lh * sl.cap + sl.len) * 16 + (lane & 15);
        uint4 x[kMaxTree];
#pragma unroll
        for (int i = 0; i < kMaxTree; ++i)
            if (i < A && sl.path[i] != i) x[i] = p[sl.path[i] * 16];
#pragma unroll
        for (int i = 0; i < kMaxTree; ++i)
            if (i < A && sl.path[i] != i) p[i * 16] = x[i];
        if (sl.pos && lane < A) sl.pos[(int64_t)lh * sl.cap + sl.len + lane] = sl.pos0 + lane;
        return;
    }
    const int64_t tiles = (sl.len + A + kCommitKeys - 1) / kCommitKeys;
    int64_t at = blockIdx.x - move_ctas;
    pdl_wait();
    if (!sl.acc || A == 0) return;
    const int GQ = Hq / Hkv, lh = (int)(at / tiles);
    if (lh >= heads) return;
    const int l = lh / Hkv, g = lh % Hkv;
    for (int i = tid; i < A * GQ; i += kCommitThreads) {
        const int64_t r = (int64_t)l * n_rows + sl.row0 + sl.path[i / GQ];
        const float* st = stats + 2 * (r * Hq + g * GQ + i % GQ);
        ml[i] = make_float2(st[0] == -INFINITY ? 0.0f : st[0], st[1] == 0.0f ? 0.0f : __fdiv_rn(1.0f, st[1]));
    }
    __syncthreads();
    float* acc = sl.acc + (int64_t)lh * sl.cap;
    const int j0 = (int)(at % tiles) * kCommitKeys;
    for (int j = j0 + tid; j < min(j0 + kCommitKeys, sl.len + A); j += kCommitThreads) {
        const int col = j < sl.len ? j : sl.len + sl.path[j - sl.len];
        float w = 0.0f;
        for (int a = 0; a < A; ++a) {
            const int64_t r = (int64_t)l * n_rows + sl.row0 + sl.path[a];
            w = __fadd_rn(w, commit_weight(scores + (r * Hq + g * GQ) * lds, lds, col, ml + a * GQ, GQ));
        }
        acc[j] = j < sl.len ? __fadd_rn(acc[j], w) : w;
    }
}

cudaError_t launch_tree_commit(const CommitBatch& b, int n_layers, int Hq, int Hkv, const float* scores, int n_rows,
                               int64_t lds, const float* stats, cudaStream_t s)
{
    const int64_t heads = (int64_t)n_layers * Hkv;
    int64_t tiles = 0;
    for (int i = 0; i < b.n_slot; ++i)
        if (b.slot[i].acc && b.slot[i].n_path > 0)
            tiles = max(tiles, (int64_t)(b.slot[i].len + b.slot[i].n_path + kCommitKeys - 1) / kCommitKeys);
    const int64_t move = (heads + kCommitThreads / 32 - 1) / (kCommitThreads / 32);
    const cudaError_t e = launch_pdl(tree_commit_kernel, dim3((unsigned)(move + heads * tiles), b.n_slot),
                                     dim3(kCommitThreads), s, b, n_layers, Hq, Hkv, scores, n_rows, lds, stats,
                                     (int)move);
    count_launches(1);
    return e;
}

// ---------------------------------------------------------------- eviction
//
// One CTA per (slot, layer, KV head).  The n = len - budget keys that leave
// are the lowest of an ordered 32-bit form of acc (NaN lowest, protected keys
// highest): a radix selection finds the n-th lowest value T, 8 bits at a pass
// over a 256-bin histogram, and how many keys equal to T leave; of those the
// ones with the highest indexes do.  Then holes (index < budget, leaving) and
// comers (index >= budget, staying) are found in ascending order and paired.
constexpr int kEvictThreads = 1024;

__device__ __forceinline__ uint32_t evict_rank(float a, int pos, const EvictSlot& sl)
{
    if (pos < sl.sinks || (int64_t)pos >= (int64_t)sl.next_pos - sl.recent) return 0xffffffffu;
    if (a != a) return 0u;
    const uint32_t u = __float_as_uint(__fadd_rn(a, 0.0f));  // -0 and 0 are equal weights
    return u >> 31 ? ~u : u | 0x80000000u;  // at most 0xff800000
}

// Exclusive prefix of flag over the CTA's threads, and their number.
__device__ __forceinline__ int evict_prefix(bool flag, int* warp_n, int* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t m = __ballot_sync(0xffffffffu, flag);
    __syncthreads();
    if (lane == 0) warp_n[warp] = __popc(m);
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < kEvictThreads / 32; ++i) {
        if (i < warp) before += warp_n[i];
        all += warp_n[i];
    }
    *total = all;
    return before + __popc(m & ((1u << lane) - 1));
}

__global__ void __launch_bounds__(kEvictThreads)
kv_evict_kernel(EvictBatch b)
{
    __shared__ int hist[256];
    __shared__ int warp_n[kEvictThreads / 32];
    __shared__ int digit, below;
    __shared__ int hole[2 * kEvictThreads], come[2 * kEvictThreads];
    pdl_trigger();
    const EvictSlot& sl = b.slot[blockIdx.y];
    const int64_t lh = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float* acc = sl.acc + lh * sl.cap;
    const int32_t* pos = sl.pos + lh * sl.cap;
    float* acc_out = sl.acc_out + lh * sl.cap;
    int32_t* pos_out = sl.pos_out + lh * sl.cap;
    pdl_wait();
    const int keep = min(sl.len, sl.budget);
    for (int j = tid; j < keep; j += kEvictThreads) {  // (holes are overwritten below)
        if (acc_out != acc) acc_out[j] = acc[j];
        if (pos_out != pos) pos_out[j] = pos[j];
    }
    const int n = sl.len - sl.budget;
    if (n <= 0) return;
    uint32_t T = 0;
    int left = n;  // keys that leave among those sharing T's leading digits
    for (int sh = 24; sh >= 0; sh -= 8) {
        __syncthreads();
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        for (int j = tid; j < sl.len; j += kEvictThreads) {
            const uint32_t u = evict_rank(acc[j], pos[j], sl);
            if (sh == 24 || (u >> (sh + 8)) == (T >> (sh + 8))) atomicAdd(&hist[(u >> sh) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int at = 0, d = 0;
            while (d < 255 && at + hist[d] < left) at += hist[d++];
            digit = d;
            below = at;
        }
        __syncthreads();
        T |= (uint32_t)digit << sh;
        left -= below;
    }
    __syncthreads();
    // keys equal to T: the first `stay` of them stay
    const int stay = hist[T & 255] - left;
    __half* kb = sl.k + lh * sl.cap * (int64_t)kHeadDim;
    __half* vb = sl.v + lh * sl.cap * (int64_t)kHeadDim;
    int eq_h = 0;  // keys equal to T before the hole cursor
    int eq_c = 0;  // and before the comer cursor
    for (int j0 = 0; j0 < sl.budget; j0 += kEvictThreads) {
        const int j = j0 + tid;
        int all;
        evict_prefix(j < sl.budget && evict_rank(acc[min(j, sl.len - 1)], pos[min(j, sl.len - 1)], sl) == T, warp_n, &all);
        eq_c += all;
    }
    int jh = 0, jc = sl.budget, nh = 0, nc = 0;
    for (;;) {
        while (nh < kEvictThreads && jh < sl.budget) {
            const int j = jh + tid;
            const uint32_t u = j < sl.budget ? evict_rank(acc[j], pos[j], sl) : 0xffffffffu;
            int all;
            const int e = eq_h + evict_prefix(j < sl.budget && u == T, warp_n, &all);
            eq_h += all;
            const bool f = j < sl.budget && (u < T || (u == T && e >= stay));
            const int at = nh + evict_prefix(f, warp_n, &all);
            if (f) hole[at] = j;
            nh += all;
            jh += kEvictThreads;
        }
        while (nc < kEvictThreads && jc < sl.len) {
            const int j = jc + tid;
            const uint32_t u = j < sl.len ? evict_rank(acc[j], pos[j], sl) : 0;
            int all;
            const int e = eq_c + evict_prefix(j < sl.len && u == T, warp_n, &all);
            eq_c += all;
            const bool f = j < sl.len && (u > T || (u == T && e < stay));
            const int at = nc + evict_prefix(f, warp_n, &all);
            if (f) come[at] = j;
            nc += all;
            jc += kEvictThreads;
        }
        __syncthreads();
        const int m = min(nh, nc);
        if (m == 0) return;
        for (int i = warp; i < m; i += kEvictThreads / 32) {
            uint4* base = reinterpret_cast<uint4*>(lane < 16 ? kb : vb) + (lane & 15);
            base[(int64_t)hole[i] * 16] = base[(int64_t)come[i] * 16];
        }
        for (int i = tid; i < m; i += kEvictThreads) {
            acc_out[hole[i]] = acc[come[i]];
            pos_out[hole[i]] = pos[come[i]];
        }
        // the unpaired ones move to the front of their list
        int h0 = 0, h1 = 0, c0 = 0, c1 = 0;
        const int i0 = m + tid, i1 = m + tid + kEvictThreads;
        if (i0 < nh) h0 = hole[i0];
        if (i1 < nh) h1 = hole[i1];
        if (i0 < nc) c0 = come[i0];
        if (i1 < nc) c1 = come[i1];
        __syncthreads();
        if (i0 < nh) hole[tid] = h0;
        if (i1 < nh) hole[tid + kEvictThreads] = h1;
        if (i0 < nc) come[tid] = c0;
        if (i1 < nc) come[tid + kEvictThreads] = c1;
        nh -= m;
        nc -= m;
        __syncthreads();
    }
}

cudaError_t launch_kv_evict(const EvictBatch& b, int n_layers, int Hkv, cudaStream_t s)
{
    const cudaError_t e = launch_pdl(kv_evict_kernel, dim3((unsigned)n_layers * Hkv, b.n_slot), dim3(kEvictThreads), s, b);
    count_launches(1);
    return e;
}

}  // namespace luce
