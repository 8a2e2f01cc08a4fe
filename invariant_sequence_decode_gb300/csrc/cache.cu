// cache.cu - what happens to a slot's cache between steps: the commit of a
// verified tree's accepted path, and eviction by accumulated attention weight.
#include <limits.h>

#include <algorithm>
#include <cmath>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"
#include "ring.cuh"

namespace luce {

// ---------------------------------------------------------------- commit
//
// Rows: one warp per (slot, layer, KV head), lanes 0..15 the 16-byte pieces of
// K's rows, lanes 16..31 of V's.  A piece is moved by one thread, so its rows
// are all read before any is written and a path may move onto itself.
//
// Weights: acc_j += sum over accepted rows r and the group's heads h of
// e^(s_rhj - m_rh) / l_rh: a stream over the scores (4 A GQ bytes per key
// against 8 of acc), four keys per thread, always eight rows of scores in flight
// (four slots of 8 layers with 16,385 to 32,757 keys: 39.9 us, 6.2 TB/s; 4, 6 or
// 10 in flight 42.9, 44.2 and 41.5; two keys per thread 61.7).
constexpr int kCommitThreads = 128;
constexpr int kCommitKeys = 4 * kCommitThreads;
constexpr int kCommitAhead = 8;

__device__ __forceinline__ float commit_exp(float x)
{
    // e^x = 2^(x log2 e): x <= 0 but for rounding, off by at most |x| 2^-24 more
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__fmul_rn(x, 1.4426950408889634f)));
    return y;
}

__global__ void __launch_bounds__(kCommitThreads)
tree_commit_kernel(const __grid_constant__ CommitBatch b, int n_layers, int Hq, int Hkv, const float* scores, int n_rows, int64_t lds,
                   const float* stats, int move_ctas)
{
    __shared__ float2 ml[kMaxTree * 8];   // (m, 1 / l) of the accepted rows' heads
    __shared__ int64_t at[kMaxTree * 8];  // and their index in stats and scores
    pdl_trigger();
    const CommitSlot& sl = b.slot[blockIdx.y];
    const int tid = threadIdx.x, A = sl.n_path, heads = n_layers * Hkv;
    if ((int)blockIdx.x < move_ctas) {
        const int lane = tid & 31, lh = blockIdx.x * (kCommitThreads / 32) + (tid >> 5);
        pdl_wait();
        if (lh >= heads || A == 0) return;
        __half* p = (lane < 16 ? sl.k : sl.v) + lh * sl.head_step + 8 * (lane & 15);
        uint4 x[kMaxTree];
#pragma unroll
        for (int i = 0; i < kMaxTree; ++i)
            if (i < A && sl.path[i] != i) x[i] = ld_placed_u4(p + sl.at(sl.len + sl.path[i]));
#pragma unroll
        for (int i = 0; i < kMaxTree; ++i)
            if (i < A && sl.path[i] != i) *reinterpret_cast<uint4*>(p + sl.at(sl.len + i)) = x[i];
        if (sl.pos && lane < A) sl.pos[(int64_t)lh * sl.cap + sl.len + lane] = sl.pos0 + lane;
        return;
    }
    const int tiles = max(1, (sl.len + kCommitKeys - 1) / kCommitKeys);  // (the first also takes the new keys)
    const int GQ = Hq / Hkv, part = blockIdx.x - move_ctas, lh = part / tiles, tile = part - lh * tiles, n = A * GQ;
    if (!sl.acc || A == 0 || lh >= heads) return;
    const int l = lh / Hkv, g = lh % Hkv;
    for (int i = tid; i < n; i += kCommitThreads)
        at[i] = ((int64_t)l * n_rows + sl.row0 + sl.path[i / GQ]) * Hq + g * GQ + i % GQ;
    __syncthreads();
    pdl_wait();
    for (int i = tid; i < n; i += kCommitThreads) {
        const float2 st = ld_placed_f2(stats + 2 * at[i]);
        // (l = 0: e^(s - inf) adds nothing, whatever s)
        ml[i] = st.y == 0.0f ? make_float2(INFINITY, 0.0f) : make_float2(st.x == -INFINITY ? 0.0f : st.x, __fdiv_rn(1.0f, st.y));
    }
    float* acc = sl.acc + (int64_t)lh * sl.cap;
    const int j = tile * kCommitKeys + 4 * tid;
    float old[4], w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    float4 s[kCommitAhead];
    auto get = [&](int i) { return ld_placed_cs_f4(scores + at[i] * lds + j); };
    auto add = [&](int i, float4 x) {
        const float2 t = ml[i];
        w[0] = __fmaf_rn(commit_exp(__fsub_rn(x.x, t.x)), t.y, w[0]);
        w[1] = __fmaf_rn(commit_exp(__fsub_rn(x.y, t.x)), t.y, w[1]);
        w[2] = __fmaf_rn(commit_exp(__fsub_rn(x.z, t.x)), t.y, w[2]);
        w[3] = __fmaf_rn(commit_exp(__fsub_rn(x.w, t.x)), t.y, w[3]);
    };
    if (j < sl.len) {
#pragma unroll
        for (int e = 0; e < 4; ++e) old[e] = j + e < sl.len ? ld_placed_f(acc + j + e) : 0.0f;
        // the first rows are on their way while the statistics settle
        if (n >= kCommitAhead) {  // (without branches)
#pragma unroll
            for (int e = 0; e < kCommitAhead; ++e) s[e] = get(e);
        } else {
#pragma unroll
            for (int e = 0; e < kCommitAhead; ++e)
                if (e < n) s[e] = get(e);
        }
    }
    __syncthreads();
    if (tile == 0)  // a warp per new key
        for (int k = tid >> 5; k < A; k += kCommitThreads / 32) {
            float x = 0.0f;
            for (int i = tid & 31; i < n; i += 32) {
                const float t = ld_placed_f(scores + at[i] * lds + sl.len + sl.path[k]);
                x = __fmaf_rn(commit_exp(__fsub_rn(t, ml[i].x)), ml[i].y, x);
            }
            x = warp_sum_butterfly(x);
            if ((tid & 31) == 0) acc[sl.len + k] = x;
        }
    if (j >= sl.len) return;
    // a row's place is taken by the one that is eight on
    int i0 = 0;
    for (; i0 + 2 * kCommitAhead <= n; i0 += kCommitAhead) {
#pragma unroll
        for (int e = 0; e < kCommitAhead; ++e) {
            add(i0 + e, s[e]);
            s[e] = get(i0 + kCommitAhead + e);
        }
    }
    if (i0 + kCommitAhead < n) {
#pragma unroll
        for (int e = 0; e < kCommitAhead; ++e) {
            add(i0 + e, s[e]);
            if (i0 + kCommitAhead + e < n) s[e] = get(i0 + kCommitAhead + e);
        }
        i0 += kCommitAhead;
    }
#pragma unroll
    for (int e = 0; e < kCommitAhead; ++e)
        if (i0 + e < n) add(i0 + e, s[e]);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (j + e < sl.len) acc[j + e] = __fadd_rn(old[e], w[e]);
}

cudaError_t launch_tree_commit(const CommitBatch& b, int n_layers, int Hq, int Hkv, const float* scores, int n_rows,
                               int64_t lds, const float* stats, cudaStream_t s)
{
    const int64_t heads = (int64_t)n_layers * Hkv;
    int64_t tiles = 0;
    for (int i = 0; i < b.n_slot; ++i)
        if (b.slot[i].acc && b.slot[i].n_path > 0)
            tiles = std::max<int64_t>(tiles, std::max(1, (b.slot[i].len + kCommitKeys - 1) / kCommitKeys));
    const int64_t move = (heads + kCommitThreads / 32 - 1) / (kCommitThreads / 32);
    const cudaError_t e = launch_pdl(tree_commit_kernel, dim3((unsigned)(move + heads * tiles), b.n_slot),
                                     dim3(kCommitThreads), s, b, n_layers, Hq, Hkv, scores, n_rows, lds, stats,
                                     (int)move);
    count_launches(1);
    return e;
}

// ---------------------------------------------------------------- eviction
//
// One cluster of C CTAs per (slot, layer, KV head), each with a slice of the
// head's keys in shared memory as an ordered 32-bit rank (NaN 0, weights by
// value, protected keys highest).  The n = len - budget lowest leave:
//   1. a radix selection finds the n-th lowest rank T and how many keys equal
//      to T leave: three passes over the slice (11, 11, 10 bits), each a
//      histogram in shared memory; every CTA finds the digit by adding up over
//      the cluster first the sums of 32 bins, then the 32 bins that matter
//      (reading whole histograms of 8 CTAs took 4,000 cycles a pass);
//   2. of the keys equal to T the first `stay` stay, counted through the
//      cluster in index order;
//   3. holes (index < budget, leaving) and comers (index >= budget, staying)
//      are listed in index order by each CTA; the i-th hole of the cluster
//      gets the i-th comer's rows, an equal run of the pairs per warp.
// No atomics but integer counts, so nothing depends on their order.
// Bound by latency while few keys leave (each step is a cluster barrier), by
// the moved rows' bytes where a prompt is cut: 64 heads from 32,757 keys to
// 4,096 in 54.4 us, of which the rows take 36 (6.5 TB/s).
constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kEvictBins = 2048;
constexpr int kEvictSlice = 16352;  // most keys of a CTA: 8 CTAs hold 130,816
constexpr int kEvictMove = 8;   // pairs of rows in flight per warp
constexpr int kEvictAhead = 8;  // keys in flight per thread

__device__ __forceinline__ uint32_t evict_rank(float a, int pos, const EvictSlot& sl)
{
    const uint32_t u = __float_as_uint(__fadd_rn(a, 0.0f));  // -0 and 0 are equal weights
    uint32_t r = u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);  // by value, at most 0xff800000
    r = a != a ? 0u : r;
    return pos < sl.sinks || pos >= sl.next_pos - sl.recent ? 0xffffffffu : r;  // (the difference is an int: neither is negative)
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait()
{
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t far_addr(const void* p, int r)
{
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(r));
    return a;
}
__device__ __forceinline__ int far_ld(uint32_t a)
{
    int v;
    asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
// Key j's row, in rows from the (layer, KV head)'s first; -1 for a page outside
// the pool.
__device__ __forceinline__ int evict_row(const EvictSlot& sl, int j)
{
    if (!sl.pages) return j;
    const int p = ld_placed_i(sl.pages + (j >> 7));
    return p < 0 || p >= sl.n_pages ? -1 : p * sl.page_rows + (j & 127);
}

// Exclusive prefix of v over the CTA's threads; *total the sum.
__device__ __forceinline__ int block_prefix(int v, int* warp_sum, int* total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int s = lane < kEvictWarps ? warp_sum[lane] : 0;
#pragma unroll
    for (int o = 1; o < kEvictWarps; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    *total = __shfl_sync(0xffffffffu, s, kEvictWarps - 1);
    const int before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
    return x - v + (warp ? before : 0);
}

// A word of CTA r's shared memory at this CTA's address p.
template <int C>
__device__ __forceinline__ int evict_word(const int* p, int r)
{
    return C > 1 ? far_ld(far_addr(p, r)) : *p;
}

// Exclusive prefix of v over the warp.
__device__ __forceinline__ int warp_prefix(int v)
{
    const int lane = threadIdx.x & 31;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x - v;
}

template <int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kEvictThreads, 2)
kv_evict_kernel(const __grid_constant__ EvictBatch b, int slice)
{
    extern __shared__ uint32_t evict_smem[];  // ranks [slice], then the lists [slice]
    __shared__ __align__(16) int hist[2][kEvictBins];
    __shared__ int warp_sum[kEvictWarps];
    __shared__ int coarse[2][kEvictBins / 32];
    __shared__ int digit, below, equal;
    __shared__ int n_hole, n_come;  // this CTA's, for the cluster
    pdl_trigger();
    const EvictSlot& sl = b.slot[blockIdx.y];
    const int64_t lh = blockIdx.x / C;
    const int me = C > 1 ? (int)cluster_rank() : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float* acc = sl.acc + lh * sl.cap;
    const int32_t* pos = sl.pos + lh * sl.cap;
    float* acc_out = sl.acc_out + lh * sl.cap;
    int32_t* pos_out = sl.pos_out + lh * sl.cap;
    uint32_t* rank = evict_smem;
    uint32_t* list = evict_smem + slice;
    const int j0 = min(me * slice, sl.len), nj = min(slice, sl.len - j0);  // this CTA's keys
    const int n = sl.len - sl.budget;
    for (int i = tid; i < 2 * kEvictBins; i += kEvictThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
    pdl_wait();
    for (int i0 = tid; i0 < nj; i0 += kEvictAhead * kEvictThreads) {
        float a[kEvictAhead];
        int p[kEvictAhead];
#pragma unroll
        for (int e = 0; e < kEvictAhead; ++e) {
            const int j = j0 + i0 + e * kEvictThreads;
            if (j < j0 + nj) {
                a[e] = ld_placed_f(acc + j);
                p[e] = ld_placed_i(pos + j);
            }
        }
#pragma unroll
        for (int e = 0; e < kEvictAhead; ++e) {
            const int i = i0 + e * kEvictThreads;
            if (i >= nj) break;
            if (j0 + i < sl.budget) {  // (holes are overwritten below)
                if (acc_out != acc) acc_out[j0 + i] = a[e];
                if (pos_out != pos) pos_out[j0 + i] = p[e];
            }
            const uint32_t u = evict_rank(a[e], p[e], sl);
            rank[i] = u;
            if (n > 0) atomicAdd(&hist[0][u >> 21], 1);
        }
    }
    if (n <= 0) return;  // (the whole cluster)

    // 1. T, `left` keys equal to it leave
    uint32_t T = 0;
    int left = n, same = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int sh = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        int* mine = hist[pass & 1];
        if (pass > 0) {
            const int width = pass == 1 ? 11 : 10;
            const uint32_t want = T >> (sh + width), bits = (1u << width) - 1;
#pragma unroll 8
            for (int i = tid; i < nj; i += kEvictThreads) {
                const uint32_t u = rank[i];
                if (u >> (sh + width) == want) atomicAdd(&mine[(u >> sh) & bits], 1);
            }
        }
        __syncthreads();
        // sums of 32 bins, for the cluster
        {
            const int4 c = reinterpret_cast<const int4*>(mine)[tid];
            int v = c.x + c.y + c.z + c.w;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if ((lane & 7) == 0) coarse[pass & 1][tid >> 3] = v;
        }
        if (C > 1) cluster_sync(); else __syncthreads();
        if (warp == 0) {
            // the 32 bins, then the bin, in which the n-th lowest falls
            int c0 = 0, c1 = 0;
#pragma unroll
            for (int r = 0; r < C; ++r) {
                c0 += evict_word<C>(&coarse[pass & 1][2 * lane], r);
                c1 += evict_word<C>(&coarse[pass & 1][2 * lane + 1], r);
            }
            int at = warp_prefix(c0 + c1);
            uint32_t in = __ballot_sync(0xffffffffu, at < left && left <= at + c0 + c1);
            int src = __ffs(in) - 1;
            const int second = at + c0 < left;
            const int group = __shfl_sync(0xffffffffu, 2 * lane + second, src);
            const int base = __shfl_sync(0xffffffffu, at + (second ? c0 : 0), src);
            c0 = 0;
#pragma unroll
            for (int r = 0; r < C; ++r) c0 += evict_word<C>(&mine[32 * group + lane], r);
            at = base + warp_prefix(c0);
            in = __ballot_sync(0xffffffffu, at < left && left <= at + c0);
            src = __ffs(in) - 1;
            if (lane == src) {
                digit = 32 * group + lane;
                below = at;
                equal = c0;
            }
        }
        __syncthreads();
        T |= (uint32_t)digit << sh;
        left -= below;
        same = equal;
        // pass 2 counts in hist[0] again, which the other CTAs have read by
        // now only if they are past pass 1's barrier: it is cleared behind that
        if (pass == 1) {
            for (int i = tid; i < kEvictBins; i += kEvictThreads) hist[0][i] = 0;
        }
        __syncthreads();
        if (left == same) {  // the whole bin leaves: its other bits need not be known
            T |= (1u << sh) - 1;
            break;
        }
    }
    const int stay = same - left;  // the first keys equal to T, in index order

    // 2. each thread's run of the slice: keys equal to T before it (those of
    // the CTAs before this one are a bin of their last histogram)
    // (runs of odd length: their words fall into different banks)
    const int run = ((nj + kEvictThreads - 1) / kEvictThreads) | 1, r0 = min(tid * run, nj), r1 = min(r0 + run, nj);
    int all;
    uint64_t low = 0, same_as = 0;  // the run's keys below T and equal to it, a bit each
    static_assert(((kEvictSlice + kEvictThreads - 1) / kEvictThreads | 1) <= 64, "a run's keys are bits of a word");
#pragma unroll 8
    for (int i = r0; i < r1; ++i) {
        const uint32_t u = rank[i];
        low |= (uint64_t)(u < T) << (i - r0);
        same_as |= (uint64_t)(u == T) << (i - r0);
    }
    if (stay > 0) {  // (the cluster alike)
        int eq_far = 0;
#pragma unroll
        for (int r = 0; r < C - 1; ++r)
            if (r < me) eq_far += evict_word<C>(&hist[0][T & 1023], r);
        const int eq = __popcll(same_as), eq_at = eq_far + block_prefix(eq, warp_sum, &all);
        // of the run's keys equal to T the first stay - eq_at stay
        for (int k = min(max(stay - eq_at, 0), eq); k > 0; --k) same_as &= same_as - 1;
    }

    // 3. holes from the list's front, comers from its back
    const uint64_t leave = low | same_as, in = r1 - r0 == 64 ? ~0ull : (1ull << (r1 - r0)) - 1;
    const int split = min(max(sl.budget - (j0 + r0), 0), 64);  // the run's keys below the budget
    const uint64_t below_budget = split == 64 ? ~0ull : (1ull << split) - 1;
    uint64_t hs = leave & below_budget & in, cs = ~leave & ~below_budget & in;
    const int found_at = block_prefix(__popcll(hs) + (__popcll(cs) << 16), warp_sum, &all);  // each at most kEvictSlice
    for (int at = found_at & 65535; hs; hs &= hs - 1) list[at++] = j0 + r0 + __ffsll(hs) - 1;
    for (int at = slice - 1 - (found_at >> 16); cs; cs &= cs - 1) list[at--] = j0 + r0 + __ffsll(cs) - 1;
    if (tid == 0) {
        n_hole = all & 65535;
        n_come = all >> 16;
    }
    if (C > 1) cluster_sync(); else __syncthreads();
    int h_before[C], c_before[C], m = 0, mc = 0;
    {
        const int hs = lane < C ? evict_word<C>(&n_hole, lane) : 0, cs = lane < C ? evict_word<C>(&n_come, lane) : 0;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            h_before[r] = m;
            c_before[r] = mc;
            m += __shfl_sync(0xffffffffu, hs, r);
            mc += __shfl_sync(0xffffffffu, cs, r);
        }
    }
    uint4* base = reinterpret_cast<uint4*>((lane < 16 ? sl.k : sl.v) + lh * sl.head_step) + (lane & 15);
    // every warp of the cluster takes an equal run of the pairs
    const int mover = me * kEvictWarps + warp, end = (int)((int64_t)m * (mover + 1) / (C * kEvictWarps));
    for (int i0 = (int)((int64_t)m * mover / (C * kEvictWarps)); i0 < end; i0 += 32) {
        const int i = i0 + lane, cnt = min(32, end - i0);
        int to = 0, from = 0;
        if (i < end) {
            int rh = 0, rc = 0;
#pragma unroll
            for (int r = 1; r < C; ++r) {
                if (i >= h_before[r]) rh = r;
                if (i >= c_before[r]) rc = r;
            }
            int hb = 0, cb = 0;
#pragma unroll
            for (int r = 0; r < C; ++r) {
                if (r == rh) hb = h_before[r];
                if (r == rc) cb = c_before[r];
            }
            if (C > 1) {
                to = far_ld(far_addr(list + (i - hb), rh));
                from = far_ld(far_addr(list + (slice - 1 - (i - cb)), rc));
            } else {
                to = (int)list[i];
                from = (int)list[slice - 1 - i];
            }
            acc_out[to] = ld_placed_f(acc + from);
            pos_out[to] = ld_placed_i(pos + from);
        }
        int dst = i < end ? evict_row(sl, to) : -1;
        const int src = i < end ? evict_row(sl, from) : -1;
        if (src < 0) dst = -1;
        for (int k = 0; k < cnt; k += kEvictMove) {
            uint4 x[kEvictMove];
#pragma unroll
            for (int d = 0; d < kEvictMove; ++d) {
                const int f = __shfl_sync(0xffffffffu, src, (k + d) & 31);
                if (k + d < cnt && f >= 0) x[d] = ld_placed_cs_u4(base + (int64_t)f * 16);
            }
#pragma unroll
            for (int d = 0; d < kEvictMove; ++d) {
                const int t = __shfl_sync(0xffffffffu, dst, (k + d) & 31);
                if (k + d < cnt && t >= 0) base[(int64_t)t * 16] = x[d];
            }
        }
    }
    if (C > 1) cluster_sync();  // the others still read this CTA's list
}

// Few keys leave (a step's new ones): a cluster of C CTAs per head, each with a
// slice of its keys, sees them as 64-bit numbers in the order in which they
// leave (the rank, of equals the last index first), no two alike.  A CTA finds
// the n lowest of its slice: the n-th lowest of its groups' (four threads')
// lowest keys bounds them from above, and only the n groups up to it hold keys
// below it, so the few keys up to the bound go to a list, where each counts the
// lower ones.  (Should the list not hold them, for they may lie in few groups,
// the lowest is taken n times.)  Of the cluster's C n keys each counts the lower
// ones again.  Up to kFewMax keys stay in one CTA's registers, those of longer
// caches are read again, by the n groups only.
// Against the selection: 32 of 2,051 keys in 512 heads 9.7 us (it takes 16.8),
// of 32,757 keys 81 (134), in 64 heads 14.7 (18.1), in 8 heads 9.9 (13.1).
constexpr int kFewKeys = 32;  // most that leave: a lane each
constexpr int kFewPer = 16;   // keys in flight per thread
constexpr int kFewThreads = 256, kFewMax = kFewPer * kFewThreads;
constexpr int kFewLongThreads = 512, kFewLongPer = 8;
constexpr int kFewList = 512;

__device__ __forceinline__ uint64_t shfl_xor_u64(uint64_t x, int o)
{
    return __shfl_xor_sync(0xffffffffu, (unsigned long long)x, o);
}
__device__ __forceinline__ uint64_t evict_key(uint32_t rank, int j)
{
    return (uint64_t)rank << 32 | (uint32_t)(INT_MAX - j);
}

// out[k] = the k-th lowest of the CTA's `found` keys at list, k < n; four
// threads count for a key.
template <int kWarps>
__device__ __forceinline__ void few_lowest(const uint64_t* list, int found, int n, uint64_t* out)
{
    const int lane = threadIdx.x & 31;
    for (int i0 = 8 * (threadIdx.x >> 5); i0 < found; i0 += 8 * kWarps) {
        const int i = i0 + (lane >> 2);
        const uint64_t mine = list[min(i, found - 1)];
        int below = 0;
#pragma unroll 4
        for (int k = lane & 3; k < found; k += 4) below += list[k] < mine;
        below += __shfl_xor_sync(0xffffffffu, below, 1);
        below += __shfl_xor_sync(0xffffffffu, below, 2);
        if (i < found && below < n) out[below] = mine;
    }
}

template <int C, int kThreads>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(kThreads, kThreads == kFewThreads ? 4 : 2)
kv_evict_few_kernel(const __grid_constant__ EvictBatch b)
{
    constexpr int kWarps = kThreads / 32, kGroups = kThreads / 4;
    constexpr bool kOnce = kThreads == kFewThreads;
    static_assert(kGroups > kFewKeys && kFewKeys % kWarps == 0 && C * kFewKeys <= kFewList && (C == 1 || !kOnce), "");
    constexpr uint64_t kNone = ~0ull;  // (above every key)
    __shared__ uint64_t low[kGroups], list[kFewList], top[kFewKeys], all_top[kFewKeys], bound;
    __shared__ int hole[kFewKeys], come[kFewKeys], n_list, n_come;
    pdl_trigger();
    const EvictSlot& sl = b.slot[blockIdx.y];
    const int64_t lh = blockIdx.x / C;
    const int me = C > 1 ? (int)cluster_rank() : 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float* acc = sl.acc + lh * sl.cap;
    const int32_t* pos = sl.pos + lh * sl.cap;
    float* acc_out = sl.acc_out + lh * sl.cap;
    int32_t* pos_out = sl.pos_out + lh * sl.cap;
    const int n = sl.len - sl.budget, slice = (sl.len + C - 1) / C;
    const int j0 = min(me * slice, sl.len), j1 = min(j0 + slice, sl.len);  // this CTA's keys
    if (tid < kFewKeys) top[tid] = kNone;
    if (tid == 0) {
        bound = kNone;
        n_list = 0;
    }
    // this thread's kPer keys from `at`, kThreads apart
    constexpr int kPer = kOnce ? kFewPer : kFewLongPer;
    auto load = [&](int at, uint64_t* key, bool copy) {
        float a[kPer];
        int p[kPer];
        if (!kOnce && at - tid + kPer * kThreads <= j1) {  // (a batch without branches)
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                a[e] = ld_placed_f(acc + at + e * kThreads);
                p[e] = ld_placed_i(pos + at + e * kThreads);
            }
        } else {
#pragma unroll
            for (int e = 0; e < kPer; ++e)
                if (at + e * kThreads < j1) {
                    a[e] = ld_placed_f(acc + at + e * kThreads);
                    p[e] = ld_placed_i(pos + at + e * kThreads);
                }
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int j = at + e * kThreads;
            key[e] = kNone;
            if (j < j1) {
                if (copy && j < sl.budget) {
                    if (acc_out != acc) acc_out[j] = a[e];
                    if (pos_out != pos) pos_out[j] = p[e];
                }
                key[e] = evict_key(evict_rank(a[e], p[e], sl), j);
            }
        }
    };
    uint64_t key[kPer], m = kNone;
    pdl_wait();
    for (int at = j0 + tid; at < j1; at += kPer * kThreads) {
        load(at, key, true);
#pragma unroll
        for (int e = 0; e < kPer; ++e) m = min(m, key[e]);
        if (kOnce) break;
    }
    if (n <= 0) return;  // (the whole cluster)
    const bool any = m != kNone;  // (else key[] holds nothing)
    m = min(m, shfl_xor_u64(m, 1));
    m = min(m, shfl_xor_u64(m, 2));
    if ((tid & 3) == 0) low[tid >> 2] = m;
    __syncthreads();
    if (n == 1) {
        if (warp == 0) {
            m = low[lane];
#pragma unroll
            for (int i = 32; i < kGroups; i += 32) m = min(m, low[i + lane]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = min(m, shfl_xor_u64(m, o));
            if (lane == 0) top[0] = m;
            __syncwarp();
        }
    } else {
        int below = 0;  // a group's four threads count together
#pragma unroll
        for (int i = 0; i < kGroups / 4; ++i) below += low[4 * i + (tid & 3)] < m;
        below += __shfl_xor_sync(0xffffffffu, below, 1);
        below += __shfl_xor_sync(0xffffffffu, below, 2);
        if (below == n - 1 && m != kNone) bound = m;  // (fewer groups with keys: all of theirs are below kNone)
        __syncthreads();
        const uint64_t most = bound;
        // f(key) for this thread's keys up to the bound
        auto each = [&](auto f) {
            if (!any || m > most) return;
            for (int at = j0 + tid; at < j1; at += kPer * kThreads) {
                if (!kOnce) load(at, key, false);
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (key[e] <= most && key[e] != kNone) f(key[e]);
                if (kOnce) break;
            }
        };
        each([&](uint64_t x) {
            const int i = atomicAdd(&n_list, 1);
            if (i < kFewList) list[i] = x;
        });
        __syncthreads();
        if (n_list <= kFewList) {
            few_lowest<kWarps>(list, n_list, n, top);
        } else {
            uint64_t last = 0;  // (below every key)
            for (int r = 0; r < n; ++r) {
                uint64_t x = kNone;
                each([&](uint64_t k) { x = k > last ? min(x, k) : x; });
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x = min(x, shfl_xor_u64(x, o));
                if (lane == 0) low[warp] = x;
                __syncthreads();
                last = low[0];
                for (int i = 1; i < kWarps; ++i) last = min(last, low[i]);
                if (tid == 0) top[r] = last;
                __syncthreads();
            }
        }
        if (C == 1) __syncthreads();
    }
    if (C > 1) {
        __syncwarp();
        cluster_sync();  // also: no key moves before all have been read
        if (tid < C * n) {
            const uint32_t far = far_addr(&top[tid % n], tid / n);
            list[tid] = (uint64_t)(uint32_t)far_ld(far + 4) << 32 | (uint32_t)far_ld(far);
        }
        __syncwarp();
        cluster_arrive();  // (a CTA stays until the others have read its top)
        __syncthreads();
        few_lowest<kWarps>(list, C * n, n, all_top);
        __syncthreads();
    }
    const uint64_t* leaving = C > 1 ? all_top : top;
    // holes and comers in ascending order: each key's place is the number of
    // its kind below it
    if (warp == 0) {
        const int left = lane < n ? INT_MAX - (int)(uint32_t)leaving[lane] : INT_MAX;
        bool stays = lane < n;  // key budget + lane
        int below = 0;
        for (int r = 0; r < n; ++r) {
            const int j = __shfl_sync(0xffffffffu, left, r);
            if (j == sl.budget + lane) stays = false;
            if (j < left) ++below;
        }
        if (left < sl.budget) hole[below] = left;
        const uint32_t mask = __ballot_sync(0xffffffffu, stays);
        if (stays) come[__popc(mask & ((1u << lane) - 1))] = sl.budget + lane;
        if (lane == 0) n_come = __popc(mask);
    }
    __syncthreads();
    const int moves = n_come;
    uint4* base = reinterpret_cast<uint4*>((lane < 16 ? sl.k : sl.v) + lh * sl.head_step) + (lane & 15);
    uint4 x[kFewKeys / kWarps];
    int dst[kFewKeys / kWarps];
#pragma unroll
    for (int e = 0; e < kFewKeys / kWarps; ++e) {
        const int i = me + C * (warp + e * kWarps);  // the cluster's CTAs in turn
        dst[e] = -1;
        if (i >= moves) continue;
        const int to = hole[i], from = come[i], src = evict_row(sl, from);
        if (src >= 0) {
            dst[e] = evict_row(sl, to);
            x[e] = ld_placed_u4(base + (int64_t)src * 16);
        }
        if (lane == 0) acc_out[to] = ld_placed_f(acc + from);
        if (lane == 1) pos_out[to] = ld_placed_i(pos + from);
    }
#pragma unroll
    for (int e = 0; e < kFewKeys / kWarps; ++e)
        if (dst[e] >= 0) base[(int64_t)dst[e] * 16] = x[e];
    __syncwarp();
    if (C > 1) cluster_wait();
}

template <int C>
static cudaError_t launch_evict(const EvictBatch& b, int heads, int max_len, cudaStream_t s)
{
    const int slice = std::max(1, (max_len + C - 1) / C);
    static std::atomic<bool> done[kMaxDevices];
    cudaError_t e = set_smem_once(kv_evict_kernel<C>, 8 * kEvictSlice, done);
    if (e == cudaSuccess)
        e = launch_pdl_smem(kv_evict_kernel<C>, dim3((unsigned)heads * C, b.n_slot), dim3(kEvictThreads), 8 * (size_t)slice, s,
                            b, slice);
    count_launches(1);
    return e;
}

template <int C, int kThreads>
static cudaError_t launch_few(const EvictBatch& b, int heads, cudaStream_t s)
{
    const cudaError_t e = launch_pdl(kv_evict_few_kernel<C, kThreads>, dim3((unsigned)heads * C, b.n_slot), dim3(kThreads), s, b);
    count_launches(1);
    return e;
}

cudaError_t launch_kv_evict(const EvictBatch& b, int n_layers, int Hkv, cudaStream_t s)
{
    int max_len = 0;
    for (int i = 0; i < b.n_slot; ++i) max_len = std::max(max_len, b.slot[i].len);
    const int heads = n_layers * Hkv;
    int most = 0;
    for (int i = 0; i < b.n_slot; ++i) most = std::max(most, b.slot[i].len - b.slot[i].budget);
    if (most <= kFewKeys) {
        if (max_len <= kFewMax) return launch_few<1, kFewThreads>(b, heads, s);
        // CTAs of more than 1,024 keys, two a multiprocessor at most (64 heads of
        // 16,384 keys: 8.2 us with 4 CTAs a head, 13.2 with 8)
        int c = 1;
        while (c < 8 && max_len / c > 2048 && (int64_t)heads * b.n_slot * c <= 152) c *= 2;
        switch (c) {
            case 1: return launch_few<1, kFewLongThreads>(b, heads, s);
            case 2: return launch_few<2, kFewLongThreads>(b, heads, s);
            case 4: return launch_few<4, kFewLongThreads>(b, heads, s);
            default: return launch_few<8, kFewLongThreads>(b, heads, s);
        }
    }
    int c = 1;
    while (c < 8 && ((max_len + c - 1) / c > kEvictSlice || (max_len / c > 4096 && (int64_t)heads * b.n_slot * c <= 152)))
        c *= 2;
    switch (c) {
        case 1: return launch_evict<1>(b, heads, max_len, s);
        case 2: return launch_evict<2>(b, heads, max_len, s);
        case 4: return launch_evict<4>(b, heads, max_len, s);
        default: return launch_evict<8>(b, heads, max_len, s);
    }
}

}  // namespace luce
