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
//
// The products.  Codes are whole numbers below 2^8 and so f16 without an error; q and
// the weights are each two f16 parts, 22 bits, whose products with a code are exact in
// the tensor cores' f32 sums.  The scales stay out of them: K's multiplies the scores,
// V's the weights of its 32 keys.  A tree has few rows (8 nodes of 8 heads are 64), so
// the keys of a tile (for the sums, the dims) are the 128 rows of a product and the
// tree's rows its columns, 16 to 128 of them: no lane works for a row that is not there.
// A then is what is turned from 8 bits, and lies in tensor memory: from shared memory a
// product of 16 columns takes 39 cycles, from there 9, and shared memory would have to
// hold the turned tile as well.
//
// What bounds it.  A tile is 33 KB and 1,430 cycles of an SM's share of the copy rate.
// Its codes are turned at 4 bytes for 6 instructions: of the 4,500 warp instructions a
// tile with up to 16 rows costs, 1,900 turn, 400 form weights, 200 issue products; issue
// slots are taken to 59 %, and most of the rest is instruction fetch, as warps of six kinds
// run code of their own, and latency within the weights' warps, of which a scheduler has one
// or two.  With many rows the weights take over (two 16-bit parts, one exponential and a
// dozen other instructions each).  Short contexts are bound by the latency of one tile's
// chain (load, turn, product, weights, product, sums) and of the merge.
//
// Measured (L2 flushed; with the merge): 4 one-token slots of 8 KV heads x 2,048 keys 12.6 us;
// 4 slots of 4 nodes 15.0; 4 paged one-token slots of 16k to 33k keys (197 MB) 53.0, 3.7
// TB/s; one slot of 16 nodes x 130,784 keys (269 MB, 43 GFLOP) 120, 2.2 TB/s and 0.36
// PFLOP/s in one f16 part (twice that with both; 102 us over an f16 cache); 4 slots of 4
// nodes, a window of 4,096 keys, 22.3.
#include <limits.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"
#include "q8kv.h"
#include "ring.cuh"
#include "tensor.cuh"

namespace luce {

constexpr int kQ8MaxChunks = 160;
constexpr int kQ8Ctas = 304;  // the CTAs that a cut aims at

// A chunk's weights, and so its sums, are 2^15 e^(s - m): the tree attention's
// reason, f16 has no digits below 2^-24.
constexpr float kQ8Up = 15.0f, kQ8Down = 1.0f / 32768.0f;

// The smallest scale of V that weights are formed with, 2^-50 (sealing gives 0 or 2^-24 / 127
// and more): a block of zeros weighs as one of this scale, and next to one of scale 2^35, the
// largest, a key's weight of 2^-41 of the largest, below which 2^17 keys leave the
// sum's digits as they are, is 2^(15 - 50 - 35 - 41) = 2^-111 in a chunk, and its chunk's factor in
// the merge 2^(-50 - 35 - 41) = 2^-126, the smallest normal number.
// (The weights of smaller scales times what is missing, where there are any: 12.6 -> 13.0
// us on 4x1 serving and 52.8 -> 53.6 on long paged, although these never run that code.)
constexpr float kQ8LeastV = 8.881784197001252e-16f;

// Scores in powers of two: e^(s - m) = 2^(log2 dot - max).  The scale's sign goes
// into q.
struct Q8Scale {
    float sign, log2;
};

// Query heads of a KV head, KV heads.
struct Q8Heads {
    int group, kv, inverse;  // inverse: 2^16 / group, rounded up
    __device__ __forceinline__ int node(int c) const { return c * inverse >> 16; }  // c / group, for c < 2^10 and groups up to 8
};

// Tiles of a chunk for a view of nt tiles, an even number: a step of the kernel takes
// two.  Of the cuts that fill kQ8Ctas CTAs 1, 2, 3 or 4 times the cheapest is taken,
// a chunk costing its steps and about one more (its q, its results).  A function of the
// tiles and the KV heads alone, so that a row's sums are cut the same way whatever else
// is in the call: with many rows, where half as many CTAs run, it is cut alike.
static int q8_chunk_tiles(int nt, int Hkv)
{
    const int all = (nt + 1) / 2;
    int best = all, least = INT_MAX;
    for (int rounds = 1; rounds <= 4; ++rounds) {
        const int n = std::min({kQ8Ctas * rounds / Hkv, all, kQ8MaxChunks});
        if (n < 1) continue;
        const int steps = (all + n - 1) / n;
        const int cost = (Hkv * n + kQ8Ctas - 1) / kQ8Ctas * (steps + 1);
        if (cost < least) {
            least = cost;
            best = steps;
        }
    }
    return 2 * std::max(best, 1);
}

int q8kv_max_chunks(int max_sealed, int Hkv)
{
    const int tiles = (max_sealed + kQ8Page - 1) / kQ8Page;
    return std::min({(tiles + 1) / 2, kQ8MaxChunks, std::max(1, 4 * kQ8Ctas / Hkv)});
}

// A chunk's row of results: part_o [row][128] and part_ml [row][8] = (m, three unused,
// l of the tiles' first to fourth block), the sums times 2^15.
size_t q8kv_part_bytes(int64_t n_part) { return (size_t)n_part * (kHeadDim + 8) * sizeof(float); }

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
        v.chunk = v.n_tile ? q8_chunk_tiles(v.n_tile, Hkv) : 2;
        v.n_chunk = (v.n_tile + v.chunk - 1) / v.chunk;
        v.part0 = part;
        part += (int64_t)v.n_chunk * v.n_nodes * Hq;
        b.order[i] = (uint8_t)i;
    }
    std::stable_sort(b.order, b.order + b.n_view, [&](int x, int y) { return b.view[x].chunk > b.view[y].chunk; });
    return part;
}

// The key that tile t of a view's starts with.
__device__ __forceinline__ int q8_tile_key(const Q8View& v, int t) { return (t < v.front ? t : t - v.front + v.back) * kQ8Page; }

// ---------------------------------------------------------------- chunks

constexpr int kQ8ScaleSlots = 16;  // tiles whose scales are held: more than lie between the producer and the weights

__device__ unsigned int g_q8kv_wait_timeouts;

// Sizes of a kernel for up to 16 NG rows of a KV head.  4 PARTS warps form scores into
// weights and add up sums, each with 32 keys and a PARTS-th of the rows; four turn K's
// codes into f16 and four V's, and of the last four one feeds the tiles, two issue the
// products and one prepares the next head's q.
template <int NG, int PARTS>
struct Q8Shape {
    static constexpr int kRows = 16 * NG;                      // columns of the products
    static constexpr int kParts = PARTS;
    static constexpr int kGroups = 2 * NG / PARTS;             // of eight columns, of a part
    static constexpr int kCols = 8 * kGroups;
    static constexpr int kWarps = 4 * PARTS;
    static constexpr int kThreads = 32 * (kWarps + 12);
    static constexpr int kCtas = PARTS == 1 ? 2 : 1;           // of a multiprocessor
    // registers of a thread on weights; a turning one has 32, one of the last four warps
    // 48: together 32,768 of a CTA of 512 launched with 64 each, 61,440 of 640 with 96
    static constexpr int kRegs = PARTS == 1 ? 144 : 184;
    // tiles in flight: what shared memory holds beside q and the weights
    static constexpr int kSlotsK = NG == 3 ? 4 : NG == 4 || NG == 5 || NG == 8 ? 3 : 2;
    static constexpr int kSlotsV = NG == 3 ? 3 : NG == 2 ? 1 : 2;
    static constexpr int kSlots = kSlotsK + kSlotsV;
    // In tensor memory: one tile of K, which is multiplied as soon as it is there, the
    // scores of a step's two, and its V, which waits for their weights: two tiles where
    // they fit (one takes 14.1 us for 13.6 with 5 rows of 32 tiles, 98 for 96 with 60 of
    // 1,015), but where rows are so many that turning ahead only keeps the weights' warps from
    // their issue slots (124 us for 119 with 80 of 1,022 tiles, 112 for 107 with 96 of 782)
    static constexpr int kTurnedV = NG == 2 || NG >= 5 ? 1 : 2;
    static constexpr int kWeights = NG == 8 ? 1 : 2;           // tiles of weights in shared memory
    // heads of q in shared memory: with two the next one's is prepared ahead by a warp of its
    // own (56.7 us for 53.4 without, at 4 rows of 4 slots), else the weights' many warps prepare
    // it when its turn comes (27 us for 24 by the one warp at 64 rows, 155 for 124 at 80)
    static constexpr int kHeads = NG == 1 ? 2 : 1;
    // scores are read twice, not held while maxima are found, where registers do not hold both
    // tiles' (held: 16.3 us for 16.0 with 20 rows, 150 for 119 with 80; read twice by 16: 54.4 for 53.4)
    static constexpr bool kTwice = NG == 2 || NG >= 5;
    static constexpr int kPart = kRows * kHeadDim * 2;         // bytes of one part of q, or of the weights
    static constexpr uint32_t kColK = 0, kColV = 64, kColS = kColV + 64 * kTurnedV, kColO = kColS + 2 * kRows;
    static constexpr uint32_t kTmem = 512 / kCtas;
    static constexpr int kBytes = kSlots * kQ8PageBytes + 2 * (kHeads + kWeights) * kPart + 1024;
    static_assert(kColO + kRows <= kTmem && 2 * NG % PARTS == 0, "tensor memory");
};

struct Q8Maps {
    CUtensorMap k[4], v[4];
};

template <typename S>
struct Q8Bars {
    uint64_t k_full[S::kSlotsK], k_empty[S::kSlotsK];    // a tile of K is there; has been turned
    uint64_t v_full[S::kSlotsV], v_empty[S::kSlotsV];
    uint64_t ka_full, ka_free;                           // K of a tile is f16 in tensor memory; has been multiplied
    uint64_t va_full[S::kTurnedV], va_free[S::kTurnedV];
    uint64_t s_full, s_free[2];                          // S of a step is complete; its tiles' have been read
    uint64_t p_full[S::kWeights], p_free;                // a tile's weights are in place; have been multiplied (where there is one place)
    uint64_t o_full, o_free;                             // O of a step is complete; has been read
    uint64_t q_full[S::kHeads], q_free[S::kHeads];       // a head's q is in place; has been multiplied, its units read
    uint64_t done[2];                                    // every S, every O that was issued is complete
};

// Chunks of one (view, KV head) that a CTA takes one after the other: `chunks` of
// them from number c on, tiles t0 .. t0 + tiles - 1; views in b.order, head, chunk.
struct Q8Run {
    int view, g, c, chunks, tiles, t0;
};

__device__ __forceinline__ Q8Run q8_run(const Q8Batch& b, int Hkv, int u, int end)
{
    Q8Run t;
    const int u0 = u;
    int at = 0;
    while (at + 1 < b.n_view && u >= Hkv * b.view[b.order[at]].n_chunk) u -= Hkv * b.view[b.order[at++]].n_chunk;
    t.view = b.order[at];
    const Q8View& v = b.view[t.view];
    t.g = u / v.n_chunk;
    t.c = u - t.g * v.n_chunk;
    t.chunks = min(v.n_chunk - t.c, end - u0);
    t.t0 = t.c * v.chunk;
    t.tiles = min(t.chunks * v.chunk, v.n_tile - t.t0);
    return t;
}

// The CTA's runs.  Chunks of one step: neighbours u0 .. u1 - 1 (heads change least).
// Longer ones: of every `step` of them one, from the longest on, back and forth, so
// that the CTAs' shares are alike (4 windows of unlike slots 27 us, as neighbours 36).
struct Q8Share {
    int u0, u1, step;
};

template <typename F>
__device__ __forceinline__ void q8_each_run(const Q8Batch& b, int Hkv, const Q8Share& w, F f)
{
    int u = w.u0;
    for (int round = 1; u < w.u1; ++round) {
        const Q8Run t = q8_run(b, Hkv, u, w.step ? u + 1 : w.u1);
        u = !w.step ? u + t.chunks : round & 1 ? (round + 1) * w.step - 1 - w.u0 : round * w.step + w.u0;
        if (!f(t)) return;
    }
}

// 16 lanes by 8 columns of tensor memory: v[0], v[1] are lane t / 4's columns 2 (t % 4)
// and the next, v[2], v[3] lane t / 4 + 8's.  Not there before tm_loaded.
__device__ __forceinline__ void tm_ld_frag(uint32_t addr, float* v)
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(addr));
}
template <int N>
__device__ __forceinline__ void tm_loaded(float* v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));  // (no use of them moves ahead of the wait)
}

// Four 8 x 8 matrices of f16 pairs, stored turned: a lane's address is a row of what is
// stored, a column of what the registers hold.
__device__ __forceinline__ void st_matrix_turned(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// Four codes as f16 pairs, exactly: 1152 + code by its bits, less 1152.
__device__ __forceinline__ void q8_half_codes(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    w ^= 0x80808080u;
    const uint32_t a = __byte_perm(w, 0x64646464u, 0x4140), b = __byte_perm(w, 0x64646464u, 0x4342);
    asm("{ .reg .b32 n; mov.b32 n, 0x64806480; sub.rn.f16x2 %0, %1, n; }" : "=r"(lo) : "r"(a));
    asm("{ .reg .b32 n; mov.b32 n, 0x64806480; sub.rn.f16x2 %0, %1, n; }" : "=r"(hi) : "r"(b));
}

// A step's tiles: two, or one at a run's end.
__device__ __forceinline__ int q8_step_tiles(const Q8Run& t, int k) { return min(2, t.tiles - k); }

// A place in the CTA's tiles; the tile's page is on its way when its turn comes.
struct Q8Cursor {
    int u, round, tile, tiles, view, g, page;

    __device__ __forceinline__ void enter(const Q8Batch& b, int Hkv, const Q8Share& w)
    {
        const Q8Run t = q8_run(b, Hkv, u, w.step ? u + 1 : w.u1);
        u = !w.step ? u + t.chunks : round & 1 ? (round + 1) * w.step - 1 - w.u0 : round * w.step + w.u0;
        ++round;
        tile = t.t0;
        tiles = t.tiles;
        view = t.view;
        g = t.g;
    }
    __device__ __forceinline__ void fetch(const Q8Batch& b)
    {
        const Q8View& v = b.view[view];
        const int span = q8_tile_key(v, tile) / kQ8Page;
        page = v.table ? ld_placed_i(v.table + span) : span;
    }
    __device__ __forceinline__ bool start(const Q8Batch& b, int Hkv, const Q8Share& w)
    {
        u = w.u0;
        round = 1;
        tiles = 0;
        if (u >= w.u1) return false;
        enter(b, Hkv, w);
        fetch(b);
        return true;
    }
    __device__ __forceinline__ bool next(const Q8Batch& b, int Hkv, const Q8Share& w)
    {
        if (--tiles > 0) {
            ++tile;
        } else {
            if (u >= w.u1) return false;
            enter(b, Hkv, w);
        }
        fetch(b);
        return true;
    }
};

__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity)
{
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done)
                 : "r"(smem_addr(b)), "r"(parity)
                 : "memory");
    return done != 0;
}

// The producer: tiles of K (with their scales) and of V, each into the next place of
// its own ring that is free.  Gives up where no place becomes free for kWaitLimitNs.
template <typename S>
__device__ void q8_produce(const Q8Maps& maps, const Q8Batch& b, int Hkv, const Q8Share& w, uint8_t* tiles, float (*scales)[8],
                           Q8Bars<S>& bar)
{
    unsigned int* late = &g_q8kv_wait_timeouts;
    int nk = 0, nv = 0;
    pdl_wait();
    pdl_trigger();
    Q8Cursor k, v;
    bool more_k = k.start(b, Hkv, w), more_v = v.start(b, Hkv, w);
    uint64_t since = global_ns();
    while (more_k || more_v) {
        bool moved = false;
        if (more_k && mbar_test(&bar.k_empty[nk % S::kSlotsK], ((nk / S::kSlotsK) & 1) ^ 1)) {
            const Q8View& o = b.view[k.view];
            uint64_t* full = &bar.k_full[nk % S::kSlotsK];
            float* to = scales[nk % kQ8ScaleSlots];
            const bool in = k.page >= 0 && k.page < o.n_pages;  // (else outside the map: zeros)
            // the scales come with the tile; the weights' warps read them behind S, which
            // the turning warps' wait for this tile has come before
            if (!in)
                for (int e = 0; e < 8; ++e) to[e] = 0.0f;
            mbar_expect_tx(full, kQ8PageBytes + (in ? 32 : 0));
            if (in)
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 32, [%2];" ::"r"(smem_addr(to)),
                             "l"(o.scales + k.page * o.scale_stride + k.g * kQ8PageScales), "r"(smem_addr(full))
                             : "memory");
            tma_load_4d(tiles + nk % S::kSlotsK * kQ8PageBytes, &maps.k[k.view], 0, 0, k.g, in ? k.page : o.n_pages, full);
            ++nk;
            more_k = k.next(b, Hkv, w);
            moved = true;
        }
        if (more_v && mbar_test(&bar.v_empty[nv % S::kSlotsV], ((nv / S::kSlotsV) & 1) ^ 1)) {
            const Q8View& o = b.view[v.view];
            uint64_t* full = &bar.v_full[nv % S::kSlotsV];
            mbar_expect_tx(full, kQ8PageBytes);
            tma_load_4d(tiles + (S::kSlotsK + nv % S::kSlotsV) * kQ8PageBytes, &maps.v[v.view], 0, 0, v.g,
                        v.page >= 0 && v.page < o.n_pages ? v.page : o.n_pages, full);
            ++nv;
            more_v = v.next(b, Hkv, w);
            moved = true;
        }
        if (moved) {
            since = global_ns();
        } else if (global_ns() - since > kWaitLimitNs) {
            atomicAdd(late, 1u);
            break;
        } else {
            __nanosleep(32);
        }
    }
    ring_drain<S::kSlotsK>(bar.k_full, nk, late);
    ring_drain<S::kSlotsV>(bar.v_full, nv, late);
}

__device__ __forceinline__ uint4 lds128_at(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// One operand's codes, [lane's row][128], into tensor memory as f16, from the row's
// first piece of 16 in the tile's swizzle.  (A loop of 32 codes a round: unrolled to 64
// or 128 its code is fetched more slowly than it runs, 57 and 58 us for 55 where 4 slots
// are longest.)
__device__ __forceinline__ void q8_turn(uint32_t from, uint32_t to)
{
#pragma unroll 1
    for (int e = 0; e < 8; e += 2) {
        const uint4 x = lds128_at(from ^ (e << 4)), y = lds128_at(from ^ ((e + 1) << 4));
        uint32_t o[16];
        q8_half_codes(x.x, o[0], o[1]);
        q8_half_codes(x.y, o[2], o[3]);
        q8_half_codes(x.z, o[4], o[5]);
        q8_half_codes(x.w, o[6], o[7]);
        q8_half_codes(y.x, o[8], o[9]);
        q8_half_codes(y.y, o[10], o[11]);
        q8_half_codes(y.z, o[12], o[13]);
        q8_half_codes(y.w, o[14], o[15]);
        tm_st16(to + 8 * e, o);
    }
    tm_wait_st();
}

// The turning warps of K, or of V: a row of 128 codes per thread.
template <int SLOTS, int TURNED>
__device__ void q8_turn_tiles(int n, const uint8_t* tiles, uint32_t to, int row, uint64_t* full, uint64_t* empty, uint64_t* free, uint64_t* done)
{
    unsigned int* late = &g_q8kv_wait_timeouts;
    const uint32_t from = smem_addr(tiles) + row * 128 + ((row & 7) << 4);
    int st = 0, x = 0;
    uint32_t filled = 0, freed = 1;  // the parities of the places' next uses
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
        const bool there = mbar_wait(&full[st], filled, late) && mbar_wait(&free[x], freed, late);
        if (!__all_sync(0xffffffffu, there)) return;
        tm_after();
        q8_turn(from + st * kQ8PageBytes, to + 64 * x);
        warp_arrive(&done[x]);
        if ((row & 31) == 0) mbar_arrive(&empty[st]);
        if (++st == SLOTS) {
            st = 0;
            filled ^= 1;
        }
        if (++x == TURNED) {
            x = 0;
            freed ^= 1;
        }
    }
}

// A product's steps, 128 x kRows x 16 each: A in tensor memory from column a, B rows of
// 256 bytes in two halves.  The low parts go first: an accumulation loses digits by
// the sum's size, and theirs is small.
template <typename S>
__device__ __forceinline__ void q8_multiply(uint32_t d, uint32_t a, uint32_t bytes, bool adds, uint32_t elected)
{
    constexpr uint32_t idesc = (1u << 4) | ((uint32_t)(S::kRows / 8) << 17) | (8u << 24);  // D f32, A and B f16
    // (told to be the warp's, as they are: else every product moves its own copies)
    d = __shfl_sync(0xffffffffu, d, 0);
    a = __shfl_sync(0xffffffffu, a, 0);
    const uint64_t desc = tree_desc(__shfl_sync(0xffffffffu, bytes, 0), 16, 1024);
#pragma unroll
    for (int ks = 0; ks < 16; ++ks)
        tree_mma(d, a + 8 * (ks & 7), desc + ((ks < 8 ? S::kPart : 0) + (ks >> 2 & 1) * (S::kPart / 2)) / 16 + 2 * (ks & 3), idesc,
                 adds || ks > 0, elected);
}

// The products are issued by a warp each: S of a tile as soon as its K is there, and
// its O behind its weights.  A step of 16 columns takes the tensor cores 9 cycles
// and its issue about as many slots of a scheduler that five other warps use: by one
// warp, the 32 steps of a tile took 2,100 cycles.
template <typename S>
__device__ void q8_scores(const Q8Batch& b, int Hkv, const Q8Share& w, uint32_t q, uint32_t tmem, Q8Bars<S>& bar)
{
    unsigned int* late = &g_q8kv_wait_timeouts;
    const uint32_t elected = elect_one();
    int n = 0, head = -1, last = -1, used[2] = {0, 0};  // tiles, heads, of the places of scores
    q8_each_run(b, Hkv, w, [&](const Q8Run& t) {
        bool ok = true;
        if (t.view * Hkv + t.g != last) {
            if (last >= 0) tree_commit_mma(&bar.q_free[head % S::kHeads], elected);
            last = t.view * Hkv + t.g;
            ++head;
            ok = __all_sync(0xffffffffu, mbar_wait(&bar.q_full[head % S::kHeads], (head / S::kHeads) & 1, late));
        }
        for (int k = 0; ok && k < t.tiles; ++k, ++n) {
            // (of a tile's two places of scores each has its own uses: a run's last step may have one tile)
            const bool there = mbar_wait(&bar.ka_full, n & 1, late) && mbar_wait(&bar.s_free[k & 1], ((k & 1 ? used[1] : used[0]) & 1) ^ 1, late);
            if (!(ok = __all_sync(0xffffffffu, there))) break;  // (the warp leaves as one)
            (k & 1 ? used[1] : used[0]) += 1;
            tm_after();
            q8_multiply<S>(tmem + S::kColS + S::kRows * (k & 1), tmem + S::kColK, q + head % S::kHeads * 2 * S::kPart, false, elected);
            tree_commit_mma(&bar.ka_free, elected);
            if ((k & 1) || k + 1 == t.tiles) tree_commit_mma(&bar.s_full, elected);
        }
        return ok;
    });
    // also after an expired wait, tensor memory is not freed under a product
    tree_commit_mma(&bar.done[0], elected);
    mbar_wait(&bar.done[0], 0, late);
}

template <typename S>
__device__ void q8_sums(const Q8Batch& b, int Hkv, const Q8Share& w, uint32_t weights, uint32_t tmem, Q8Bars<S>& bar)
{
    unsigned int* late = &g_q8kv_wait_timeouts;
    const uint32_t elected = elect_one();
    int i = 0, n = 0, used[2] = {0, 0};  // steps, tiles, of the places of weights
    q8_each_run(b, Hkv, w, [&](const Q8Run& t) {
        for (int k = 0; k < t.tiles; ++k, ++n) {
            const int to = n % S::kTurnedV, p = (k & 1) % S::kWeights;
            const bool there = mbar_wait(&bar.va_full[to], (n / S::kTurnedV) & 1, late) &&
                               mbar_wait(&bar.p_full[p], (p ? used[1] : used[0]) & 1, late) &&
                               ((k & 1) || i == 0 || mbar_wait(&bar.o_free, (i - 1) & 1, late));
            if (!__all_sync(0xffffffffu, there)) return false;
            (p ? used[1] : used[0]) += 1;
            tm_after();
            q8_multiply<S>(tmem + S::kColO, tmem + S::kColV + 64 * to, weights + p * 2 * S::kPart, k & 1, elected);
            tree_commit_mma(&bar.va_free[to], elected);
            if (S::kWeights == 1) tree_commit_mma(&bar.p_free, elected);
            if ((k & 1) || k + 1 == t.tiles) {
                tree_commit_mma(&bar.o_full, elected);
                ++i;
            }
        }
        return true;
    });
    tree_commit_mma(&bar.done[1], elected);
    mbar_wait(&bar.done[1], 0, late);
}

// A head's rows of q, in units of a power of two each, as two f16 parts in the products'
// layout: 16 lanes a row, rows first, first + step, ..  A loop with the next row on its
// way: a kernel's first instructions are fetched more slowly than they run.
template <typename S>
__device__ __forceinline__ void q8_prepare(const float* q, const Q8Batch& b, const Q8Heads& heads, const Q8Run& t, const Q8Scale& scale,
                                           uint8_t* parts, float (*unit_s)[S::kCols], int (*from_s)[S::kCols], int first, int step)
{
    const Q8View& v = b.view[t.view];
    const int R = v.n_nodes * heads.group, piece = threadIdx.x & 15;
    const float* head_q = q + ((int64_t)v.row0 * heads.kv + t.g) * heads.group * kHeadDim + 8 * piece;
    const int from = v.sealed + v.tail - v.window;
    float4 x, y;
    int path;
    auto load = [&](int c) {
        x = y = make_float4(0, 0, 0, 0);
        path = 0;
        if (c < R) {
            const int node = heads.node(c);
            const float* p = head_q + ((int64_t)node * heads.kv * heads.group + c - node * heads.group) * kHeadDim;
            x = ld_placed_f4(p);
            y = ld_placed_f4(p + 4);
            path = b.row[v.row0 + node].n_path;
        }
    };
    load(first);
#pragma unroll 1
    for (int c = first; c < S::kRows; c += step) {  // (kRows and step are even: a warp's halves go round as often)
        const float4 x0 = x, y0 = y;
        const int from0 = from + path;
        load(c + step);
        float big = fmaxf(fmaxf(fmaxf(fabsf(x0.x), fabsf(x0.y)), fmaxf(fabsf(x0.z), fabsf(x0.w))),
                          fmaxf(fmaxf(fabsf(y0.x), fabsf(y0.y)), fmaxf(fabsf(y0.z), fabsf(y0.w))));
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, d));
        // the row's unit puts its largest element into [2^14, 2^15), the smallest normal
        // numbers and what is below them, whose own digits end at 2^-149, into 2^0 and less
        const int exp = max((__float_as_int(big) >> 23) - 127 - 14, -126);
        const float into = __fmul_rn(scale.sign, __int_as_float((127 - exp) << 23));
        uint4 hi, lo;
        tree_split(__fmul_rn(x0.x, into), __fmul_rn(x0.y, into), hi.x, lo.x);
        tree_split(__fmul_rn(x0.z, into), __fmul_rn(x0.w, into), hi.y, lo.y);
        tree_split(__fmul_rn(y0.x, into), __fmul_rn(y0.y, into), hi.z, lo.z);
        tree_split(__fmul_rn(y0.z, into), __fmul_rn(y0.w, into), hi.w, lo.w);
        uint8_t* at = parts + (piece >> 3) * (S::kPart / 2) + (c >> 3) * 1024 + (c & 7) * 128 + (((piece & 7) ^ (c & 7)) << 4);
        *reinterpret_cast<uint4*>(at) = hi;
        *reinterpret_cast<uint4*>(at + S::kPart) = lo;
        if (piece == 0) {
            const int part = (c >> 3) % S::kParts, col = (c >> 3) / S::kParts * 8 + (c & 7);
            unit_s[part][col] = __fmul_rn(scale.log2, __int_as_float((127 + exp) << 23));
            from_s[part][col] = from0;
        }
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Maxima over the eight lanes that share lane % 4: each value's ends in one lane of
// them or in several; value k of what is left is value k + `first` of all.
template <int N, int OFF>
__device__ __forceinline__ void q8_maxima(float* v, int lane, int& first)
{
    if constexpr (OFF >= 4) {
        if constexpr (N % 2 == 0) {
            constexpr int H = N / 2;
            const bool upper = lane & OFF;
#pragma unroll
            for (int e = 0; e < H; ++e) {
                const float give = upper ? v[e] : v[e + H], keep = upper ? v[e + H] : v[e];
                v[e] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, OFF));
            }
            if (upper) first += H;
            q8_maxima<H, OFF / 2>(v, lane, first);
        } else {
#pragma unroll
            for (int e = 0; e < N; ++e) v[e] = fmaxf(v[e], __shfl_xor_sync(0xffffffffu, v[e], OFF));
            q8_maxima<N, OFF / 2>(v, lane, first);
        }
    }
}
constexpr int q8_left(int n, int off = 16) { return off < 4 ? n : q8_left(n % 2 == 0 ? n / 2 : n, off / 2); }

// kCtas CTAs an SM, each with its share of all chunks.
template <int NG, int PARTS>
__global__ void __launch_bounds__(Q8Shape<NG, PARTS>::kThreads, Q8Shape<NG, PARTS>::kCtas)
q8kv_chunk_kernel(const __grid_constant__ Q8Maps maps, const float* q, const __grid_constant__ Q8Batch b, Q8Heads heads, int units,
                  bool runs, Q8Scale scale, float* __restrict__ part_o, float* __restrict__ part_ml)
{
    using S = Q8Shape<NG, PARTS>;
    const int Hkv = heads.kv;
    extern __shared__ uint8_t q8_smem[];
    uint8_t* tiles = q8_smem + ((1024u - (smem_addr(q8_smem) & 1023u)) & 1023u);
    uint8_t* qs = tiles + S::kSlots * kQ8PageBytes;       // q: high and low part, two halves of the dims each
    uint8_t* ps = qs + 2 * S::kHeads * S::kPart;          // weights, the same way
    __shared__ Q8Bars<S> bar;
    __shared__ uint32_t tmem_at;
    __shared__ __align__(16) float scales[kQ8ScaleSlots][8];
    // by part, and by the step's parity: its columns are the groups of eight PARTS e + part, numbered through
    __shared__ float mx[2][PARTS][4][S::kCols];           // the columns' maxima of a warp's keys, by step parity
    __shared__ float unit_s[S::kHeads][PARTS][S::kCols];             // a score's power of two per unit of its product
    __shared__ __align__(8) int from_s[S::kHeads][PARTS][S::kCols];  // the first key in the row's window
    // by warp: what turns a column's products into exponents (a factor, an offset),
    // for each of a step's tiles, and what O so far is multiplied by, by step parity
    __shared__ __align__(8) float factor_s[S::kWarps][2][S::kCols], offset_s[S::kWarps][2][S::kCols];
    __shared__ __align__(8) float alpha_s[2][S::kWarps][S::kCols];
    __shared__ volatile int bail[PARTS][2];               // a wait of the part's warps expired, by step parity
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == S::kWarps + 10) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_at)), "r"(S::kTmem));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int i = 0; i < S::kSlotsK; ++i) {
            mbar_init(&bar.k_full[i], 1);
            mbar_init(&bar.k_empty[i], 4);
        }
        for (int i = 0; i < S::kSlotsV; ++i) {
            mbar_init(&bar.v_full[i], 1);
            mbar_init(&bar.v_empty[i], 4);
        }
        mbar_init(&bar.ka_full, 4);
        mbar_init(&bar.ka_free, 1);
        for (int i = 0; i < S::kTurnedV; ++i) {
            mbar_init(&bar.va_full[i], 4);
            mbar_init(&bar.va_free[i], 1);
        }
        mbar_init(&bar.s_full, 1);
        mbar_init(&bar.s_free[0], S::kWarps);
        mbar_init(&bar.s_free[1], S::kWarps);
        mbar_init(&bar.p_free, 1);
        for (int i = 0; i < PARTS; ++i) bail[i][0] = bail[i][1] = 0;
        for (int i = 0; i < S::kWeights; ++i) mbar_init(&bar.p_full[i], S::kWarps);
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_free, S::kWarps);
        for (int i = 0; i < S::kHeads; ++i) {
            mbar_init(&bar.q_full[i], S::kHeads == 1 ? S::kWarps : 1);
            mbar_init(&bar.q_free[i], 1 + S::kWarps);
        }
        mbar_init(&bar.done[0], 1);
        mbar_init(&bar.done[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tmem = tmem_at;
    if (tid < 2 * b.n_view) {
        const int view = tid % b.n_view;
        const CUtensorMap* m = tid < b.n_view ? &maps.k[view] : &maps.v[view];
        if (b.view[view].n_chunk > 0)  // (a view without blocks has no map)
            asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    Q8Share w = {(int)blockIdx.x, units, (int)gridDim.x};
    if (runs)
        w = Q8Share{(int)((int64_t)units * blockIdx.x / gridDim.x), (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x), 0};
    unsigned int* late = &g_q8kv_wait_timeouts;

    if (warp >= S::kWarps + 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == S::kWarps + 8 && lane == 0) q8_produce(maps, b, Hkv, w, tiles, scales, bar);
        if (warp > S::kWarps + 8) {
            if (S::kHeads > 1) {
                // the first head's q by all three of these warps, which have nothing else to
                // do before
                pdl_wait();
                q8_prepare<S>(q, b, heads, q8_run(b, Hkv, w.u0, w.u0 + 1), scale, qs, unit_s[0], from_s[0],
                                 (tid - 32 * (S::kWarps + 9)) >> 4, 6);
                asm volatile("bar.sync 15, 96;" ::: "memory");
            }
            if (warp == S::kWarps + 9) q8_scores(b, Hkv, w, smem_addr(qs), tmem, bar);
            if (warp == S::kWarps + 10) q8_sums(b, Hkv, w, smem_addr(ps), tmem, bar);
            if (S::kHeads > 1 && warp == S::kWarps + 11) {
                int head = -1, last = -1;
                q8_each_run(b, Hkv, w, [&](const Q8Run& t) {
                    if (t.view * Hkv + t.g == last) return true;
                    last = t.view * Hkv + t.g;
                    const int to = ++head % S::kHeads;
                    if (head > 0) {
                        if (!__all_sync(0xffffffffu, mbar_wait(&bar.q_free[to], ((head / S::kHeads) & 1) ^ 1, late))) return false;
                        q8_prepare<S>(q, b, heads, t, scale, qs + to * 2 * S::kPart, unit_s[to], from_s[to], lane >> 4, 2);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.q_full[to]);
                    return true;
                });
            }
        }
        __syncwarp();
    } else if (warp >= S::kWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
        int n = 0;
        q8_each_run(b, Hkv, w, [&](const Q8Run& t) {
            n += t.tiles;
            return true;
        });
        const int row = 32 * (warp & 3) + lane;
        const uint32_t lanes = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        if (warp < S::kWarps + 4)
            q8_turn_tiles<S::kSlotsK, 1>(n, tiles, lanes + S::kColK, row, bar.k_full, bar.k_empty, &bar.ka_free, &bar.ka_full);
        else
            q8_turn_tiles<S::kSlotsV, S::kTurnedV>(n, tiles + S::kSlotsK * kQ8PageBytes, lanes + S::kColV, row, bar.v_full, bar.v_empty,
                                                   bar.va_free, bar.va_full);
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegs));
        // The warp's keys are its block of the tile, 32 quad ..; its columns the groups of
        // eight PARTS e + part, e < G.  Of them a thread has keys lane / 4 + 8 i and columns 2 (lane
        // % 4) and the next: of O the same columns, dims 32 quad + lane / 4 + 8 i.  What is
        // the same for a column's keys (maximum, factor, correction) a lane forms per
        // column, and the threads pick it up from shared memory: formed by each
        // thread for its own columns it took twice the instructions of the weights.
        // (a lane's columns are those whose maxima it ends with)
        constexpr int G = S::kGroups, kCols = S::kCols, kMine = q8_left(2 * G);
        int col[kMine];
        const int part = warp >> 2, quad = warp & 3, pair2 = 2 * (lane & 3);
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16) + 8 * part;
        const uint32_t row_at = (quad >> 1) * (S::kPart / 2) + part * 1024 + (lane & 7) * 128 +
                                (((4 * (quad & 1) + (lane >> 3)) ^ (lane & 7)) << 4);  // where its keys' weights go
        uint64_t o[G][4], l[G];        // pairs of columns
        float m[kMine];                // of the lane's columns
        int i = 0, n = 0, head = -1, last = -1;  // steps, tiles, heads
        bool ok = true, gone = false;
        int freed = 0;                 // tiles whose weights have been given to be multiplied
        // the chunk whose last step's O is still to come: its rows of results (-1: it is not a
        // chunk's last step), how many they are, their weights' sums and maxima
        int64_t end_row = -1;
        int end_left = 0;
        uint64_t end_l[G];
        float end_m[kMine];
        {
            float none[2 * G] = {};
            int first = 0;
            q8_maxima<2 * G, 16>(none, lane, first);
#pragma unroll
            for (int e = 0; e < kMine; ++e) col[e] = 8 * ((first + e) >> 1) + pair2 + ((first + e) & 1);
        }
        auto part_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(1 + part) : "memory"); };
        // adds O of step j
        auto take = [&](int j) {
            ok = __all_sync(0xffffffffu, ok && mbar_wait(&bar.o_full, j & 1, late));
            tm_after();
            constexpr int B = G <= 3 ? G : 2;  // groups at a time
#pragma unroll
            for (int e0 = 0; e0 < G; e0 += B) {
                float x[B][8];
#pragma unroll
                for (int e = e0; e < e0 + B && e < G; ++e) {
                    tm_ld_frag(lanes + S::kColO + 8 * PARTS * e, x[e - e0]);
                    tm_ld_frag(lanes + (16u << 16) + S::kColO + 8 * PARTS * e, x[e - e0] + 4);
                }
                tm_loaded<8 * B>(&x[0][0]);
                if (e0 + B >= G) warp_arrive(&bar.o_free);
#pragma unroll
                for (int e = e0; e < e0 + B && e < G; ++e) {
                    const uint64_t a = *reinterpret_cast<const uint64_t*>(&alpha_s[j & 1][warp][8 * e + pair2]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[e][c] = fma2(o[e][c], a, pair(x[e - e0][2 * c], x[e - e0][2 * c + 1]));
                }
            }
            if (__builtin_expect(end_row < 0, 1)) return;
            float* ml = part_ml + 8 * (end_row + 8 * part);
            float* po = part_o + (end_row + 8 * part + pair2) * kHeadDim + 32 * quad + (lane >> 2);
            asm volatile("" : "+l"(ml), "+l"(po));  // (one address each, not one for every store)
            const int left = ok ? end_left - 8 * part : 0;
#pragma unroll
            for (int e = 0; e < G; ++e) {
                const float2 mine = unpair(end_l[e]);
                float x[2] = {mine.x, mine.y};
#pragma unroll
                for (int d = 0; d < 2; ++d) {
#pragma unroll
                    for (int f = 4; f < 32; f <<= 1) x[d] = __fadd_rn(x[d], __shfl_xor_sync(0xffffffffu, x[d], f));
                    const int c = 8 * PARTS * e + d;
                    if (c + pair2 < left) {
                        if ((lane >> 2) == 0) ml[8 * (c + pair2) + 4 + quad] = x[d];
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const float2 y = unpair(o[e][f]);
                            po[c * kHeadDim + 8 * f] = d ? y.y : y.x;
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) o[e][c] = 0;  // (what the next chunk's first correction, 0, meets is finite)
            }
#pragma unroll
            for (int e = 0; e < kMine; ++e) {
                const int c = 8 * PARTS * (col[e] >> 3) + (col[e] & 7);
                if (quad == 0 && col[e] < kCols && c < left) ml[8 * c] = end_m[e];
            }
        };
#pragma unroll
        for (int e = 0; e < G; ++e)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[e][c] = 0;
        q8_each_run(b, Hkv, w, [&](const Q8Run& t) {
            const Q8View& v = b.view[t.view];
            const int R = v.n_nodes * heads.group;
            if (t.view * Hkv + t.g != last) {
                __syncwarp();
                if (last >= 0 && lane == 0) mbar_arrive(&bar.q_free[head % S::kHeads]);  // (its units have been read)
                last = t.view * Hkv + t.g;
                ++head;
                if (head == 0) pdl_wait();  // (q is there, and the results' place is free)
                // With room for one head's q it is prepared by these warps, which have nothing
                // else to do by then: each part's rows by its own
                if (S::kHeads == 1) {
                    if (head > 0) ok = ok && mbar_wait(&bar.q_free[0], (head & 1) ^ 1, late);
                    q8_prepare<S>(q, b, heads, t, scale, qs, unit_s[0], from_s[0], tid >> 4, 8 * PARTS);
                    warp_arrive(&bar.q_full[0]);
                }
                ok = ok && mbar_wait(&bar.q_full[head % S::kHeads], (head / S::kHeads) & 1, late);
            }
            // (out of the views' table, once)
            const int sealed = v.sealed, front = v.front, skip = v.back - v.front, sinks = v.sinks, chunk = v.chunk, tile0 = t.t0;
            const int edge = v.window > 0 ? v.sealed + v.tail + v.n_nodes - v.window : INT_MIN;  // keys from here on are in every row's window
            const float* units = unit_s[head % S::kHeads][part];
            const int* froms = from_s[head % S::kHeads][part];
            int64_t pr = v.part0 + ((int64_t)t.c * Hkv + t.g) * R;  // the chunk's rows of results
            int kc = 0;                                              // the chunk's tiles so far
            auto key_of = [&](int k) { return (tile0 + k + (tile0 + k < front ? 0 : skip)) * kQ8Page; };
            // A step from tile k on.  `masked`: some row's window begins in it or behind it
            // (code of its own: the scores it overwrites cost the others moves).
            auto step = [&](auto with_mask, int k, int two) {
                constexpr bool masked = decltype(with_mask)::value;
                const int buf = i & 1;
                if (kc == 0) {
#pragma unroll
                    for (int e = 0; e < G; ++e) l[e] = 0;
#pragma unroll
                    for (int e = 0; e < kMine; ++e) m[e] = -INFINITY;
                }
                ok = ok && mbar_wait(&bar.s_full, i & 1, late);
                tm_after();
                // scores: both tiles', held from the maxima on where there are few, else read
                // twice, `B` groups at a time
                constexpr int B = G <= 5 ? G : G / 2;
                float s[S::kTwice ? 1 : 2][B][8], factor[2][kMine], lv[2], iv[2], best[kMine];
                auto load_s = [&](int x, int e0) {
                    float(*to)[8] = s[S::kTwice ? 0 : x];
                    [[maybe_unused]] const int key0 = key_of(k + x);
#pragma unroll
                    for (int e = 0; e < B; ++e) {
                        tm_ld_frag(lanes + S::kColS + S::kRows * x + 8 * PARTS * (e0 + e), to[e]);
                        tm_ld_frag(lanes + (16u << 16) + S::kColS + S::kRows * x + 8 * PARTS * (e0 + e), to[e] + 4);
                    }
                    tm_loaded<8 * B>(&to[0][0]);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < B; ++e) {
                            const int2 key1 = *reinterpret_cast<const int2*>(&froms[8 * (e0 + e) + pair2]);
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const int key = key0 + kQ8Block * quad + (lane >> 2) + 8 * (c >> 1);
                                if (key >= sinks && key < (c & 1 ? key1.y : key1.x)) to[e][c] = -INFINITY;
                            }
                        }
                    }
                };
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float* sc = scales[(n + x) % kQ8ScaleSlots];
                    const bool valid = x < two && key_of(k + x) + kQ8Block * quad < sealed;
                    const float ks = valid ? sc[quad] : 0.0f;
                    // V's scale goes into the weights as a power of two: 2^(s + log2 vs - m) is
                    // what multiplies a code, and over vs the weight itself.  (A block of zeros
                    // weighs as one of the smallest scale.  A block that no row sees may have
                    // any scale: NaN becomes the smallest, infinity the largest, whose logarithm is
                    // finite, so that its scores of -inf give weights of 0.)
                    const float vs = fminf(fmaxf(valid ? sc[4 + quad] : 0.0f, kQ8LeastV), 3.402823466e38f);
                    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lv[x]) : "f"(vs));
                    if (!valid) lv[x] = -INFINITY;  // (whatever its scores are)
                    iv[x] = __frcp_rn(vs);
                    float top[2 * G];
#pragma unroll
                    for (int e0 = 0; e0 < G; e0 += B) {
                        load_s(x, e0);
#pragma unroll
                        for (int e = 0; e < B; ++e) {
                            const float* y = s[S::kTwice ? 0 : x][e];
                            top[2 * (e0 + e)] = fmaxf(max3(y[0], y[2], y[4]), y[6]);
                            top[2 * (e0 + e) + 1] = fmaxf(max3(y[1], y[3], y[5]), y[7]);
                        }
                    }
                    int first = 0;
                    q8_maxima<2 * G, 16>(top, lane, first);
#pragma unroll
                    for (int e = 0; e < kMine; ++e) {
                        // (rounded up: no weight is above 2^15 by more than its exponent's own rounding)
                        factor[x][e] = fmaxf(__fmul_rn(units[col[e]], ks), 1e-37f);
                        const float y = __fadd_ru(__fmul_ru(top[e], factor[x][e]), lv[x]);
                        best[e] = x ? fmaxf(best[e], y) : y;
                    }
                }
                if (!S::kTwice) {
                    warp_arrive(&bar.s_free[0]);
                    if (two == 2 && lane == 0) mbar_arrive(&bar.s_free[1]);
                }
#pragma unroll
                for (int e = 0; e < kMine; ++e) mx[buf][part][quad][col[e]] = best[e];
                // all four warps of a part meet here, an expired wait or not, and leave together
                if (!ok) bail[part][buf] = 1;
                part_sync();
                if (bail[part][buf]) {
                    gone = true;
                    return;
                }
#pragma unroll
                for (int e = 0; e < kMine; ++e) {
                    const float* x = &mx[buf][part][0][col[e]];
                    const float now = fmaxf(m[e], max3(fmaxf(x[0], x[kCols]), x[2 * kCols], x[3 * kCols]));
                    const float at = now == -INFINITY ? 0.0f : now;
#pragma unroll
                    for (int d = 0; d < 2; ++d) {
                        factor_s[warp][d][col[e]] = factor[d][e];
                        offset_s[warp][d][col[e]] = __fadd_rn(__fsub_rn(kQ8Up, at), lv[d]);
                    }
                    alpha_s[buf][warp][col[e]] = tree_exp2(__fsub_rn(m[e], at));  // 0 for m = -inf
                    m[e] = now;
                }
                __syncwarp();
                if (i > 0) take(i - 1);  // (behind its products the weights' places are free)
#pragma unroll(NG == 2 ? 1 : 2)
                for (int x = 0; x < 2; ++x) {  // (as a loop less code is fetched: 15.7 us for 16.0 with 20 rows; with 80, 125 for 119)
                    if (x == 1 && two == 1) break;
                    const uint32_t to = smem_addr(ps) + (x % S::kWeights) * 2 * S::kPart + row_at;
                    const float inverse = x ? iv[1] : iv[0];
                    const uint64_t iv2 = pair(inverse, inverse);
                    if (x == 1 && S::kWeights == 1) ok = ok && mbar_wait(&bar.p_free, freed & 1, late);
#pragma unroll
                    for (int e = 0; e < G; ++e) {
                        if (S::kTwice && e % B == 0) {
                            load_s(x, e);
                            if (e + B >= G) warp_arrive(&bar.s_free[x]);
                        }
                        // (pairs as they lie: put together from single values they cost moves)
                        const uint64_t f = *reinterpret_cast<const uint64_t*>(&factor_s[warp][x][8 * e + pair2]);
                        const uint64_t up = *reinterpret_cast<const uint64_t*>(&offset_s[warp][x][8 * e + pair2]);
                        uint64_t p[4];
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float* y = &s[S::kTwice ? 0 : x][e % B][2 * c];
                            const float2 z = unpair(fma2(pair(y[0], y[1]), f, up));
                            const float p0 = tree_exp2(z.x), p1 = tree_exp2(z.y);
                            p[c] = pair(p0, p1);
                            tree_split(p0, p1, hi[c], lo[c]);
                        }
                        const uint64_t sum = add2(add2(p[0], p[1]), add2(p[2], p[3]));
                        if (x == 0) l[e] = fma2(l[e], *reinterpret_cast<const uint64_t*>(&alpha_s[buf][warp][8 * e + pair2]), 0);
                        l[e] = fma2(sum, iv2, l[e]);
                        st_matrix_turned(to + 1024 * PARTS * e, hi[0], hi[1], hi[2], hi[3]);
                        st_matrix_turned(to + 1024 * PARTS * e + S::kPart, lo[0], lo[1], lo[2], lo[3]);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_full[x % S::kWeights]);
                }
                freed += two;
                n += two;
                end_row = -1;
                kc += two;
                if (kc == chunk || k + 2 >= t.tiles) {  // the chunk's last step
                    end_row = pr;
                    end_left = R;
#pragma unroll
                    for (int e = 0; e < G; ++e) end_l[e] = l[e];
#pragma unroll
                    for (int e = 0; e < kMine; ++e) end_m[e] = m[e];
                    kc = 0;
                    pr += (int64_t)Hkv * R;
                }
            };
            for (int k = 0; k < t.tiles && !gone; k += 2, ++i) {
                const int two = q8_step_tiles(t, k);
                bool masked = false;
                for (int x = 0; x < two; ++x) masked = masked || (key_of(k + x) < edge && key_of(k + x) + kQ8Page > sinks);
                if (masked)
                    step(std::true_type{}, k, two);
                else
                    step(std::false_type{}, k, two);
            }
            if (gone) return false;
            return true;
        });
        if (!gone && i > 0) take(i - 1);
    }
    tm_before();
    __syncthreads();
    if (warp == S::kWarps + 10) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmem));
}

__global__ void q8kv_wait_expiry_kernel(uint64_t limit_ns)
{
    __shared__ uint64_t bar;
    if (threadIdx.x != 0) return;
    mbar_init(&bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    mbar_wait(&bar, 0, &g_q8kv_wait_timeouts, limit_ns);
}

cudaError_t launch_q8kv_wait_expiry(uint64_t limit_ns, cudaStream_t s)
{
    q8kv_wait_expiry_kernel<<<1, 32, 0, s>>>(limit_ns);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t read_q8kv_wait_timeouts(uint32_t* count, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_q8kv_wait_timeouts, sizeof(uint32_t));
    if (e == cudaSuccess && reset) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_q8kv_wait_timeouts, &zero, sizeof(uint32_t));
    }
    return e;
}

// The maps of the views' codes: dims (byte, row, head, page), a box a page of one
// head, zeros outside.  Made anew by each call: two of them take 0.1 us.
static bool q8_maps(const Q8Batch& b, int Hkv, Q8Maps* maps)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tree_map_encoder();
    if (!enc) return false;
    for (int i = 0; i < b.n_view; ++i) {
        const Q8View& v = b.view[i];
        if (v.n_chunk == 0) continue;
        const cuuint64_t dims[4] = {128, 128, (cuuint64_t)Hkv, (cuuint64_t)v.n_pages};
        const cuuint64_t strides[3] = {128, kQ8PageBytes, (cuuint64_t)v.page_stride};
        const cuuint32_t box[4] = {128, 128, 1, 1}, step[4] = {1, 1, 1, 1};
        for (int kv = 0; kv < 2; ++kv)
            if (enc(kv ? &maps->v[i] : &maps->k[i], CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<int8_t*>(kv ? v.v_codes : v.k_codes), dims,
                    strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return false;
    }
    return true;
}

template <int NG, int PARTS>
static cudaError_t launch_chunks(const Q8Maps& maps, const float* q, const Q8Batch& b, int Hq, int Hkv, int64_t units, bool runs,
                                 const Q8Scale& scale, float* part_o, float* part_ml, cudaStream_t s)
{
    using S = Q8Shape<NG, PARTS>;
    const Q8Heads heads = {Hq / Hkv, Hkv, (65536 + Hq / Hkv - 1) / (Hq / Hkv)};
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    static std::atomic<bool> done[kMaxDevices];
    cudaError_t e = set_smem_once(q8kv_chunk_kernel<NG, PARTS>, S::kBytes, done);
    if (e == cudaSuccess)
        e = launch_pdl_smem(q8kv_chunk_kernel<NG, PARTS>, dim3((unsigned)std::min<int64_t>(sms * S::kCtas, units)), dim3(S::kThreads),
                            S::kBytes, s, maps, q, b, heads, (int)units, runs, scale, part_o, part_ml);
    if (e == cudaSuccess) count_launches(1);
    return e;
}

// ---------------------------------------------------------------- merge

// Merge of one (row, query head): the chunks' results, the tail's keys and the
// path's.  One CTA of 4 warps.  Scores of the f16 keys: 16 lanes a key, eight dims
// each, key 8 i + 2 warp + lane / 16 in step i.  Sums: four dims a lane, warp w takes
// chunks w, w + 4, .. in order, then f16 keys w, w + 4, .. in order; the four are added
// in order.  Bound by latency: K and V of the first 32 f16 keys (a tail that is sealed
// at every step), statistics and the first 20 chunks' sums are all asked for before
// anything is used; a warp leaves its loops where its keys end.  Of 640 CTAs, 16 nodes
// of 40 heads, five fit a multiprocessor.  Measured, 160 and 640 CTAs with the chunks before
// them: 12.6 and 15.1 us; 64 keys in flight 13.8 and 15.7; loops that run to their full
// length 13.2 and 15.4; six CTAs a multiprocessor 13.0 and 15.5.  (Eight warps took 1 us
// less with 160 CTAs and 1 us more with 640; one order of summation serves both, as a row's
// bits do not depend on the others.)
constexpr int kQ8MergeWarps = 4, kQ8MergeThreads = 32 * kQ8MergeWarps;
constexpr int kQ8Ahead = 5;  // chunk sums in flight per warp
constexpr int kQ8Keys = 32;  // f16 keys in flight
constexpr int kQ8MaxKeys = kQ8MaxTail + kMaxTree;

__global__ void __launch_bounds__(kQ8MergeThreads, 5)
q8kv_merge_kernel(const float* q, const __grid_constant__ Q8Batch b, int Hq, int Hkv, Q8Scale scale, const float* part_o,
                  const float* part_ml, float* __restrict__ out)
{
    __shared__ float ps[kQ8MaxKeys];                    // the f16 keys' products
    __shared__ float ms[kQ8MaxChunks], ls[kQ8MaxChunks];  // the chunks' maxima and sums
    __shared__ float4 os[kQ8MergeWarps][kHeadDim / 4];  // the warps' sums
    pdl_trigger();
    const int h = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const TreeRow& row = b.row[r];
    const Q8View& v = b.view[row.view];
    const int GQ = Hq / Hkv, g = h / GQ, R = v.n_nodes * GQ, nch = v.n_chunk, tail = v.tail, n = tail + row.n_path;
    const int64_t pr0 = v.part0 + (int64_t)g * R + row.node * GQ + h % GQ, pstep = (int64_t)Hkv * R;
    const size_t rh = (size_t)r * Hq + h;
    // f16 key a: the tail's, then the path's.  It is seen at a position below `sinks` or from `from` on
    const int sinks = v.window ? max(0, v.sinks - v.sealed) : n, from = v.window ? n - v.window : 0;
    const __half *kb = v.k + g * v.head_stride, *vb = v.v + g * v.head_stride;
    const uint32_t tok = (uint32_t)v.tok_stride;  // (below 2^32: one multiplication a key)
    auto place = [&](int a) { return (uint64_t)(uint32_t)(a < tail ? a : tail + row.path[a - tail]) * tok; };
    auto seen = [&](int a) { return a < n && (a < sinks || a >= from); };
    pdl_wait();
    const int part = lane & 15;
    const float4 q0 = ld_placed_f4(q + rh * kHeadDim + 8 * part), q1 = ld_placed_f4(q + rh * kHeadDim + 8 * part + 4);
    constexpr int kK = kQ8Keys / (2 * kQ8MergeWarps), kV = kQ8Keys / kQ8MergeWarps;
    uint4 kx[kK];
    uint2 vx[kV];
    auto load_k = [&](int base) {
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            if (base + 2 * kQ8MergeWarps * i + 2 * warp >= n) break;  // (the warp as one)
            const int a = base + 2 * kQ8MergeWarps * i + 2 * warp + (lane >> 4);
            kx[i] = make_uint4(0, 0, 0, 0);
            if (seen(a)) kx[i] = ld_placed_u4(kb + place(a) + 8 * part);
        }
    };
    auto load_v = [&](int base) {
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int a = base + kQ8MergeWarps * i + warp;
            if (a >= n) break;
            vx[i] = make_uint2(0, 0);
            if (seen(a)) vx[i] = ld_placed_u2(vb + place(a) + 4 * lane);
        }
    };
    load_k(0);
    load_v(0);
    for (int c = tid; c < nch; c += kQ8MergeThreads) {
        const float* ml = part_ml + 8 * (pr0 + c * pstep);
        const float4 x = ld_placed_cg_f4(ml + 4);
        ms[c] = ld_placed_f(ml);
        ls[c] = __fmul_rn(__fadd_rn(__fadd_rn(x.x, x.y), __fadd_rn(x.z, x.w)), kQ8Down);  // (here, as the factor may be small)
    }
    float4 ov[kQ8Ahead];
    auto load_o = [&](int j) {
#pragma unroll
        for (int e = 0; e < kQ8Ahead; ++e) {
            const int c = kQ8MergeWarps * (j + e) + warp;
            if (c < nch) ov[e] = ld_placed_cg_f4(part_o + (pr0 + c * pstep) * kHeadDim + 4 * lane);
        }
    };
    load_o(0);
    for (int base = 0; base < n; base += kQ8Keys) {
        if (base > 0) load_k(base);
#pragma unroll
        for (int i = 0; i < kK; ++i) {
            if (base + 2 * kQ8MergeWarps * i + 2 * warp >= n) break;
            const int a = base + 2 * kQ8MergeWarps * i + 2 * warp + (lane >> 4);
            const float4 k0 = half4(make_uint2(kx[i].x, kx[i].y)), k1 = half4(make_uint2(kx[i].z, kx[i].w));
            float dot = __fmaf_rn(q0.w, k0.w, __fmaf_rn(q0.z, k0.z, __fmaf_rn(q0.y, k0.y, __fmul_rn(q0.x, k0.x))));
            dot = __fmaf_rn(q1.w, k1.w, __fmaf_rn(q1.z, k1.z, __fmaf_rn(q1.y, k1.y, __fmaf_rn(q1.x, k1.x, dot))));
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) dot = __fadd_rn(dot, __shfl_xor_sync(0xffffffffu, dot, o));
            if (part == 0 && a < n) ps[a] = seen(a) ? __fmul_rn(__fmul_rn(dot, scale.sign), scale.log2) : -INFINITY;
        }
    }
    __syncthreads();
    // every warp for itself: the largest of all, and the weights' sum
    float M = -INFINITY, L = 0.0f;
    for (int c = lane; c < nch; c += 32) M = fmaxf(M, ms[c]);
    for (int a = lane; a < n; a += 32) M = fmaxf(M, ps[a]);
    M = warp_max(M);  // (a row sees itself: there is one)
    for (int c = lane; c < nch; c += 32) L = __fmaf_rn(ls[c], tree_exp2(__fsub_rn(ms[c], M)), L);
    for (int a = lane; a < n; a += 32) L = __fadd_rn(L, tree_exp2(__fsub_rn(ps[a], M)));
    L = warp_sum_butterfly(L);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int j = 0; kQ8MergeWarps * j < nch; j += kQ8Ahead) {
        if (j > 0) load_o(j);
#pragma unroll
        for (int e = 0; e < kQ8Ahead; ++e) {
            const int c = kQ8MergeWarps * (j + e) + warp;
            if (c < nch) axpy4(o, ov[e], __fmul_rn(tree_exp2(__fsub_rn(ms[c], M)), kQ8Down));
        }
    }
    for (int base = 0; base < n; base += kQ8Keys) {
        if (base > 0) load_v(base);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
            const int a = base + kQ8MergeWarps * i + warp;
            if (a >= n) break;
            axpy4(o, half4(vx[i]), tree_exp2(__fsub_rn(ps[a], M)));
        }
    }
    os[warp][lane] = o;
    __syncthreads();
    const float* of = &os[0][0].x + tid;
    const float O = __fadd_rn(__fadd_rn(of[0], of[kHeadDim]), __fadd_rn(of[2 * kHeadDim], of[3 * kHeadDim]));
    out[rh * kHeadDim + tid] = __fdiv_rn(O, L);
}

cudaError_t launch_q8kv_attention(const float* q, const Q8Batch& b, int Hq, int Hkv, float scale, void* part, float* out,
                                  cudaStream_t s)
{
    int64_t units = 0, n_part = 0;
    bool runs = true;
    int rows = 0;  // the most of a KV head
    for (int i = 0; i < b.n_view; ++i) {
        const Q8View& v = b.view[i];
        units += (int64_t)v.n_chunk * Hkv;
        n_part += (int64_t)v.n_chunk * v.n_nodes * Hq;
        if (v.n_chunk == 0) continue;
        runs = runs && v.chunk == 2;
        rows = std::max(rows, v.n_nodes * (Hq / Hkv));
    }
    float* part_o = (float*)part;
    float* part_ml = part_o + n_part * kHeadDim;
    const Q8Scale sc = {scale < 0 ? -1.0f : 1.0f, (float)(std::fabs((double)scale) * 1.4426950408889634)};
    if (units > 0) {
        Q8Maps maps{};
        if (!q8_maps(b, Hkv, &maps)) return cudaErrorInvalidValue;
        // The least width that holds the rows of a KV head (a product's time goes with it).  Up to
        // 32 rows the weights are little work and two CTAs of 16 warps share a multiprocessor, so
        // that one's chain fills the other's waits (13.7 us for 15.2 with 5 rows, 18.7 for 20.3
        // with 20, 58 for 67 on long slots); above, one CTA with twice the warps on weights and
        // all of tensor memory, which holds 48 rows and more only then.
        const auto launch = rows <= 16 ? launch_chunks<1, 1> : rows <= 32 ? launch_chunks<2, 1> : rows <= 48 ? launch_chunks<3, 2>
                            : rows <= 64 ? launch_chunks<4, 2> : rows <= 80 ? launch_chunks<5, 2> : rows <= 96 ? launch_chunks<6, 2>
                                         : launch_chunks<8, 2>;
        const cudaError_t e = launch(maps, q, b, Hq, Hkv, units, runs, sc, part_o, part_ml, s);
        if (e != cudaSuccess) return e;
    }
    const cudaError_t e = launch_pdl(q8kv_merge_kernel, dim3(Hq, b.n_row), dim3(kQ8MergeThreads), s, q, b, Hq, Hkv, sc,
                                     (const float*)part_o, (const float*)part_ml, out);
    if (e != cudaSuccess) return e;
    count_launches(1);
    return cudaSuccess;
}

}  // namespace luce
