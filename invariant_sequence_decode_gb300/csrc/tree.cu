// tree.cu - attention of the nodes of draft trees over slots' caches.
//
// A slot verifies a tree of drafted tokens: node j sees the cache's prefix
// (keys 0 .. len-1), its ancestors and itself, whose K/V rows sit behind the
// prefix at len + node.  For row r of node j and query head h
//   out = sum_i e^(s_i - m) v_i / l,  s_i = scale q.k_i,  m = max s_i,  l = sum e^(s_i - m).
// The prefix, which every node of the tree sees, is cut into chunks of
// tree_chunk_keys(len, Hkv) keys; each chunk yields (m, l, sum e^(s - m) v) per row
// and the merge adds the chunks in order, then the node's own path, key by key
// from the prefix down to the node.  A node's bits so follow from its prefix
// and its path alone: the other branches of its tree, which lie between its
// ancestors in the cache, take no part in any of its sums.  Prefixes of at most
// kTreeShort keys take tree_short_kernel, which has no chunks and no merge.
//
// Prefix chunks (tree_chunk_kernel).  A tree's n nodes and a KV head's GQ query
// heads make R = n GQ <= 128 rows that share every key, so both products run
// as 128-row tcgen05.mma tiles, row = tensor-memory lane: S = Q K^T over tiles
// of 128 keys, then O = P V.  K and V are f16; q and p are fp32 and go in as
// two f16 parts each, x = hi + lo, both parts multiplied in.  The parts hold x
// to within 2^-22, the size of an fp32 sum's own error (one f16 part would lose
// 2^-11), or to within 2^-25 where that is more; so q is held in units of a power
// of two that puts its row's largest element into [2^14, 2^15), and p is
// 2^15 e^(s - m): an element of q is off by 2^-22 of itself or 2^-39 of its row's
// largest, a weight by 2^-22 of itself or 2^-40 of the largest one so far.
// Long prefixes are bound by reading K and V (64 KB a tile: at full rate an SM
// gets one in about 2,860 cycles), with the products (2,080 cycles) and the
// softmax (1,050 of them exponentials) close behind, so what matters is that
// none of the three pauses: one CTA an SM walks its share of all chunks, a
// producer warp keeps up to six 32 KB tiles in flight by TMA, one warp issues
// the products, and 256 threads (two to a row, 64 keys each) turn S into P in
// place in tensor memory and add each tile's O into registers with the running
// maximum's correction; a tile takes 2,650 cycles.  16 nodes of 40 heads over
// 130,800 keys of 8 heads: 102 us, the chunks alone 89 at 6.0 TB/s.  Short ones
// are bound by one tile's chain (K, S, softmax, P V, O: 6 us) and the merge (4 us).
#include <limits.h>

#include <algorithm>
#include <cmath>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"
#include "ring.cuh"

namespace luce {

constexpr int kTreeTile = 128;  // keys of a tile, and rows of the products
constexpr int kMaxTreeChunks = 160;
// Longest prefix that tree_short_kernel takes.  It reads the prefix once per row
// and head, the chunks once per KV head: at 64 keys it takes 3.2 us for one row
// of 8 heads and 7.3 for 16 rows of 40, through chunks 6.8 and 9.9; at 128 keys
// 4.6 and 13.0 against 6.5 and 9.3.
constexpr int kTreeShort = 64;
constexpr int kTreeCtas = 152;  // the CTAs that a cut aims at: one per multiprocessor

// Tiles of a chunk for a prefix of nt tiles.  A chunk costs its tiles and about
// one more (its q, its results); one view's chunks, Hkv heads, go to kTreeCtas
// CTAs in rounds.  Of the cuts that fill 1, 2, 3 or 4 rounds the cheapest is
// taken, the one with fewer chunks of equals: 130,800 keys of 8 heads make 19
// chunks of 54 tiles (8-tile chunks, 128 a head: 129 against 90 us, replayed).
static int tree_chunk_tiles(int nt, int Hkv)
{
    int best = nt, least = INT_MAX;
    for (int rounds = 1; rounds <= 4; ++rounds) {
        const int n = std::min({kTreeCtas * rounds / Hkv, nt, kMaxTreeChunks});
        if (n < 1) continue;
        const int tiles = (nt + n - 1) / n;
        const int cost = (Hkv * n + kTreeCtas - 1) / kTreeCtas * (tiles + 1);
        if (cost < least) {
            least = cost;
            best = tiles;
        }
    }
    return std::max(best, 1);
}

bool tree_is_short(int len) { return len <= kTreeShort; }

int tree_chunk_keys(int len, int Hkv) { return kTreeTile * tree_chunk_tiles((len + kTreeTile - 1) / kTreeTile, Hkv); }

int tree_max_chunks(int max_len, int Hkv)
{
    if (tree_is_short(max_len)) return 0;
    return std::min({(max_len + kTreeTile - 1) / kTreeTile, kMaxTreeChunks, std::max(1, 4 * kTreeCtas / Hkv)});
}

// A view chunk's partial results: part_o [row][128] and part_ml [row][4] = (m,
// l of the keys 0..63 of its tiles, l of the keys 64..127, unused), the sums
// times 2^15, with
// row = part0 + (chunk * Hkv + g) * R + i, i = node * GQ + head of the group.
size_t tree_part_bytes(int64_t n_part) { return (size_t)n_part * (kHeadDim + 4) * sizeof(float); }

__device__ __forceinline__ const __half* flat_key(const TreeView& v, const __half* base, int g, int key)
{
    return base + (int64_t)g * v.head_stride + (int64_t)key * v.tok_stride;
}

// The key's row; nullptr for a page outside the pool.
__device__ __forceinline__ const __half* tree_key(const TreeView& v, const __half* base, int g, int key)
{
    if (!v.pages) return flat_key(v, base, g, key);
    const int p = ld_placed_i(v.pages + (key >> 7));
    if (p < 0 || p >= v.n_pages) return nullptr;
    return base + (int64_t)p * v.page_stride + (int64_t)g * v.head_stride + (int64_t)(key & 127) * v.tok_stride;
}

// ---------------------------------------------------------------- chunks

// 8 warps on S, P and O; a warpgroup of which one warp feeds the tiles and one
// issues the products.  384 threads get 168 registers each (64,512 in all);
// the second kind gives up to 40, the first then has 232: 256 * 232 + 128 * 40.
constexpr int kTreeThreads = 384;
constexpr int kTreeStages = 3;     // tiles of K in flight, and of V
constexpr int kTreeTileBytes = kTreeTile * kHeadDim * 2;
constexpr int kTreeSmem = 2 * kTreeStages * kTreeTileBytes + 1024;
// tensor memory, 512 columns: S/P twice, O, q's two parts
constexpr uint32_t kColS = 0, kColO = 256, kColQ = 384;
constexpr float kLn2 = 0.6931471805599453f;
// A chunk's weights (and so its sums) are 2^kTreeUp e^(s - m): f16 has no digits
// below 2^-24, and one dominant key would take those of the chunk's others.
constexpr float kTreeUp = 15.0f, kTreeDown = 1.0f / 32768.0f;

__device__ unsigned int g_tree_wait_timeouts;

constexpr int kStageRow = 20;  // floats from row to row: 16-byte pieces of eight rows in different banks

struct TreeMaps {
    CUtensorMap k[4], v[4];
};

// The scale of the scores.  The sign goes into q (exactly), so that a tile's
// largest product is its largest score; weights are powers of two,
// e^(s - m) = 2^(log2 dot - max), log2 = |scale| log2 e.
struct TreeScale {
    float sign, abs, log2;
    float natural;  // of a maximum: ln 2 (0 for a scale of 0)
};

struct TreeBars {
    uint64_t k_full[kTreeStages], k_empty[kTreeStages], v_full[kTreeStages], v_empty[kTreeStages];
    uint64_t s_full[2];    // S of a tile is complete
    uint64_t p_full[2];    // and its P is in place
    uint64_t p_read[2];    // and that P has been multiplied
    uint64_t o_full;       // O of a tile is complete
    uint64_t o_free;       // and has been read
    uint64_t q_full;       // q's parts are in place
    uint64_t done;         // every product that was issued is complete
};

// Chunks of one (view, KV head) that a CTA takes one after the other: `chunks`
// of them from number c on, in the order view, head, chunk.
struct TreeRun {
    int view, g, c, chunks, tiles, key0, nkey;
};

// The run at chunk u of all: up to chunk `end` of all, or of one chunk.
__device__ __forceinline__ TreeRun tree_run(const TreeBatch& b, int Hkv, int u, int end)
{
    TreeRun t;
    const int u0 = u;
    t.view = 0;
    while (t.view + 1 < b.n_view && u >= Hkv * b.view[t.view].n_chunk) u -= Hkv * b.view[t.view++].n_chunk;
    const TreeView& v = b.view[t.view];
    t.g = u / v.n_chunk;
    t.c = u - t.g * v.n_chunk;
    t.chunks = min(v.n_chunk - t.c, end - u0);
    t.key0 = t.c * v.chunk;
    t.nkey = min(t.chunks * v.chunk, v.len - t.key0);
    t.tiles = (t.nkey + kTreeTile - 1) / kTreeTile;
    return t;
}

__device__ __forceinline__ uint64_t tree_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    // 128-byte swizzle; start address, leading and stride byte offsets in units of 16
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// D[128][128] (+)= A (tensor memory, f16) * B (shared memory), one 16-wide
// step, by the lane whose `elected` is set.  The whole warp comes here: issued
// from a branch of one thread, each product cost 152 cycles (its descriptor
// goes through registers that only a converged warp has at hand) against 64.
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

// 64 columns of this warp's 32 lanes of tensor memory, waited for.
__device__ __forceinline__ void tm_ld64(uint32_t addr, float* v)
{
    uint32_t r[64];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,"
        "%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%64];\n"
        " tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]), "=r"(r[32]),
          "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]), "=r"(r[40]),
          "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]), "=r"(r[48]),
          "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]), "=r"(r[56]),
          "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
        : "r"(addr));
#pragma unroll
    for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

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

__device__ __forceinline__ void st_v8(float* p, const float* v)
{
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
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

// The producer: K and V tiles of the CTA's chunks, in order.  Returns the
// tiles issued.
__device__ int tree_produce(const TreeMaps& maps, const TreeBatch& b, int Hkv, int u0, int u1, int step, uint8_t* tiles, TreeBars& bar)
{
    int i = 0;
    for (int u = u0, next; u < u1; u = next) {
        const TreeRun t = tree_run(b, Hkv, u, step ? u + 1 : u1);
        next = step ? u + step : u + t.chunks;
        const TreeView& v = b.view[t.view];
        if (u == u0) {
            pdl_wait();
            pdl_trigger();
        }
        for (int k = 0; k < t.tiles; ++k, ++i) {
            const int st = i % kTreeStages;
            const uint32_t free = ((i / kTreeStages) & 1) ^ 1;
            const int key = t.key0 + k * kTreeTile;
            int page = 0, y = key;
            if (v.pages) {
                page = ld_placed_i(v.pages + (key >> 7));
                if (page < 0 || page >= v.n_pages) page = v.n_pages;  // outside the map: zeros
                y = 0;
            }
            uint8_t* kt = tiles + st * kTreeTileBytes;
            uint8_t* vt = kt + kTreeStages * kTreeTileBytes;
            if (!mbar_wait(&bar.k_empty[st], free, &g_tree_wait_timeouts)) return i;
            mbar_expect_tx(&bar.k_full[st], kTreeTileBytes);
            tma_load_4d(kt, &maps.k[t.view], 0, y, t.g, page, &bar.k_full[st]);
            tma_load_4d(kt + kTreeTileBytes / 2, &maps.k[t.view], 64, y, t.g, page, &bar.k_full[st]);
            if (!mbar_wait(&bar.v_empty[st], free, &g_tree_wait_timeouts)) {
                ring_drain<kTreeStages>(bar.k_full, i + 1, &g_tree_wait_timeouts);
                return i;
            }
            mbar_expect_tx(&bar.v_full[st], kTreeTileBytes);
            tma_load_4d(vt, &maps.v[t.view], 0, y, t.g, page, &bar.v_full[st]);
            tma_load_4d(vt + kTreeTileBytes / 2, &maps.v[t.view], 64, y, t.g, page, &bar.v_full[st]);
        }
    }
    return i;
}

// The products, issued by one warp in the order S of tile i, P V of tile i - 1:
// while a tile's softmax runs the tensor cores have the other product of the
// tiles beside it.  One warp for both, each product's 16 steps in one go:
// issued by a warp each, the steps of S and P V alternated on the tensor cores
// and both took twice their time, with the softmax waiting for the one and the
// buffer for the other (3,050 cycles a tile against 2,650).  The issue loops
// stay loops: unrolled whole, their code (4 KB each) fell out of the
// instruction cache at every chunk's end and cost 8,000 cycles to fetch again.
// The warp sits in the scheduler of the last row quarter, which has rows to
// work on in the widest calls only.
__device__ void tree_products(const TreeBatch& b, int Hkv, int u0, int u1, int step, uint32_t tiles, uint32_t tmem,
                              TreeBars& bar)
{
    // D f32, A and B f16, 128 x 128; P V's B (V) is N-major
    constexpr uint32_t idesc_s = (1u << 4) | (16u << 17) | (8u << 24), idesc_o = idesc_s | (1u << 16);
    const uint32_t elected = elect_one();
    unsigned int* late = &g_tree_wait_timeouts;
    int i = 0, heads = 0, last = -1;
    auto values = [&](int j) {
        const int st = j % kTreeStages;
        const bool there = mbar_wait(&bar.v_full[st], (j / kTreeStages) & 1, late) &&
                           mbar_wait(&bar.p_full[j & 1], (j >> 1) & 1, late) &&
                           (j == 0 || mbar_wait(&bar.o_free, (j - 1) & 1, late));
        if (!__all_sync(0xffffffffu, there)) return false;  // (the warp leaves as one)
        tm_after();
        const uint32_t p = tmem + kColS + 128 * (j & 1) + 32;
        const uint64_t d = tree_desc(tiles + (kTreeStages + st) * kTreeTileBytes, kTreeTileBytes / 2, 1024);
        // the low parts first: an accumulation loses digits by the sum's size,
        // and theirs is small
#pragma unroll 4
        for (int ks = 0; ks < 16; ++ks)
            tree_mma(tmem + kColO, p + 64 * (ks >> 2 & 1) + 8 * (ks & 3) - 32 * (ks >> 3), d + 128 * (ks & 7), idesc_o,
                     ks > 0, elected);
        tree_commit_mma(&bar.o_full, elected);
        tree_commit_mma(&bar.p_read[j & 1], elected);
        tree_commit_mma(&bar.v_empty[st], elected);
        return true;
    };
    auto all = [&] {
        for (int u = u0, next; u < u1; u = next) {
            const TreeRun t = tree_run(b, Hkv, u, step ? u + 1 : u1);
            next = step ? u + step : u + t.chunks;
            if (t.view * Hkv + t.g != last) {
                last = t.view * Hkv + t.g;
                if (!__all_sync(0xffffffffu, mbar_wait(&bar.q_full, heads++ & 1, late))) return;
            }
            for (int k = 0; k < t.tiles; ++k, ++i) {
                const int st = i % kTreeStages;
                // (the first two buffers are free)
                const bool there = mbar_wait(&bar.k_full[st], (i / kTreeStages) & 1, late) &&
                                   mbar_wait(&bar.p_read[i & 1], ((i >> 1) & 1) ^ 1, late);
                if (!__all_sync(0xffffffffu, there)) return;
                tm_after();
                const uint32_t s = tmem + kColS + 128 * (i & 1);
                const uint64_t d = tree_desc(tiles + st * kTreeTileBytes, 16, 1024);
#pragma unroll 4
                for (int ks = 0; ks < 16; ++ks)  // the low parts first, as above
                    tree_mma(s, tmem + kColQ + 8 * (ks ^ 8), d + (ks >> 2 & 1) * (kTreeTileBytes / 32) + 2 * (ks & 3),
                             idesc_s, ks > 0, elected);
                tree_commit_mma(&bar.s_full[i & 1], elected);
                tree_commit_mma(&bar.k_empty[st], elected);
                if (i > 0 && !values(i - 1)) return;
            }
        }
        if (i > 0) values(i - 1);
    };
    all();
    // also after an expired wait, tensor memory is not freed under a product
    tree_commit_mma(&bar.done, elected);
    mbar_wait(&bar.done, 0, late);
}

// One CTA an SM, each with its share of all chunks.
__global__ void __launch_bounds__(kTreeThreads, 1)
tree_chunk_kernel(const __grid_constant__ TreeMaps maps, const float* q, const __grid_constant__ TreeBatch b,
                  int Hq, int Hkv, int units, bool runs, TreeScale scale, float* __restrict__ part_o, float* __restrict__ part_ml,
                  float* __restrict__ scores, int64_t lds)
{
    extern __shared__ uint8_t tree_smem[];
    uint8_t* tiles = tree_smem + ((1024u - (smem_addr(tree_smem) & 1023u)) & 1023u);
    __shared__ TreeBars bar;
    __shared__ uint32_t tmem_at;
    __shared__ float mx[2][2][kTreeTile];  // a row's maxima of a tile's two halves, by tile parity
    __shared__ float qmx[2][kTreeTile];    // and of |q|'s two halves
    __shared__ volatile int bail[4];       // a wait of the row quarter's warps expired
    // A warp's 32 rows, 16 columns at a time, on their way between a row per
    // thread and 64 bytes of a row per four threads: global loads and stores by
    // a row per thread touch 32 lines an instruction (q's took 3,000 cycles)
    __shared__ __align__(16) float stage[8][32 * kStageRow];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&tmem_at)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    if (tid == 0) {
        for (int i = 0; i < kTreeStages; ++i) {
            mbar_init(&bar.k_full[i], 1);
            mbar_init(&bar.k_empty[i], 1);
            mbar_init(&bar.v_full[i], 1);
            mbar_init(&bar.v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 8);
            mbar_init(&bar.p_read[i], 1);
        }
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_free, 8);
        mbar_init(&bar.q_full, 8);
        mbar_init(&bar.done, 1);
        for (int i = 0; i < 4; ++i) bail[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tmem = tmem_at;
    if (tid < 2 * b.n_view) {
        const int view = tid % b.n_view;
        const CUtensorMap* m = tid < b.n_view ? &maps.k[view] : &maps.v[view];
        if (b.view[view].n_chunk > 0)  // (a short prefix has no map)
            asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
    }
    // one-tile chunks: a run of them each (a run's heads change least); longer
    // ones: every gridDim.x-th, as chunks of unlike views then spread evenly
    int u0 = blockIdx.x, u1 = units, step = gridDim.x;
    if (runs) {
        u0 = (int)((int64_t)units * blockIdx.x / gridDim.x);
        u1 = (int)((int64_t)units * (blockIdx.x + 1) / gridDim.x);
        step = 0;
    }
    unsigned int* late = &g_tree_wait_timeouts;

    // Each role waits for the kernels before this one right before it first
    // needs what they wrote.  The producer's thread then lets the merge be
    // launched, which waits for this kernel before it reads anything.
    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 8 && lane == 0) {
            const int n = tree_produce(maps, b, Hkv, u0, u1, step, tiles, bar);
            ring_drain<kTreeStages>(bar.k_full, n, late);
            ring_drain<kTreeStages>(bar.v_full, n, late);
        }
        if (warp == 11) tree_products(b, Hkv, u0, u1, step, smem_addr(tiles), tmem, bar);
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int half = warp >> 2, quad = warp & 3, row = 32 * quad + lane, GQ = Hq / Hkv;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        uint64_t o[32];                         // the chunk's sum, dims 64 half .. 64 half + 63
        float* st = stage[warp];
        const int piece = 4 * (lane & 3);       // of the row 8 i + lane / 4, i = 0..3, that this thread loads and stores
        int far_row[4];                         // those rows' place in q and scores, from the view's head
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int rr = 32 * quad + 8 * e + (lane >> 2);
            far_row[e] = rr / GQ * Hq + rr % GQ;
        }
        int i = 0, last = -1, R = 0;
        float unit = 0.0f;                      // the row's power of two: q is held in units of it
        bool ok = true, left = false;
        // the tile whose O is still to come: its correction of the sum before
        // it (none: the chunk's first), whether the warp has rows in it, the
        // row of results that the sums go to after it (-1: it is not the
        // chunk's last) with their maximum and weights' sum
        float prev_alpha = 0.0f, prev_m = 0.0f, prev_l = 0.0f;
        bool prev_first = true, prev_live = false;
        int64_t prev_row = -1;
        auto take = [&](int j) {
            const bool done = __all_sync(0xffffffffu, mbar_wait(&bar.o_full, j & 1, late));
            tm_after();
            if (prev_live && done) {
                if (prev_first) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = 0;
                }
                const uint64_t al = pair(prev_alpha, prev_alpha);
                float x[64];
                tm_ld64(lanes + kColO + 64 * half, x);
                warp_arrive(&bar.o_free);  // (the next tile's P V waits for this)
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = fma2(o[e], al, pair(x[2 * e], x[2 * e + 1]));
            } else {
                warp_arrive(&bar.o_free);
            }
            if (prev_row >= 0 && done) {
                float* to = part_o + prev_row * kHeadDim + 64 * half;
                if (half == 0) part_ml[4 * prev_row] = prev_m;
                part_ml[4 * prev_row + 1 + half] = prev_l;
#pragma unroll
                for (int e = 0; e < 32; e += 4) {
                    const float2 a = unpair(o[e]), c = unpair(o[e + 1]), d = unpair(o[e + 2]), f = unpair(o[e + 3]);
                    const float x[8] = {a.x, a.y, c.x, c.y, d.x, d.y, f.x, f.y};
                    st_v8(to + 2 * e, x);
                }
            }
            return done;
        };
        for (int u = u0, next; !left && u < u1; u = next) {
            const TreeRun t = tree_run(b, Hkv, u, step ? u + 1 : u1);
            next = step ? u + step : u + t.chunks;
            const TreeView& v = b.view[t.view];
            const int64_t head = (int64_t)v.row0 * Hq + t.g * GQ;
            if (t.view * Hkv + t.g != last) {  // (S of every tile of the last head is complete: its q is free)
                last = t.view * Hkv + t.g;
                R = v.n_nodes * GQ;
                if (u == u0) pdl_wait();
                if (32 * quad < R) {
                    float4 x[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const bool in = 32 * quad + 8 * (e & 3) + (lane >> 2) < R;
                        x[e] = in ? ld_placed_f4(q + (head + far_row[e & 3]) * kHeadDim + 64 * half + 16 * (e >> 2) + piece)
                                  : make_float4(0, 0, 0, 0);
                    }
                    // the row's unit puts its largest element into [2^14, 2^15)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float big = 0.0f;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const float4 y = x[4 * c + e];
                            big = fmaxf(big, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w))));
                        }
                        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                        if ((lane & 3) == 0) qmx[half][32 * quad + 8 * e + (lane >> 2)] = big;
                    }
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
                    const int exp = max((__float_as_int(fmaxf(qmx[0][row], qmx[1][row])) >> 23) - 127 - 14, -112);
                    unit = __int_as_float((127 + exp) << 23);
                    const float into = __fmul_rn(scale.sign, __int_as_float((127 - exp) << 23));
                    uint32_t hi[32], lo[32];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<float4*>(st + (8 * e + (lane >> 2)) * kStageRow + piece) = x[4 * c + e];
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 y = *reinterpret_cast<const float4*>(st + lane * kStageRow + 4 * e);
                            const int at = 8 * c + 2 * e;
                            tree_split(__fmul_rn(y.x, into), __fmul_rn(y.y, into), hi[at], lo[at]);
                            tree_split(__fmul_rn(y.z, into), __fmul_rn(y.w, into), hi[at + 1], lo[at + 1]);
                        }
                        __syncwarp();
                    }
                    tm_st32(lanes + kColQ + 32 * half, hi);
                    tm_st32(lanes + kColQ + 64 + 32 * half, lo);
                } else {
                    // no rows here: products of zeros draw less power than of
                    // what happens to lie there
                    uint32_t zero[32] = {};
                    tm_st32(lanes + kColQ + 32 * half, zero);
                    tm_st32(lanes + kColQ + 64 + 32 * half, zero);
                }
                tm_wait_st();
                warp_arrive(&bar.q_full);
            }
            const bool live = 32 * quad < R;
            const int ct = v.chunk / kTreeTile;
            int kc = 0;                                                   // the chunk's tiles so far
            int64_t pr = v.part0 + ((int64_t)t.c * Hkv + t.g) * R + row;  // the chunk's row of results
            float* sc = scores && live ? scores + head * lds + t.key0 + 64 * half : nullptr;
            float m = -INFINITY, l = 0.0f;  // m: a power of two's exponent
            for (int k = 0; k < t.tiles; ++k, ++i) {
                const int n = min(kTreeTile, t.nkey - k * kTreeTile);  // keys of the tile
                if (kc == 0) {
                    m = -INFINITY;
                    l = 0.0f;
                }
                ok = ok && mbar_wait(&bar.s_full[i & 1], (i >> 1) & 1, late);
                tm_after();
                if (n < kTreeTile) {
                    // what lies behind the last key may be anything: its weight
                    // is 0, but 0 times a NaN would not be
                    const int slot = i % kTreeStages;
                    ok = ok && mbar_wait(&bar.v_full[slot], (i / kTreeStages) & 1, late);
                    uint8_t* vt = tiles + (kTreeStages + slot) * kTreeTileBytes;
                    for (int e = tid; ok && e < (kTreeTile - n) * 16; e += 256)
                        *reinterpret_cast<uint4*>(vt + (e & 8) * (kTreeTileBytes / 16) + (n + (e >> 4)) * 128 + (e & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                float alpha = 0.0f;
                if (!ok) bail[quad] = 1;
                if (live) {
                    float s[64];
                    tm_ld64(lanes + kColS + 128 * (i & 1) + 64 * half, s);
                    if (n < kTreeTile) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (64 * half + e >= n) s[e] = -INFINITY;
                    }
                    float tops[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
                    for (int e = 4; e < 64; e += 8) {
#pragma unroll
                        for (int f = 0; f < 4; ++f)
                            tops[f] = fmaxf(tops[f], e + 4 < 64 ? fmaxf(s[e + f], s[e + 4 + f]) : s[e + f]);
                    }
                    mx[i & 1][half][row] = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
                    // the two warps of a row quarter always meet here (and
                    // below), an expired wait or not, and leave together
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
                    if ((left = bail[quad])) break;
                    // rounded up, and the weights' shift down: none is above 2^kTreeUp (the
                    // shift is exact for top >= 15, else off by one unit of itself at most)
                    const float log2 = __fmul_rn(scale.log2, unit);
                    const float top = fmaxf(m, __fmul_ru(fmaxf(mx[i & 1][0][row], mx[i & 1][1][row]), log2));
                    const float at = top == -INFINITY ? 0.0f : top, up = __fsub_rd(kTreeUp, at);
                    alpha = tree_exp2(__fsub_rn(m, at));  // 0 for m = -inf
                    m = top;
                    if (sc) {
                        const float f = __fmul_rn(scale.abs, unit);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float* x = s + 16 * c + 4 * e;
                                *reinterpret_cast<float4*>(st + lane * kStageRow + 4 * e) =
                                    make_float4(__fmul_rn(x[0], f), __fmul_rn(x[1], f), __fmul_rn(x[2], f), __fmul_rn(x[3], f));
                            }
                            __syncwarp();
                            const int at = 16 * c + piece, in = n - 64 * half - at;  // keys of the tile from this piece on
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int rr = 8 * e + (lane >> 2);
                                if (32 * quad + rr >= R) break;
                                const float4 x = *reinterpret_cast<const float4*>(st + rr * kStageRow + piece);
                                float* to = sc + far_row[e] * lds + k * kTreeTile + at;
                                if (in >= 4) {
                                    *reinterpret_cast<float4*>(to) = x;
                                } else {
                                    if (in > 0) to[0] = x.x;
                                    if (in > 1) to[1] = x.y;
                                    if (in > 2) to[2] = x.z;
                                }
                            }
                            __syncwarp();
                        }
                    }
                    const uint64_t c2 = pair(log2, log2), m2 = pair(up, up);
                    uint64_t sum[4] = {0, 0, 0, 0};
                    uint32_t hi[32], lo[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const float2 x = unpair(fma2(pair(s[2 * e], s[2 * e + 1]), c2, m2));
                        const float p0 = tree_exp2(x.x), p1 = tree_exp2(x.y);
                        sum[e & 3] = add2(sum[e & 3], pair(p0, p1));
                        tree_split(p0, p1, hi[e], lo[e]);
                    }
                    const float2 ls = unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])));
                    l = __fmaf_rn(l, alpha, __fadd_rn(ls.x, ls.y));
                    tm_st32(lanes + kColS + 128 * (i & 1) + 64 * half, hi);
                    tm_st32(lanes + kColS + 128 * (i & 1) + 64 * half + 32, lo);
                    tm_wait_st();
                } else {
                    asm volatile("bar.sync %0, 64;" ::"r"(1 + quad) : "memory");
                    if ((left = bail[quad])) break;
                }
                warp_arrive(&bar.p_full[i & 1]);
                if (i > 0) ok = take(i - 1);
                prev_alpha = alpha;
                prev_first = kc == 0;
                prev_live = live;
                prev_row = -1;
                if (++kc == ct || k + 1 == t.tiles) {  // the chunk's last tile
                    kc = 0;
                    if (row < R) {
                        prev_row = pr;
                        prev_m = m;
                        prev_l = l;
                    }
                    pr += (int64_t)Hkv * R;
                }
            }
        }
        if (!left && i > 0) ok = take(i - 1) && ok;
    }
    tm_before();
    __syncthreads();
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

__global__ void tree_wait_expiry_kernel(uint64_t limit_ns)
{
    __shared__ uint64_t bar;
    if (threadIdx.x != 0) return;
    mbar_init(&bar, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    mbar_wait(&bar, 0, &g_tree_wait_timeouts, limit_ns);
}

cudaError_t launch_tree_wait_expiry(uint64_t limit_ns, cudaStream_t s)
{
    tree_wait_expiry_kernel<<<1, 32, 0, s>>>(limit_ns);
    count_launches(1);
    return cudaGetLastError();
}

cudaError_t read_tree_wait_timeouts(uint32_t* count, bool reset)
{
    cudaError_t e = cudaMemcpyFromSymbol(count, g_tree_wait_timeouts, sizeof(uint32_t));
    if (e == cudaSuccess && reset) {
        const uint32_t zero = 0;
        e = cudaMemcpyToSymbol(g_tree_wait_timeouts, &zero, sizeof(uint32_t));
    }
    return e;
}

static PFN_cuTensorMapEncodeTiled_v12000 tree_map_encoder()
{
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// The maps of the views' K and V: dims (d, key, head, page), boxes of 64 dims
// by 128 keys, zeros outside.  Made anew by each call: two of them take 0.1 us.
static bool tree_maps(const TreeBatch& b, int Hkv, TreeMaps* maps)
{
    const PFN_cuTensorMapEncodeTiled_v12000 enc = tree_map_encoder();
    if (!enc) return false;
    for (int i = 0; i < b.n_view; ++i) {
        const TreeView& v = b.view[i];
        if (v.n_chunk == 0) continue;
        const cuuint64_t dims[4] = {kHeadDim, (cuuint64_t)v.cap, (cuuint64_t)Hkv, (cuuint64_t)v.n_pages};
        const cuuint64_t strides[3] = {(cuuint64_t)v.tok_stride * 2, (cuuint64_t)v.head_stride * 2,
                                       (cuuint64_t)(v.pages ? v.page_stride : v.head_stride) * 2};
        const cuuint32_t box[4] = {kHeadDim / 2, kTreeTile, 1, 1}, step[4] = {1, 1, 1, 1};
        for (int kv = 0; kv < 2; ++kv)
            if (enc(kv ? &maps->v[i] : &maps->k[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<__half*>(kv ? v.v : v.k),
                    dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
                return false;
    }
    return true;
}

// Merge of one (row, query head): the prefix's chunks and the node's path.
// One CTA of 4 warps, 4 dims a lane.  Warp w sums chunks w, w + 4, .. in order
// and then path keys w, w + 4, ..; the four sums are added in order.  It is
// bound by latency, not bytes (R 528 bytes a chunk), so everything it reads is
// asked for before anything is used: q, the path's K and V, the statistics and
// the first chunks' sums together.  All of it behind this kernel's own wait: q
// and the path's rows are by the kernels before the chunks, for which the chunk
// kernel has waited, but that orders nothing for the reader here.  Ahead of the
// wait only addresses are formed and lines of flat caches asked for in L2 (16
// nodes with scores 12.3 us, 13.2 without that).
constexpr int kMergeAhead = 8;  // chunk sums in flight per warp

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

// Asks for a line in L2; no value is read.
__device__ __forceinline__ void fetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory"); }

__global__ void __launch_bounds__(kHeadDim)
tree_merge_kernel(const float* q, const __grid_constant__ TreeBatch b, int Hq, int Hkv, TreeScale scale,
                  const float* part_o, const float* part_ml, float* __restrict__ out,
                  float* __restrict__ scores, int64_t lds, float* __restrict__ stats, int8_t* __restrict__ out_q,
                  float* __restrict__ out_d)
{
    __shared__ float ps[kMaxTree];            // the path's products
    __shared__ float4 os[4][kHeadDim / 4];    // the warps' sums
    pdl_trigger();
    const int h = blockIdx.x, r = b.long_row[blockIdx.y], tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const TreeRow& row = b.row[r];
    const TreeView& v = b.view[row.view];
    const int GQ = Hq / Hkv, g = h / GQ, R = v.n_nodes * GQ, np = row.n_path, nch = v.n_chunk;
    const int64_t pr0 = v.part0 + (int64_t)g * R + row.node * GQ + h % GQ, pstep = (int64_t)Hkv * R;
    const size_t rh = (size_t)r * Hq + h;
    const float* qp = q + rh * kHeadDim + 4 * lane;
    fetch_l2(qp);
    const __half *kp[4], *vp[4];
    if (!v.pages) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (warp + 4 * i < np) {
                const int key = v.len + row.path[warp + 4 * i];
                kp[i] = flat_key(v, v.k, g, key) + 4 * lane;
                vp[i] = flat_key(v, v.v, g, key) + 4 * lane;
                fetch_l2(kp[i]);
                fetch_l2(vp[i]);
            }
    }
    constexpr int kStats = kMaxTreeChunks / 32;
    const float* mlp = part_ml + 4 * (pr0 + lane * pstep);
    const float4* po = reinterpret_cast<const float4*>(part_o) + (pr0 + warp * pstep) * (kHeadDim / 4) + lane;
    int64_t ml_step = 32 * 4 * pstep, po_step = 4 * pstep * (kHeadDim / 4);
    int chunks = nch;
    asm volatile("" : "+l"(mlp), "+l"(po), "+l"(ml_step), "+l"(po_step), "+r"(chunks));  // (formed by now)
    pdl_wait();
    const float4 qv = ld_placed_f4(qp);
    uint2 kx[4], vx[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        kx[i] = vx[i] = make_uint2(0, 0);
        if (warp + 4 * i >= np) continue;
        if (v.pages) {
            const int key = v.len + row.path[warp + 4 * i];
            const __half* base = tree_key(v, v.k, g, key);
            kp[i] = base ? base + 4 * lane : nullptr;
            vp[i] = base ? v.v + (kp[i] - v.k) : nullptr;
        }
        if (kp[i]) {
            kx[i] = ld_placed_u2(kp[i]);
            vx[i] = ld_placed_u2(vp[i]);
        }
    }
    // every warp has all chunks' statistics: chunk lane + 32 j in its lane
    float w[kStats], L = 0.0f, M = -INFINITY;
    float2 ls[kStats];
#pragma unroll
    for (int j = 0; j < kStats; ++j) {
        const int c = lane + 32 * j;
        w[j] = -INFINITY;
        ls[j] = make_float2(0.0f, 0.0f);
        if (c < chunks) {
            const float4 ml = ld_placed_cg_f4(mlp + j * ml_step);
            w[j] = ml.x;
            ls[j] = make_float2(ml.y, ml.z);
        }
    }
    float4 ov[kMergeAhead];
#pragma unroll
    for (int j = 0; j < kMergeAhead; ++j)
        if (warp + 4 * j < chunks) ov[j] = ld_placed_cg_f4(po + j * po_step);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (warp + 4 * i >= np) break;
        const float4 k = half4(kx[i]);
        const float dot = warp_sum_butterfly(
            __fmaf_rn(qv.w, k.w, __fmaf_rn(qv.z, k.z, __fmaf_rn(qv.y, k.y, __fmul_rn(qv.x, k.x)))));
        if (lane == 0) ps[warp + 4 * i] = __fmul_rn(dot, scale.sign);
    }
    __syncthreads();
    if (scores && tid < v.n_nodes) {
        float x = -INFINITY;
        for (int a = 0; a < np; ++a)
            if (row.path[a] == tid) x = __fmul_rn(ps[a], scale.abs);
        scores[rh * lds + v.len + tid] = x;
    }
    float p = lane < np ? __fmul_rn(ps[lane], scale.log2) : -INFINITY;
#pragma unroll
    for (int j = 0; j < kStats; ++j) M = fmaxf(M, w[j]);
    M = warp_max(fmaxf(M, p));
    const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int j = 0; j < kStats; ++j) {
        w[j] = __fmul_rn(tree_exp2(__fsub_rn(w[j], ref)), kTreeDown);
        L = __fmaf_rn(__fadd_rn(ls[j].x, ls[j].y), w[j], L);
    }
    p = tree_exp2(__fsub_rn(p, ref));
    L = __fadd_rn(warp_sum_butterfly(L), warp_sum_butterfly(p));
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int j = 0; j < kMaxTreeChunks / 4; ++j) {  // chunk 4 j + warp: its weight is in lane (4 j + warp) & 31's w[j >> 3]
        const int c = 4 * j + warp;
        if ((j & (kMergeAhead - 1)) == 0 && j > 0) {
            if (4 * j >= chunks) break;
#pragma unroll
            for (int e = 0; e < kMergeAhead; ++e)
                if (c + 4 * e < chunks) ov[e] = ld_placed_cg_f4(po + (j + e) * po_step);
        }
        const float f = __shfl_sync(0xffffffffu, w[j >> 3], c & 31);
        if (c < chunks) axpy4(o, ov[j & (kMergeAhead - 1)], f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float f = __shfl_sync(0xffffffffu, p, warp + 4 * i);
        if (warp + 4 * i < np) axpy4(o, half4(vx[i]), f);
    }
    os[warp][lane] = o;
    __syncthreads();
    const float* of = &os[0][0].x;
    const float O = __fadd_rn(__fadd_rn(of[tid], of[kHeadDim + tid]), __fadd_rn(of[2 * kHeadDim + tid], of[3 * kHeadDim + tid]));
    const float val = __fdiv_rn(O, L);
    out[rh * kHeadDim + tid] = val;
    if (stats && tid == 0) *reinterpret_cast<float2*>(stats + 2 * rh) = make_float2(__fmul_rn(M, scale.natural), L);
    if (out_q) {
        float dd;
        const int code = q8_quantize_lane(val, &dd);
        out_q[rh * kHeadDim + tid] = (int8_t)code;
        if (lane == 0) out_d[(rh * kHeadDim + tid) / 32] = dd;
    }
}

// Short prefixes: one CTA of 8 warps per (row, query head) over the keys that
// the row sees, prefix then path.  Scores: eight lanes to a key, 16 dims each,
// key 32 i + 4 warp + lane / 8 in step i; values: four dims a lane, warp w sums
// keys w, w + 8, .. in order and the eight sums are added in order.  Bound by
// latency: K and V of all steps are asked for at once.
constexpr int kShortThreads = 256;
constexpr int kShortKeys = kTreeShort + kMaxTree;
constexpr int kShortSteps = (kShortKeys + 31) / 32;

__global__ void __launch_bounds__(kShortThreads)
tree_short_kernel(const float* q, const __grid_constant__ TreeBatch b, int Hq, int Hkv, TreeScale scale,
                  float* __restrict__ out, float* __restrict__ scores, int64_t lds, float* __restrict__ stats,
                  int8_t* __restrict__ out_q, float* __restrict__ out_d)
{
    __shared__ float ps[32 * kShortSteps];    // the keys' products
    __shared__ float4 os[8][kHeadDim / 4];    // the warps' sums
    pdl_trigger();
    const int h = blockIdx.x, r = b.short_row[blockIdx.y], tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const TreeRow& row = b.row[r];
    const TreeView& v = b.view[row.view];
    const int g = h / (Hq / Hkv), n = v.len + row.n_path;
    const size_t rh = (size_t)r * Hq + h;
    auto key_at = [&](int a) { return a < v.len ? a : v.len + row.path[a - v.len]; };
    pdl_wait();
    const int part = lane & 7;  // dims 16 part .. 16 part + 15
    float4 qv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) qv[e] = ld_placed_f4(q + rh * kHeadDim + 16 * part + 4 * e);
    uint4 kx[kShortSteps][2];
#pragma unroll
    for (int i = 0; i < kShortSteps; ++i) {
        const int a = 32 * i + 4 * warp + (lane >> 3);
        kx[i][0] = kx[i][1] = make_uint4(0, 0, 0, 0);
        const __half* kp = a < n ? tree_key(v, v.k, g, key_at(a)) : nullptr;
        if (kp) {
            kx[i][0] = ld_placed_u4(kp + 16 * part);
            kx[i][1] = ld_placed_u4(kp + 16 * part + 8);
        }
    }
    constexpr int kPer = (kShortKeys + 7) / 8;
    uint2 vx[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int a = warp + 8 * i;
        vx[i] = make_uint2(0, 0);
        const __half* vp = a < n ? tree_key(v, v.v, g, key_at(a)) : nullptr;
        if (vp) vx[i] = ld_placed_u2(vp + 4 * lane);
    }
#pragma unroll
    for (int i = 0; i < kShortSteps; ++i) {
        const int a = 32 * i + 4 * warp + (lane >> 3);
        float dot = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint4 x = kx[i][e >> 1];
            const float4 k = half4(e & 1 ? make_uint2(x.z, x.w) : make_uint2(x.x, x.y));
            dot = __fmaf_rn(qv[e].w, k.w, __fmaf_rn(qv[e].z, k.z, __fmaf_rn(qv[e].y, k.y, __fmaf_rn(qv[e].x, k.x, dot))));
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) dot = __fadd_rn(dot, __shfl_xor_sync(0xffffffffu, dot, o));
        if (part == 0) ps[a] = a < n ? __fmul_rn(dot, scale.sign) : -INFINITY;
    }
    __syncthreads();
    if (scores) {
        float* sc = scores + rh * lds;
        if (tid < v.len) sc[tid] = __fmul_rn(ps[tid], scale.abs);
        if (tid >= kShortThreads - kMaxTree && tid - (kShortThreads - kMaxTree) < v.n_nodes) {
            const int node = tid - (kShortThreads - kMaxTree);
            float x = -INFINITY;
            for (int a = 0; a < row.n_path; ++a)
                if (row.path[a] == node) x = __fmul_rn(ps[v.len + a], scale.abs);
            sc[v.len + node] = x;
        }
    }
    // every warp has all keys' weights: key lane + 32 i in its lane
    float p[kShortSteps], M = -INFINITY, L = 0.0f;
#pragma unroll
    for (int i = 0; i < kShortSteps; ++i) {
        p[i] = 32 * i + lane < n ? __fmul_rn(ps[32 * i + lane], scale.log2) : -INFINITY;
        M = fmaxf(M, p[i]);
    }
    M = warp_max(M);
    const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int i = 0; i < kShortSteps; ++i) {
        p[i] = tree_exp2(__fsub_rn(p[i], ref));
        L = __fadd_rn(L, p[i]);
    }
    L = warp_sum_butterfly(L);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const float f = __shfl_sync(0xffffffffu, p[i >> 2], (warp + 8 * i) & 31);
        if (warp + 8 * i < n) axpy4(o, half4(vx[i]), f);
    }
    os[warp][lane] = o;
    __syncthreads();
    if (tid < kHeadDim) {
        const float* of = &os[0][0].x + tid;
        float O = of[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) O = __fadd_rn(O, of[e * kHeadDim]);
        const float val = __fdiv_rn(O, L);
        out[rh * kHeadDim + tid] = val;
        if (stats && tid == 0) *reinterpret_cast<float2*>(stats + 2 * rh) = make_float2(__fmul_rn(M, scale.natural), L);
        if (out_q) {
            float dd;
            const int code = q8_quantize_lane(val, &dd);
            out_q[rh * kHeadDim + tid] = (int8_t)code;
            if (lane == 0) out_d[(rh * kHeadDim + tid) / 32] = dd;
        }
    }
}

cudaError_t launch_tree_attention(const float* q, const TreeBatch& b, int Hq, int Hkv, float scale, void* part,
                                  float* out, float* scores, int64_t lds, float* stats, int8_t* out_q, float* out_d,
                                  cudaStream_t s)
{
    int64_t units = 0, n_part = 0;
    bool runs = true;
    for (int i = 0; i < b.n_view; ++i) {
        units += (int64_t)b.view[i].n_chunk * Hkv;
        runs = runs && b.view[i].chunk == kTreeTile;
        n_part += (int64_t)b.view[i].n_chunk * b.view[i].n_nodes * Hq;
    }
    float* part_o = (float*)part;
    float* part_ml = part_o + n_part * kHeadDim;
    // (a scale of 0 weighs all keys alike: its exponents are 0 to within 2^-100)
    const TreeScale sc = {scale < 0 ? -1.0f : 1.0f, std::fabs(scale),
                          std::max((float)(std::fabs((double)scale) * 1.4426950408889634), 1e-37f),
                          scale == 0 ? 0.0f : kLn2};
    if (units > 0) {
        TreeMaps maps{};
        if (!tree_maps(b, Hkv, &maps)) return cudaErrorInvalidValue;
        const int sms = sm_count();
        if (sms <= 0) return cudaErrorInvalidDevice;
        static std::atomic<bool> done[kMaxDevices];
        cudaError_t e = set_smem_once(tree_chunk_kernel, kTreeSmem, done);
        if (e == cudaSuccess)
            e = launch_pdl_smem(tree_chunk_kernel, dim3((unsigned)std::min<int64_t>(sms, units)), dim3(kTreeThreads),
                                kTreeSmem, s, maps, q, b, Hq, Hkv, (int)units, runs, sc, part_o, part_ml, scores, lds);
        if (e != cudaSuccess) return e;
        count_launches(1);
        e = launch_pdl(tree_merge_kernel, dim3(Hq, b.n_long), dim3(kHeadDim), s, q, b, Hq, Hkv, sc, (const float*)part_o,
                       (const float*)part_ml, out, scores, lds, stats, out_q, out_d);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    if (b.n_short > 0) {
        const cudaError_t e = launch_pdl(tree_short_kernel, dim3(Hq, b.n_short), dim3(kShortThreads), s, q, b, Hq, Hkv, sc,
                                         out, scores, lds, stats, out_q, out_d);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    return cudaSuccess;
}

}  // namespace luce
