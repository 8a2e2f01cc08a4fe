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
//
// Prefix chunks (tree_chunk_kernel).  A tree's n nodes and a KV head's GQ query
// heads make R = n GQ <= 128 rows that share every key, so both products run
// as 128-row tcgen05.mma tiles, row = tensor-memory lane: S = Q K^T over tiles
// of 128 keys, then O = P V.  K and V are f16; q and p are fp32 and go in as
// two f16 parts each, x = hi + lo, both parts multiplied in: the products then
// carry 2^-22 of q and p, the size of an fp32 sum's own error, where one f16
// part would lose 2^-11.
// The kernel is bound by reading K and V (64 KB a tile; at full rate an SM gets
// one in about 2,800 cycles, the four products take about 1,024), so what
// matters is that loads never pause: one CTA an SM walks its share of all
// chunks, a producer warp keeps up to six 32 KB tiles in flight by TMA, one
// thread issues the products, and 256 threads (two to a row, 64 keys each)
// turn S into P in place in tensor memory and add each tile's O into registers
// with the running maximum's correction.
#include <math.h>

#include <algorithm>

#include "cache.h"
#include "common.cuh"
#include "kernels.h"
#include "ring.cuh"

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

constexpr int kMaxTreeChunks = 128;
constexpr int kTreeTile = 128;  // keys of a tile, and rows of the products

// A view chunk's partial results: part_o [row][128] and part_ml [row][4] = (m,
// l of the keys 0..63 of its tiles, l of the keys 64..127, unused), with
// row = part0 + (chunk * Hkv + g) * R + i, i = node * GQ + head of the group.
size_t tree_part_bytes(int64_t n_part) { return (size_t)n_part * (kHeadDim + 4) * sizeof(float); }

__device__ __forceinline__ const __half* tree_key(const TreeView& v, const __half* base, int g, int key)
{
    if (!v.pages) return base + (int64_t)g * v.head_stride + (int64_t)key * v.tok_stride;
    const int p = __ldg(v.pages + (key >> 7));
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
constexpr float kLog2e = 1.4426950408889634f;

__device__ unsigned int g_tree_wait_timeouts;

struct TreeMaps {
    CUtensorMap k[4], v[4];
};

struct TreeBars {
    uint64_t k_full[kTreeStages], k_empty[kTreeStages], v_full[kTreeStages], v_empty[kTreeStages];
    uint64_t s_full[2];    // S of a tile is complete
    uint64_t p_full[2];    // and its P is in place
    uint64_t o_full;       // O of a tile is complete
    uint64_t o_free;       // and has been read
    uint64_t q_full;       // q's parts are in place
    uint64_t x_full[4];    // the maxima of a row quarter's two halves are exchanged
};

// A chunk of a (view, KV head), in the order view, head, chunk.
struct TreeUnit {
    int view, g, c, tiles, key0, nkey;
};

__device__ __forceinline__ TreeUnit tree_unit(const TreeBatch& b, int Hkv, int u)
{
    TreeUnit t;
    t.view = 0;
    while (t.view + 1 < b.n_view && u >= Hkv * b.view[t.view].n_chunk) u -= Hkv * b.view[t.view++].n_chunk;
    const TreeView& v = b.view[t.view];
    t.g = u / v.n_chunk;
    t.c = u - t.g * v.n_chunk;
    t.key0 = t.c * v.chunk;
    t.nkey = min(v.chunk, v.len - t.key0);
    t.tiles = (t.nkey + kTreeTile - 1) / kTreeTile;
    return t;
}

// The first chunk that begins at or behind tile `at` of all tiles.
__device__ __forceinline__ int tree_first_unit(const TreeBatch& b, int Hkv, int at)
{
    int u = 0;
    for (int i = 0; i < b.n_view; ++i) {
        const TreeView& v = b.view[i];
        const int nt = (v.len + kTreeTile - 1) / kTreeTile, ct = v.chunk / kTreeTile;
        if (at < nt * Hkv) return u + at / nt * v.n_chunk + (at % nt + ct - 1) / ct;
        at -= nt * Hkv;
        u += Hkv * v.n_chunk;
    }
    return u;
}

__device__ __forceinline__ uint64_t tree_desc(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    // 128-byte swizzle; start address, leading and stride byte offsets in units of 16
    return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// D[128][128] (+)= A (tensor memory, f16) * B (shared memory); one 16-wide step.
__device__ __forceinline__ void tree_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate));
}

__device__ __forceinline__ void tree_commit_mma(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
__device__ __forceinline__ void tm_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 or 64 columns of this warp's 32 lanes of tensor memory, waited for.
__device__ __forceinline__ void tm_ld32(uint32_t addr, float* v)
{
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        " tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
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

// e^x = 2^(x log2 e), within about 2^-22 for the x <= 0 that it is given.
__device__ __forceinline__ float tree_exp(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(__fmul_rn(x, kLog2e)));
    return y;
}

// Two fp32 values as f16 pairs, x = hi + lo; the first in the low half.
__device__ __forceinline__ void tree_split(float x0, float x1, uint32_t& hi, uint32_t& lo)
{
    const __half2 h = __floats2half2_rn(x0, x1);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(__fsub_rn(x0, f.x), __fsub_rn(x1, f.y));
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}

__device__ __forceinline__ void st_v8(float* p, const float* v)
{
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// The producer: K and V tiles of the CTA's chunks, in order.  Returns the
// tiles issued.
__device__ int tree_produce(const TreeMaps& maps, const TreeBatch& b, int Hkv, int u0, int u1, uint8_t* tiles, TreeBars& bar)
{
    int i = 0;
    for (int u = u0; u < u1; ++u) {
        const TreeUnit t = tree_unit(b, Hkv, u);
        const TreeView& v = b.view[t.view];
        for (int k = 0; k < t.tiles; ++k, ++i) {
            const int st = i % kTreeStages;
            const uint32_t free = ((i / kTreeStages) & 1) ^ 1;
            const int key = t.key0 + k * kTreeTile;
            int page = 0, y = key;
            if (v.pages) {
                page = __ldg(v.pages + (key >> 7));
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

// The products: S of tile i is issued before P V of tile i - 1, so the tensor
// cores work on one tile while the other's softmax runs.
__device__ void tree_products(const TreeBatch& b, int Hkv, int u0, int u1, uint32_t tiles, uint32_t tmem, TreeBars& bar)
{
    // D f32, A and B f16, 128 x 128; P V's B (V) is N-major
    constexpr uint32_t idesc_s = (1u << 4) | (16u << 17) | (8u << 24), idesc_o = idesc_s | (1u << 16);
    unsigned int* late = &g_tree_wait_timeouts;
    int i = 0, heads = 0, last = -1;
    auto values = [&](int j) {
        const int st = j % kTreeStages;
        if (!mbar_wait(&bar.p_full[j & 1], (j >> 1) & 1, late) || !mbar_wait(&bar.v_full[st], (j / kTreeStages) & 1, late) ||
            (j > 0 && !mbar_wait(&bar.o_free, (j - 1) & 1, late)))
            return false;
        tm_after();
        const uint32_t vt = tiles + (kTreeStages + st) * kTreeTileBytes, p = tmem + kColS + 128 * (j & 1);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
            const uint64_t d = tree_desc(vt + 2048 * ks, kTreeTileBytes / 2, 1024);
            const uint32_t a = p + 64 * (ks >> 2) + 8 * (ks & 3);
            tree_mma(tmem + kColO, a, d, idesc_o, ks > 0);
            tree_mma(tmem + kColO, a + 32, d, idesc_o, true);
        }
        tree_commit_mma(&bar.v_empty[st]);
        tree_commit_mma(&bar.o_full);
        return true;
    };
    for (int u = u0; u < u1; ++u) {
        const TreeUnit t = tree_unit(b, Hkv, u);
        if (t.view * Hkv + t.g != last) {
            last = t.view * Hkv + t.g;
            if (!mbar_wait(&bar.q_full, heads++ & 1, late)) return;
        }
        for (int k = 0; k < t.tiles; ++k, ++i) {
            const int st = i % kTreeStages;
            // P of tile i - 2 is read, its S and P may be overwritten
            if ((i > 1 && !mbar_wait(&bar.o_full, (i - 2) & 1, late)) ||
                !mbar_wait(&bar.k_full[st], (i / kTreeStages) & 1, late))
                return;
            tm_after();
            const uint32_t kt = tiles + st * kTreeTileBytes, s = tmem + kColS + 128 * (i & 1);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint64_t d = tree_desc(kt + (ks >> 2) * (kTreeTileBytes / 2) + 32 * (ks & 3), 16, 1024);
                tree_mma(s, tmem + kColQ + 8 * ks, d, idesc_s, ks > 0);
                tree_mma(s, tmem + kColQ + 64 + 8 * ks, d, idesc_s, true);
            }
            tree_commit_mma(&bar.k_empty[st]);
            tree_commit_mma(&bar.s_full[i & 1]);
            if (i > 0 && !values(i - 1)) return;
        }
    }
    if (i > 0) values(i - 1);
}

// One CTA an SM; CTA c takes the chunks that begin in its share of all tiles.
__global__ void __launch_bounds__(kTreeThreads, 1)
tree_chunk_kernel(const __grid_constant__ TreeMaps maps, const float* __restrict__ q, const __grid_constant__ TreeBatch b,
                  int Hq, int Hkv, int all_tiles, float scale, float* __restrict__ part_o, float* __restrict__ part_ml,
                  float* __restrict__ scores, int64_t lds)
{
    extern __shared__ uint8_t tree_smem[];
    uint8_t* tiles = tree_smem + ((1024u - (smem_addr(tree_smem) & 1023u)) & 1023u);
    __shared__ TreeBars bar;
    __shared__ uint32_t tmem_at;
    __shared__ float mx[2][2][kTreeTile];  // a row's maxima of a tile's two halves, by tile parity
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
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
            mbar_init(&bar.p_full[i], 256);
        }
        mbar_init(&bar.o_full, 1);
        mbar_init(&bar.o_free, 256);
        mbar_init(&bar.q_full, 256);
        for (int i = 0; i < 4; ++i) mbar_init(&bar.x_full[i], 64);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tm_before();
    __syncthreads();
    tm_after();
    const uint32_t tmem = tmem_at;
    const int u0 = tree_first_unit(b, Hkv, (int)((int64_t)all_tiles * blockIdx.x / gridDim.x));
    const int u1 = tree_first_unit(b, Hkv, (int)((int64_t)all_tiles * (blockIdx.x + 1) / gridDim.x));
    unsigned int* late = &g_tree_wait_timeouts;
    pdl_wait();

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
        if (warp == 8 && lane == 0) {
            asm volatile("fence.proxy.async;" ::: "memory");  // the step's own rows were written by plain stores
            const int n = tree_produce(maps, b, Hkv, u0, u1, tiles, bar);
            ring_drain<kTreeStages>(bar.k_full, n, late);
            ring_drain<kTreeStages>(bar.v_full, n, late);
        }
        if (warp == 9 && lane == 0) tree_products(b, Hkv, u0, u1, smem_addr(tiles), tmem, bar);
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        const int half = warp >> 2, quad = warp & 3, row = 32 * quad + lane, GQ = Hq / Hkv;
        const uint32_t lanes = tmem + ((uint32_t)(32 * quad) << 16);
        float o[64];                            // the chunk's sum, dims 64 half .. 64 half + 63
        int i = 0, last = -1, R = 0, xn = 0;
        bool ok = true;
        // the tile whose O is still to come: its correction of the sum before
        // it, whether the warp has rows in it, where the sum goes after it
        float prev_alpha = 0.0f;
        bool prev_live = false;
        float* prev_out = nullptr;
        auto take = [&](int j) {
            if (!mbar_wait(&bar.o_full, j & 1, late)) return false;
            tm_after();
            if (prev_live) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x[32];
                    tm_ld32(lanes + kColO + 64 * half + 32 * c, x);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        o[32 * c + e] = prev_alpha == 0.0f ? x[e] : __fmaf_rn(o[32 * c + e], prev_alpha, x[e]);
                }
            }
            tm_before();
            mbar_arrive(&bar.o_free);
            if (prev_out) {
#pragma unroll
                for (int e = 0; e < 64; e += 8) st_v8(prev_out + e, o + e);
            }
            return true;
        };
        for (int u = u0; ok && u < u1; ++u) {
            const TreeUnit t = tree_unit(b, Hkv, u);
            const TreeView& v = b.view[t.view];
            if (t.view * Hkv + t.g != last) {  // (S of every tile of the last head is complete: its q is free)
                last = t.view * Hkv + t.g;
                R = v.n_nodes * GQ;
                if (32 * quad < R) {
                    uint32_t hi[32], lo[32];
                    const float* qr = q + ((size_t)(v.row0 + row / GQ) * Hq + t.g * GQ + row % GQ) * kHeadDim + 64 * half;
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float4 x = row < R ? *reinterpret_cast<const float4*>(qr + 4 * e) : make_float4(0, 0, 0, 0);
                        tree_split(x.x, x.y, hi[2 * e], lo[2 * e]);
                        tree_split(x.z, x.w, hi[2 * e + 1], lo[2 * e + 1]);
                    }
                    tm_st32(lanes + kColQ + 32 * half, hi);
                    tm_st32(lanes + kColQ + 64 + 32 * half, lo);
                    tm_wait_st();
                }
                tm_before();
                mbar_arrive(&bar.q_full);
            }
            const bool live = 32 * quad < R, valid = row < R;
            const int64_t pr = v.part0 + ((int64_t)t.c * Hkv + t.g) * R + row;
            float* sc = scores && valid ? scores + ((size_t)(v.row0 + row / GQ) * Hq + t.g * GQ + row % GQ) * lds + t.key0 +
                                              64 * half
                                        : nullptr;
            float m = -INFINITY, l = 0.0f;
            for (int k = 0; k < t.tiles; ++k, ++i) {
                const int n = min(kTreeTile, t.nkey - k * kTreeTile);  // keys of the tile
                if (!(ok = mbar_wait(&bar.s_full[i & 1], (i >> 1) & 1, late))) break;
                tm_after();
                if (n < kTreeTile) {
                    // what lies behind the last key may be anything: its weight
                    // is 0, but 0 times a NaN would not be
                    const int st = i % kTreeStages;
                    if (!(ok = mbar_wait(&bar.v_full[st], (i / kTreeStages) & 1, late))) break;
                    uint8_t* vt = tiles + (kTreeStages + st) * kTreeTileBytes;
                    for (int e = tid; e < (kTreeTile - n) * 16; e += 256)
                        *reinterpret_cast<uint4*>(vt + (e & 8) * (kTreeTileBytes / 16) + (n + (e >> 4)) * 128 + (e & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                float alpha = 0.0f;
                if (live) {
                    float s[64];
                    tm_ld64(lanes + kColS + 128 * (i & 1) + 64 * half, s);
                    float top = -INFINITY;
#pragma unroll
                    for (int e = 0; e < 64; ++e) s[e] = __fmul_rn(s[e], scale);
                    if (n < kTreeTile) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (64 * half + e >= n) s[e] = -INFINITY;
                    }
                    if (sc) {
                        float* to = sc + k * kTreeTile;
#pragma unroll
                        for (int e = 0; e < 64; e += 4) {
                            if (64 * half + e + 3 < n)
                                *reinterpret_cast<float4*>(to + e) = make_float4(s[e], s[e + 1], s[e + 2], s[e + 3]);
                            else
#pragma unroll
                                for (int f = e; f < e + 4; ++f)
                                    if (64 * half + f < n) to[f] = s[f];
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 64; ++e) top = fmaxf(top, s[e]);
                    mx[xn & 1][half][row] = top;
                    mbar_arrive(&bar.x_full[quad]);
                    if (!(ok = mbar_wait(&bar.x_full[quad], xn & 1, late))) break;
                    top = fmaxf(m, fmaxf(mx[xn & 1][0][row], mx[xn & 1][1][row]));
                    ++xn;
                    const float at = top == -INFINITY ? 0.0f : top;
                    if (k > 0) alpha = tree_exp(__fsub_rn(m, at));  // 0 for m = -inf
                    m = top;
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    uint32_t hi[32], lo[32];
#pragma unroll
                    for (int e = 0; e < 64; e += 2) {
                        const float p0 = tree_exp(__fsub_rn(s[e], at)), p1 = tree_exp(__fsub_rn(s[e + 1], at));
                        sum[e & 2] = __fadd_rn(sum[e & 2], p0);
                        sum[(e & 2) + 1] = __fadd_rn(sum[(e & 2) + 1], p1);
                        tree_split(p0, p1, hi[e / 2], lo[e / 2]);
                    }
                    l = __fmaf_rn(l, alpha, __fadd_rn(__fadd_rn(sum[0], sum[1]), __fadd_rn(sum[2], sum[3])));
                    tm_st32(lanes + kColS + 128 * (i & 1) + 64 * half, hi);
                    tm_st32(lanes + kColS + 128 * (i & 1) + 64 * half + 32, lo);
                    tm_wait_st();
                }
                tm_before();
                mbar_arrive(&bar.p_full[i & 1]);
                if (i > 0 && !(ok = take(i - 1))) break;
                prev_alpha = alpha;
                prev_live = live;
                prev_out = valid && k + 1 == t.tiles ? part_o + pr * kHeadDim + 64 * half : nullptr;
                if (prev_out) {
                    if (half == 0) part_ml[4 * pr] = m;
                    part_ml[4 * pr + 1 + half] = l;
                }
            }
        }
        if (ok && i > 0) ok = take(i - 1);
        // after an expired wait products may still be running: wait once more
        // (bounded) for the last of them before tensor memory is freed
        if (!ok && tid == 0 && i > 0) mbar_wait(&bar.o_full, (i - 1) & 1, late);
    }
    tm_before();
    __syncthreads();
    if (warp == 9) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
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

// The maps of the views' K and V: dims (d, key, head, page), boxes of 64 dims
// by 128 keys.
static bool tree_maps(const TreeBatch& b, int Hkv, TreeMaps* maps)
{
    for (int i = 0; i < b.n_view; ++i) {
        const TreeView& v = b.view[i];
        if (v.n_chunk == 0) continue;
        const cuuint64_t dims[4] = {kHeadDim, (cuuint64_t)v.cap, (cuuint64_t)Hkv, (cuuint64_t)v.n_pages};
        const cuuint64_t strides[3] = {(cuuint64_t)v.tok_stride * 2, (cuuint64_t)v.head_stride * 2,
                                       (cuuint64_t)(v.pages ? v.page_stride : v.head_stride) * 2};
        const cuuint32_t box[4] = {kHeadDim / 2, kTreeTile, 1, 1};
        if (!encode_map_once(&maps->k[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, v.k, dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B) ||
            !encode_map_once(&maps->v[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, v.v, dims, strides, box,
                             CU_TENSOR_MAP_SWIZZLE_128B))
            return false;
    }
    return true;
}

// Merge of one (row, query head): the prefix's chunks in order, then the
// node's path from the prefix down.  One thread per dim.
__global__ void __launch_bounds__(kHeadDim)
tree_merge_kernel(const float* __restrict__ q, const __grid_constant__ TreeBatch b, int Hq, int Hkv, float scale,
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
            const float m = __ldcg(part_ml + 4 * (pr0 + c * pstep));
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
            const float* ml = part_ml + 4 * (pr0 + c * pstep);
            L = __fmaf_rn(__fadd_rn(__ldcg(ml + 1), __ldcg(ml + 2)), f, L);
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
    int64_t tiles = 0, n_part = 0;
    for (int i = 0; i < b.n_view; ++i) {
        tiles += (int64_t)((b.view[i].len + kTreeTile - 1) / kTreeTile) * Hkv;
        n_part += (int64_t)b.view[i].n_chunk * b.view[i].n_nodes * Hq;
    }
    float* part_o = (float*)part;
    float* part_ml = part_o + n_part * kHeadDim;
    if (tiles > 0) {
        TreeMaps maps{};
        if (!tree_maps(b, Hkv, &maps)) return cudaErrorInvalidValue;
        const int sms = sm_count();
        if (sms <= 0) return cudaErrorInvalidDevice;
        static std::atomic<bool> done[kMaxDevices];
        cudaError_t e = set_smem_once(tree_chunk_kernel, kTreeSmem, done);
        if (e == cudaSuccess)
            e = launch_pdl_smem(tree_chunk_kernel, dim3((unsigned)std::min<int64_t>(sms, tiles)), dim3(kTreeThreads),
                                kTreeSmem, s, maps, q, b, Hq, Hkv, (int)tiles, scale, part_o, part_ml, scores, lds);
        if (e != cudaSuccess) return e;
        count_launches(1);
    }
    const cudaError_t e =
        launch_pdl(tree_merge_kernel, dim3(Hq, b.n_row), dim3(kHeadDim), s, q, b, Hq, Hkv, scale,
                   (const float*)part_o, (const float*)part_ml, out, scores, lds, stats, out_q, out_d);
    count_launches(1);
    return e;
}

}  // namespace luce
