// cache.h - launchers of the kernels over a slot's cache: tree attention, the
// commit of an accepted path, eviction (internal).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace luce {

#ifdef __CUDACC__
// Loads of what an earlier kernel may still be writing when this one starts:
// none may move ahead of the wait for it (pdl_wait).  A load through a const
// __restrict__ pointer, __ldg or __ldcg may be, as what it reads counts as
// constant for the kernel's whole life; these keep their place.
__device__ __forceinline__ float4 ld_placed_f4(const void* p)
{
    float4 r;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "l"(p) : "memory");
    return r;
}
// The same past L1: data that other kernels wrote and that is read once.
__device__ __forceinline__ float4 ld_placed_cg_f4(const void* p)
{
    float4 r;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
// The same, first to leave the caches.
__device__ __forceinline__ float4 ld_placed_cs_f4(const void* p)
{
    float4 r;
    asm volatile("ld.global.cs.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}
__device__ __forceinline__ float2 ld_placed_f2(const void* p)
{
    float2 r;
    asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(r.x), "=f"(r.y) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ float ld_placed_f(const void* p)
{
    float r;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(r) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ int ld_placed_i(const void* p)
{
    int r;
    asm volatile("ld.global.s32 %0, [%1];" : "=r"(r) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ uint2 ld_placed_u2(const void* p)
{
    uint2 r;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ uint4 ld_placed_cs_u4(const void* p)
{
    uint4 r;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ uint4 ld_placed_u4(const void* p)
{
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}
#endif

constexpr int kMaxTree = 16;  // nodes of a slot's tree, and rows of a call

// A slot's tree over its cache for one layer.  Flat cache (pages == nullptr):
// element d of key j of KV head g is k[g*head_stride + j*tok_stride + d].
// Paged cache: key j lives in page pages[j / 128], page p at k + p*page_stride;
// an entry outside [0, n_pages) names no page.
struct TreeView {
    const __half* k;
    const __half* v;
    const int32_t* pages;
    int64_t head_stride;
    int64_t tok_stride;
    int64_t page_stride;
    int64_t part0;  // the view's first row of partial results
    int32_t n_pages;
    int32_t cap;
    int32_t len;
    int32_t n_nodes;
    int32_t row0;
    int32_t chunk;    // keys of a chunk: tree_chunk_keys(len, Hkv)
    int32_t n_chunk;  // chunks of the prefix; 0: it is short
};

// A row's node: its path from the prefix (ascending, the node itself last).
struct TreeRow {
    uint8_t view;
    uint8_t node;
    uint8_t n_path;
    uint8_t path[kMaxTree];
};

struct TreeBatch {
    TreeView view[4];
    TreeRow row[kMaxTree];
    int32_t n_view;
    int32_t n_row;
    int32_t n_short, n_long;  // rows whose prefix is short, or cut into chunks
    uint8_t short_row[kMaxTree], long_row[kMaxTree];
};

// Whether a prefix is taken whole rather than cut into chunks.
bool tree_is_short(int len);

// Keys of a chunk of a prefix of len keys: a function of len and the model's KV
// heads alone, so that a row's sums are cut the same way whatever else is in
// the call.
int tree_chunk_keys(int len, int Hkv);

// The most chunks of a prefix of at most max_len keys.
int tree_max_chunks(int max_len, int Hkv);

// Bytes of partial results of n_part rows (view chunks x KV heads x the rows
// of a KV head).
size_t tree_part_bytes(int64_t n_part);

// out [T][Hq][128]; scores [T][Hq][lds] and stats [T][Hq][2] nullable; out_q,
// out_d (nullable): out's q8_0 codes and scales.
cudaError_t launch_tree_attention(const float* q, const TreeBatch& b, int Hq, int Hkv, float scale, void* part,
                                  float* out, float* scores, int64_t lds, float* stats, int8_t* out_q, float* out_d,
                                  cudaStream_t s);

// One wait of limit_ns on a barrier that nothing completes, counted as the tree attention's.
cudaError_t launch_tree_wait_expiry(uint64_t limit_ns, cudaStream_t s);

// Bounded waits of the tree attention that expired on the current device.
cudaError_t read_tree_wait_timeouts(uint32_t* count, bool reset);

// In each (layer, KV head) lh, row at(len + path[i]) moves to row at(len + i), in
// elements from k + lh * head_step and v + lh * head_step.
struct CommitSlot {
    __half* k;
    __half* v;
    float* acc;
    int32_t* pos;
    int64_t head_step;
    int64_t span[2];  // rows of the 128 keys that hold key len, and of the next 128, in elements
    int32_t len;
    int32_t cap;
    int32_t row0;
    int32_t pos0;
    int32_t n_path;
    uint8_t path[kMaxTree];

    // key's row of a head: nodes lie less than 128 keys behind len
    __host__ __device__ int64_t at(int key) const { return span[(key >> 7) - (len >> 7)] + (int64_t)(key & 127) * 128; }
};
struct CommitBatch {
    CommitSlot slot[4];
    int32_t n_slot;
};
cudaError_t launch_tree_commit(const CommitBatch& b, int n_layers, int Hq, int Hkv, const float* scores, int n_rows,
                               int64_t lds, const float* stats, cudaStream_t s);

// Key j of (layer, KV head) lh is at lh * head_step + j * 128 elements, or, in
// pages, at lh * head_step + (pages[j / 128] * page_rows + j % 128) * 128.
struct EvictSlot {
    __half* k;
    __half* v;
    const float* acc;
    const int32_t* pos;
    float* acc_out;
    int32_t* pos_out;
    const int32_t* pages;
    int64_t head_step;
    int32_t page_rows;
    int32_t n_pages;
    int32_t len;
    int32_t cap;
    int32_t budget;
    int32_t sinks;
    int32_t recent;
    int32_t next_pos;
};
struct EvictBatch {
    EvictSlot slot[4];
    int32_t n_slot;
};
cudaError_t launch_kv_evict(const EvictBatch& b, int n_layers, int Hkv, cudaStream_t s);

}  // namespace luce
