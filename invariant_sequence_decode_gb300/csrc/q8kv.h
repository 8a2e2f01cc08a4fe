// q8kv.h - launchers of the kernels over a slot's cache in 8 bits: attention,
// the sealing of whole blocks, the pass that norms, rotates and appends
// (internal).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "cache.h"
#include "kernels.h"

namespace luce {

constexpr int kQ8Block = 32;        // tokens that share a scale
constexpr int kQ8Page = 128;        // tokens of a page
constexpr int kQ8PageBytes = kQ8Page * 128;  // codes of a page's K (or V) of one head
constexpr int kQ8PageScales = 8;    // scales of a page and head: K's four blocks, V's four
constexpr int kQ8MaxTail = 112;     // f16 keys between the sealed blocks and the tree

// A slot for one layer: sealed keys in pages of codes, behind them the f16 tail
// and the tree.  Page p's codes of KV head g start at p * page_stride + g *
// kQ8PageBytes, its scales at p * scale_stride + g * kQ8PageScales.
struct Q8View {
    const int8_t* k_codes;   // [128 keys][128 dims]
    const int8_t* v_codes;   // [128 dims][128 keys]
    const float* scales;
    const int32_t* table;    // page of each 128-key span; nullptr: page i is span i's
    const __half* k;         // tail: element d of row i of KV head g at g*head_stride + i*tok_stride + d
    const __half* v;
    int64_t page_stride;
    int64_t scale_stride;
    int64_t head_stride;
    int64_t tok_stride;
    int64_t part0;           // the view's first row of partial results
    int32_t n_pages;
    int32_t sealed;          // keys in whole blocks
    int32_t tail;            // f16 keys of the prefix behind them
    int32_t n_nodes;
    int32_t row0;
    int32_t window;          // 0: none
    int32_t sinks;
    // 128-key tiles that some row may see: the first `front` and those from `back` on
    int32_t front, back, n_tile;
    int32_t chunk;           // tiles of a chunk
    int32_t n_chunk;
};

struct Q8Batch {
    Q8View view[4];
    TreeRow row[kMaxTree];
    int32_t n_view;
    int32_t n_row;
    uint8_t order[4];  // the views, those with the longest chunks first
};

// Cuts the views' tiles into chunks; returns the rows of partial results.
int64_t q8kv_chunks(Q8Batch& b, int Hq, int Hkv);

// The most chunks of a view with at most max_sealed keys in blocks.
int q8kv_max_chunks(int max_sealed, int Hkv);

// Bytes of n_part rows of partial results.
size_t q8kv_part_bytes(int64_t n_part);

// out [T][Hq][128].
cudaError_t launch_q8kv_attention(const float* q, const Q8Batch& b, int Hq, int Hkv, float scale, void* part, float* out,
                                  cudaStream_t s);

// Bounded waits of that attention that expired on the current device; one that does.
cudaError_t read_q8kv_wait_timeouts(uint32_t* count, bool reset);
cudaError_t launch_q8kv_wait_expiry(uint64_t limit_ns, cudaStream_t s);

// A slot whose tail's whole blocks are sealed, in every (layer, KV head) lh: row
// i of the tail is at (lh * cap + i) * 128, a page's codes at (page * heads + lh) *
// kQ8PageBytes, its scales at (page * heads + lh) * kQ8PageScales.
struct Q8SealSlot {
    __half* k;
    __half* v;
    int8_t* k_codes;
    int8_t* v_codes;
    float* scales;
    const int32_t* table;    // nullptr: page i is span i's
    int32_t n_pages;
    int32_t n;               // rows of the tail
    int32_t cap;
    int32_t sealed;
};
struct Q8SealBatch {
    Q8SealSlot slot[4];
    int32_t n_slot;
};
cudaError_t launch_q8kv_seal(const Q8SealBatch& b, int n_layers, int Hkv, cudaStream_t s);

// Rows row0 .. row0 + n - 1 of a projection go to positions at0 .. of a cache.
struct AppendView {
    __half* k;
    __half* v;
    int64_t head_stride;
    int64_t tok_stride;
    int32_t row0;
    int32_t n;
    int32_t at0;
};
struct AppendViews {
    AppendView view[4];
    int32_t n_view;
};
// The axis of each of the 64 pairs, two bits each.
struct PairAxes {
    uint32_t bits[4];
};
cudaError_t launch_qk_norm_rope(const float* qkv, int64_t ld, int T, int Hq, int Hkv, const AppendViews& views,
                                const float* q_gamma, const float* k_gamma, float eps, const int32_t* pos,
                                const PairAxes& axes, const RopeFreq& f, float* q, cudaStream_t s);

}  // namespace luce
