// api_cache.h - checks of the cache entry points that the decode step shares.
#pragma once

#include <stdint.h>

#include "../../include/luce.h"
#include "cache.h"
#include "q8kv.h"

namespace luce {

// The paths of a tree's nodes, entered into rows[row0 ..]; LUCE_OK or the
// refusal.  parent: nullptr for a chain.
int tree_path(const int32_t* parent, int n_nodes, TreeRow* rows, int view, int row0, const char* who);

// Cuts the views' prefixes into chunks and tells their rows apart by it;
// returns the rows of partial results.
int64_t tree_chunks(TreeBatch& b, int Hq, int Hkv);

// A byte range that a call reads or writes.  Two that overlap are refused
// unless both are read, or they are the same slot's input and output of one
// non-zero pair, starting at the same byte.
struct ByteRange {
    uintptr_t lo, hi;
    int slot;
    const char* what;
    bool written;
    int pair;
};
int check_apart(const ByteRange* r, int n, const char* who);

static inline ByteRange range_of(const void* p, int64_t bytes, int slot, const char* what, bool written, int pair = 0)
{
    return ByteRange{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, slot, what, written, pair};
}

// Slots may share a pool, each with its own rows; pools that are not one overlap
// nothing.
void add_pool(ByteRange* r, int* nr, const void* p, int64_t bytes, int slot, const char* what);

// Sizes of an entry point over the caches of every layer.
int check_layers(int n_seq, int n_layers, int Hkv, int D, const void* slots, const char* who);

// A view of a cache in 8 bits, checked and entered into the batch; covered: the
// rows that earlier views claimed.
int add_q8kv_view(Q8Batch& b, int s, const luce_q8kv_view& v, int Hkv, bool* covered, const char* who);

}  // namespace luce
