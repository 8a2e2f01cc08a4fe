// api_cache.h - checks of the cache entry points that the decode step shares.
#pragma once

#include <stdint.h>

#include "cache.h"

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

}  // namespace luce
