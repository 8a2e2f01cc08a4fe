// api_cache.cu - the C ABI over a slot's cache: tree attention, the commit of
// an accepted path, eviction (see include/luce.h for the contract).
#include <math.h>
#include <stdio.h>

#include <algorithm>

#include "../../include/luce.h"
#include "api.h"
#include "api_cache.h"
#include "cache.h"
#include "kernels.h"

using namespace luce;

static_assert(LUCE_MAX_TREE == kMaxTree && LUCE_MAX_ROWS == kMaxTree && LUCE_MAX_SEQ == 4, "sizes of the batches");

// ------------------------------------------------------------ ranges

int luce::check_apart(const ByteRange* r, int n, const char* who)
{
    for (int a = 0; a < n; ++a)
        for (int c = 0; c < a; ++c) {
            const bool apart = r[a].hi <= r[c].lo || r[c].hi <= r[a].lo;
            const bool both_read = !r[a].written && !r[c].written;
            const bool in_place = r[a].slot == r[c].slot && r[a].pair && r[a].pair == r[c].pair && r[a].lo == r[c].lo;
            if (apart || both_read || in_place) continue;
            char at[2][24] = {"", ""};  // (-1: no slot's own)
            if (r[a].slot >= 0) snprintf(at[0], sizeof at[0], " of slot %d", r[a].slot);
            if (r[c].slot >= 0) snprintf(at[1], sizeof at[1], " of slot %d", r[c].slot);
            return fail(LUCE_EINVAL, "%s: the %s%s overlaps the %s%s", who, r[a].what, at[0], r[c].what, at[1]);
        }
    return LUCE_OK;
}

static ByteRange range_of(const void* p, int64_t bytes, int slot, const char* what, bool written, int pair = 0)
{
    return ByteRange{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes, slot, what, written, pair};
}

// ------------------------------------------------------------ trees

int luce::tree_path(const int32_t* parent, int n_nodes, TreeRow* rows, int view, int row0, const char* who)
{
    for (int j = 0; j < n_nodes; ++j) {
        const int p = parent ? parent[j] : j - 1;
        REQUIRE(p >= -1 && p < j, LUCE_EINVAL, "%s: view %d node %d has parent %d outside [-1, %d)", who, view, j, p, j);
        TreeRow& r = rows[row0 + j];
        r.view = (uint8_t)view;
        r.node = (uint8_t)j;
        r.n_path = 0;
        if (p >= 0)
            for (; r.n_path < rows[row0 + p].n_path; ++r.n_path) r.path[r.n_path] = rows[row0 + p].path[r.n_path];
        r.path[r.n_path++] = (uint8_t)j;
    }
    return LUCE_OK;
}

int64_t luce::tree_chunks(TreeBatch& b, int Hq, int Hkv)
{
    int64_t part = 0;
    for (int i = 0; i < b.n_view; ++i) {
        TreeView& v = b.view[i];
        v.chunk = tree_chunk_keys(v.len, Hkv);
        v.n_chunk = tree_is_short(v.len) ? 0 : (v.len + v.chunk - 1) / v.chunk;
        v.part0 = part;
        part += (int64_t)v.n_chunk * v.n_nodes * Hq;
    }
    b.n_short = b.n_long = 0;
    for (int r = 0; r < b.n_row; ++r)
        if (b.view[b.row[r].view].n_chunk == 0) b.short_row[b.n_short++] = (uint8_t)r;
        else b.long_row[b.n_long++] = (uint8_t)r;
    return part;
}

size_t luce_tree_attn_workspace_size(int n_rows, int Hq, int Hkv, int D, int max_len)
{
    if (n_rows < 1 || n_rows > LUCE_MAX_ROWS || Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 8 || Hkv > 4096 ||
        D != LUCE_HEAD_DIM || max_len < 0 || max_len > LUCE_MAX_KEYS)
        return 0;
    return std::max<size_t>(256, tree_part_bytes((int64_t)tree_max_chunks(max_len, Hkv) * n_rows * Hq));
}

static int check_tree_call(const float* q, const void* views, int n_seq, int Hq, int Hkv, int D, float scale,
                           const float* out, const float* scores, int64_t lds, const float* stats, const void* ws,
                           const char* who)
{
    REQUIRE(q && out && ws && views, LUCE_EINVAL, "%s: null q/out/ws/views", who);
    REQUIRE(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0, LUCE_EINVAL, "%s: Hq=%d must be a multiple of Hkv=%d", who, Hq,
            Hkv);
    REQUIRE(Hq / Hkv <= 8, LUCE_EUNSUPPORTED, "%s: group size %d > 8", who, Hq / Hkv);
    REQUIRE(Hkv <= 4096, LUCE_EUNSUPPORTED, "%s: %d KV heads > 4096", who, Hkv);
    REQUIRE(D == LUCE_HEAD_DIM, LUCE_EUNSUPPORTED, "%s: head_dim %d (only %d)", who, D, LUCE_HEAD_DIM);
    REQUIRE(isfinite(scale), LUCE_EINVAL, "%s: scale must be finite", who);
    REQUIRE(aligned(q, 16) && aligned(out, 4) && aligned(stats, 8) && aligned(ws, 256), LUCE_EINVAL,
            "%s: q must be 16-byte, stats 8-byte, ws 256-byte aligned", who);
    REQUIRE(!scores || (aligned(scores, 16) && lds >= 1 && lds % 4 == 0), LUCE_EINVAL,
            "%s: scores must be 16-byte aligned and lds=%lld a positive multiple of 4", who, (long long)lds);
    REQUIRE(n_seq >= 1 && n_seq <= LUCE_MAX_SEQ, LUCE_EINVAL,
            "%s: n_seq=%d outside 1..%d (more than %d sequences are refused)", who, n_seq, LUCE_MAX_SEQ,
            LUCE_MAX_SEQ);
    return LUCE_OK;
}

// A view's sizes and rows, entered into the batch.
static int add_tree_view(TreeBatch& b, int s, int len, int n_nodes, int row0, const int32_t* parent, bool* covered,
                         const float* scores, int64_t lds, const char* who)
{
    REQUIRE(n_nodes >= 1 && n_nodes <= LUCE_MAX_TREE, LUCE_EINVAL, "%s: view %d has %d nodes (1..%d)", who, s, n_nodes,
            LUCE_MAX_TREE);
    REQUIRE(len >= 0, LUCE_EINVAL, "%s: view %d len=%d < 0", who, s, len);
    REQUIRE(len <= LUCE_MAX_KEYS - n_nodes, LUCE_EUNSUPPORTED, "%s: view %d has %d + %d keys (at most %d)", who, s, len,
            n_nodes, LUCE_MAX_KEYS);
    REQUIRE(!scores || lds >= len + n_nodes, LUCE_EINVAL, "%s: lds=%lld < the %d keys of view %d", who, (long long)lds,
            len + n_nodes, s);
    REQUIRE(row0 >= 0 && row0 <= LUCE_MAX_ROWS - n_nodes, LUCE_EINVAL, "%s: view %d rows out of range", who, s);
    for (int j = 0; j < n_nodes; ++j) {
        REQUIRE(!covered[row0 + j], LUCE_EINVAL, "%s: row %d claimed twice", who, row0 + j);
        covered[row0 + j] = true;
    }
    const int rc = tree_path(parent, n_nodes, b.row, s, row0, who);
    if (rc) return rc;
    b.view[s].len = len;
    b.view[s].n_nodes = n_nodes;
    b.view[s].row0 = row0;
    b.n_view = s + 1;
    b.n_row = std::max(b.n_row, row0 + n_nodes);
    return LUCE_OK;
}

// What a view's rows read.  (Tiles reach further, but use nothing of it.)
static void add_view_ranges(ByteRange* r, int* nr, const TreeView& v, int s, int Hkv)
{
    const int64_t keys = v.len + v.n_nodes;
    const int64_t elems = v.pages ? v.page_stride * (v.n_pages - 1) + v.head_stride * Hkv
                                  : v.head_stride * (Hkv - 1) + v.tok_stride * (keys - 1) + LUCE_HEAD_DIM;
    r[(*nr)++] = range_of(v.k, elems * 2, s, "K", false);
    r[(*nr)++] = range_of(v.v, elems * 2, s, "V", false);
    if (v.pages) r[(*nr)++] = range_of(v.pages, (keys + LUCE_PAGE_KEYS - 1) / LUCE_PAGE_KEYS * 4, s, "table", false);
}

static int run_tree(TreeBatch& b, const bool* covered, const float* q, int Hq, int Hkv, float scale, float* out,
                    float* scores, int64_t lds, float* stats, void* ws, size_t ws_bytes, void* stream, const char* who)
{
    for (int r = 0; r < b.n_row; ++r) REQUIRE(covered[r], LUCE_EINVAL, "%s: row %d belongs to no view", who, r);
    const size_t need = std::max<size_t>(256, tree_part_bytes(tree_chunks(b, Hq, Hkv)));
    REQUIRE(ws_bytes >= need, LUCE_ENOSPACE, "%s: workspace %zu bytes < %zu needed", who, ws_bytes, need);
    ByteRange r[3 * LUCE_MAX_SEQ + 5];
    int nr = 0;
    const int64_t heads = (int64_t)b.n_row * Hq;
    for (int s = 0; s < b.n_view; ++s) add_view_ranges(r, &nr, b.view[s], s, Hkv);
    // (a row's q is read before its out is written)
    r[nr++] = range_of(q, heads * LUCE_HEAD_DIM * 4, -1, "q", false, 1);
    r[nr++] = range_of(out, heads * LUCE_HEAD_DIM * 4, -1, "out", true, 1);
    if (scores) r[nr++] = range_of(scores, heads * lds * 4, -1, "scores", true);
    if (stats) r[nr++] = range_of(stats, heads * 8, -1, "stats", true);
    r[nr++] = range_of(ws, need, -1, "workspace", true);
    const int rc = check_apart(r, nr, who);
    if (rc) return rc;
    return cuda_status(launch_tree_attention(q, b, Hq, Hkv, scale, ws, out, scores, lds, stats, nullptr, nullptr,
                                             (cudaStream_t)stream),
                       who);
}

int luce_tree_attn(const float* q, const luce_treeview* views, int n_seq, int Hq, int Hkv, int D, float scale,
                   float* out, float* scores, int64_t lds, float* stats, void* ws, size_t ws_bytes, void* stream)
{
    const char* who = "tree_attn";
    int rc = check_tree_call(q, views, n_seq, Hq, Hkv, D, scale, out, scores, lds, stats, ws, who);
    if (rc) return rc;
    TreeBatch b{};
    bool covered[LUCE_MAX_ROWS] = {};
    for (int s = 0; s < n_seq; ++s) {
        const luce_treeview& v = views[s];
        REQUIRE(v.k && v.v && aligned(v.k, 16) && aligned(v.v, 16), LUCE_EINVAL,
                "%s: view %d cache null or not 16-byte aligned", who, s);
        if ((rc = add_tree_view(b, s, v.len, v.n_nodes, v.row0, v.parent, covered, scores, lds, who))) return rc;
        REQUIRE(v.len + v.n_nodes <= v.cap, LUCE_EINVAL, "%s: view %d len=%d + nodes=%d exceeds cap=%d", who, s, v.len,
                v.n_nodes, v.cap);
        REQUIRE(v.tok_stride >= D && v.tok_stride % 8 == 0 && v.tok_stride < ((int64_t)1 << 32), LUCE_EINVAL,
                "%s: view %d tok_stride must be a multiple of 8, at least D", who, s);
        REQUIRE(Hkv == 1 || (v.head_stride % 8 == 0 && v.head_stride >= (int64_t)v.cap * v.tok_stride &&
                             v.head_stride < ((int64_t)1 << 38)),
                LUCE_EINVAL, "%s: view %d head_stride must be a multiple of 8 and keep the heads apart", who, s);
        REQUIRE((int64_t)v.cap * v.tok_stride < ((int64_t)1 << 38), LUCE_EINVAL, "%s: view %d spans 2^38 elements or more",
                who, s);
        TreeView& t = b.view[s];
        t.k = reinterpret_cast<const __half*>(v.k);
        t.v = reinterpret_cast<const __half*>(v.v);
        t.tok_stride = v.tok_stride;
        t.head_stride = Hkv == 1 ? (int64_t)v.cap * v.tok_stride : v.head_stride;
        t.page_stride = t.head_stride * Hkv;
        t.n_pages = 1;
        t.cap = v.cap;
    }
    return run_tree(b, covered, q, Hq, Hkv, scale, out, scores, lds, stats, ws, ws_bytes, stream, who);
}

int luce_tree_attn_paged(const float* q, const luce_pagedtreeview* views, int n_seq, int Hq, int Hkv, int D,
                         float scale, float* out, float* scores, int64_t lds, float* stats, void* ws, size_t ws_bytes,
                         void* stream)
{
    const char* who = "tree_attn_paged";
    int rc = check_tree_call(q, views, n_seq, Hq, Hkv, D, scale, out, scores, lds, stats, ws, who);
    if (rc) return rc;
    TreeBatch b{};
    bool covered[LUCE_MAX_ROWS] = {};
    for (int s = 0; s < n_seq; ++s) {
        const luce_pagedtreeview& v = views[s];
        REQUIRE(v.k_pool && v.v_pool && aligned(v.k_pool, 16) && aligned(v.v_pool, 16), LUCE_EINVAL,
                "%s: view %d pool null or not 16-byte aligned", who, s);
        REQUIRE(v.table && aligned(v.table, 4), LUCE_EINVAL, "%s: view %d table null or misaligned", who, s);
        REQUIRE(v.n_pages >= 1, LUCE_EINVAL, "%s: view %d n_pages=%d", who, s, v.n_pages);
        if ((rc = add_tree_view(b, s, v.len, v.n_nodes, v.row0, v.parent, covered, scores, lds, who))) return rc;
        TreeView& t = b.view[s];
        t.k = reinterpret_cast<const __half*>(v.k_pool);
        t.v = reinterpret_cast<const __half*>(v.v_pool);
        t.pages = v.table;
        t.n_pages = v.n_pages;
        t.cap = LUCE_PAGE_KEYS;
        t.tok_stride = D;
        t.head_stride = (int64_t)LUCE_PAGE_KEYS * D;
        const int64_t page = t.head_stride * Hkv;
        REQUIRE(v.page_stride == 0 || (v.page_stride >= page && v.page_stride % 8 == 0 && v.page_stride < ((int64_t)1 << 38)),
                LUCE_EINVAL, "%s: view %d page_stride must be a multiple of 8 and keep the pages apart", who, s);
        t.page_stride = v.page_stride ? v.page_stride : page;
    }
    return run_tree(b, covered, q, Hq, Hkv, scale, out, scores, lds, stats, ws, ws_bytes, stream, who);
}

// ------------------------------------------------------------ pools

static const char* const kPoolK = "K pool";
static const char* const kPoolV = "V pool";

// Slots may share a pool, each with its own rows; pools that are not one overlap
// nothing.
static void add_pool(ByteRange* r, int* nr, const void* p, int64_t bytes, int slot, const char* what)
{
    const ByteRange n = range_of(p, bytes, slot, what, true);
    for (int i = 0; i < *nr; ++i)
        if (r[i].what == what && r[i].lo == n.lo) {
            r[i].hi = std::max(r[i].hi, n.hi);
            return;
        }
    r[(*nr)++] = n;
}

static int check_layers(int n_seq, int n_layers, int Hkv, int D, const void* slots, const char* who)
{
    REQUIRE(slots, LUCE_EINVAL, "%s: null slots", who);
    REQUIRE(n_seq >= 1 && n_seq <= LUCE_MAX_SEQ, LUCE_EINVAL, "%s: n_seq=%d outside 1..%d", who, n_seq, LUCE_MAX_SEQ);
    REQUIRE(D == LUCE_HEAD_DIM, LUCE_EUNSUPPORTED, "%s: head_dim %d (only %d)", who, D, LUCE_HEAD_DIM);
    REQUIRE(n_layers >= 1 && Hkv >= 1 && (int64_t)n_layers * Hkv <= (1 << 20), LUCE_EINVAL,
            "%s: n_layers=%d and Hkv=%d must be positive, %d heads at most in all", who, n_layers, Hkv, 1 << 20);
    return LUCE_OK;
}

// ------------------------------------------------------------ commit

namespace {

// What a commit's flat and paged slots share, entered into the batch.
struct CommitArgs {
    int len, cap, n_path, row0;
    const int32_t* path;
    float* acc;
    int32_t* pos;
    int pos0;
};

}  // namespace

static int check_commit_call(int n_seq, int n_layers, int Hq, int Hkv, int D, const void* slots, const char* who)
{
    const int rc = check_layers(n_seq, n_layers, Hkv, D, slots, who);
    if (rc) return rc;
    REQUIRE(Hq >= Hkv && Hq % Hkv == 0, LUCE_EINVAL, "%s: Hq=%d must be a multiple of Hkv=%d", who, Hq, Hkv);
    REQUIRE(Hq / Hkv <= 8, LUCE_EUNSUPPORTED, "%s: group size %d > 8", who, Hq / Hkv);
    return LUCE_OK;
}

static int add_commit_slot(CommitSlot& o, const CommitArgs& c, int s, int64_t heads, const float* scores, int n_rows,
                           int64_t lds, const float* stats, ByteRange* r, int* nr, bool* any_acc, const char* who)
{
    REQUIRE(aligned(c.acc, 4) && aligned(c.pos, 4), LUCE_EINVAL, "%s: slot %d acc or pos misaligned", who, s);
    REQUIRE(c.n_path >= 0 && c.n_path <= LUCE_MAX_TREE, LUCE_EINVAL, "%s: slot %d n_path=%d outside 0..%d", who, s,
            c.n_path, LUCE_MAX_TREE);
    REQUIRE(c.n_path == 0 || c.path, LUCE_EINVAL, "%s: slot %d has a null path", who, s);
    REQUIRE(c.len >= 0 && c.cap >= 1 && c.len <= c.cap, LUCE_EINVAL, "%s: slot %d len=%d outside [0, cap=%d]", who, s,
            c.len, c.cap);
    REQUIRE(c.len <= LUCE_MAX_KEYS - c.n_path, LUCE_EUNSUPPORTED, "%s: slot %d would hold %d + %d keys (at most %d)", who, s,
            c.len, c.n_path, LUCE_MAX_KEYS);
    REQUIRE(c.pos0 >= 0 && c.pos0 <= INT32_MAX - LUCE_MAX_TREE, LUCE_EINVAL, "%s: slot %d pos0=%d", who, s, c.pos0);
    int last = -1;
    for (int i = 0; i < c.n_path; ++i) {
        REQUIRE(c.path[i] > last && c.path[i] < LUCE_MAX_TREE && (int64_t)c.len + c.path[i] < c.cap, LUCE_EINVAL,
                "%s: slot %d path[%d]=%d must ascend, below %d and within the cache", who, s, i, c.path[i],
                LUCE_MAX_TREE);
        last = c.path[i];
        o.path[i] = (uint8_t)last;
    }
    if (c.acc && c.n_path > 0) {
        *any_acc = true;
        REQUIRE(scores && stats, LUCE_EINVAL, "%s: slot %d has acc, but scores or stats is null", who, s);
        REQUIRE(c.row0 >= 0 && (int64_t)c.row0 + last < n_rows, LUCE_EINVAL,
                "%s: slot %d rows %d + %d outside the %d score rows", who, s, c.row0, last, n_rows);
        REQUIRE(lds > (int64_t)c.len + last, LUCE_EINVAL, "%s: lds=%lld does not reach slot %d's key %d", who,
                (long long)lds, s, c.len + last);
    }
    o.acc = c.acc;
    o.pos = c.pos;
    o.len = c.len;
    o.cap = c.cap;
    o.row0 = c.row0;
    o.pos0 = c.pos0;
    o.n_path = c.n_path;
    if (c.acc) r[(*nr)++] = range_of(c.acc, heads * c.cap * 4, s, "acc", true);
    if (c.pos) r[(*nr)++] = range_of(c.pos, heads * c.cap * 4, s, "pos", true);
    return LUCE_OK;
}

static int run_commit(const CommitBatch& b, int n_layers, int Hq, int Hkv, const float* scores, int n_rows, int64_t lds,
                      const float* stats, ByteRange* r, int nr, bool any_acc, void* stream, const char* who)
{
    if (any_acc) {
        REQUIRE(n_rows >= 1 && n_rows <= LUCE_MAX_ROWS, LUCE_EINVAL, "%s: n_rows=%d outside 1..%d", who, n_rows,
                LUCE_MAX_ROWS);
        REQUIRE(aligned(scores, 16) && lds % 4 == 0 && lds < ((int64_t)1 << 31) && aligned(stats, 8), LUCE_EINVAL,
                "%s: scores must be 16-byte, stats 8-byte aligned and lds=%lld a multiple of 4", who, (long long)lds);
        r[nr++] = range_of(scores, (int64_t)n_layers * n_rows * Hq * lds * 4, -1, "scores", false);
        r[nr++] = range_of(stats, (int64_t)n_layers * n_rows * Hq * 8, -1, "stats", false);
    }
    const int rc = check_apart(r, nr, who);
    if (rc) return rc;
    bool any = false;
    for (int s = 0; s < b.n_slot; ++s) any = any || b.slot[s].n_path > 0;
    if (!any) return ok();
    return cuda_status(launch_tree_commit(b, n_layers, Hq, Hkv, scores, n_rows, lds, stats, (cudaStream_t)stream), who);
}

int luce_tree_commit(const luce_commit_slot* slots, int n_seq, int n_layers, int Hq, int Hkv, int D,
                     const float* scores, int n_rows, int64_t lds, const float* stats, void* stream)
{
    const char* who = "tree_commit";
    int rc = check_commit_call(n_seq, n_layers, Hq, Hkv, D, slots, who);
    if (rc) return rc;
    CommitBatch b{};
    b.n_slot = n_seq;
    ByteRange r[4 * LUCE_MAX_SEQ + 2];
    int nr = 0;
    bool any_acc = false;
    const int64_t heads = (int64_t)n_layers * Hkv;
    for (int s = 0; s < n_seq; ++s) {
        const luce_commit_slot& c = slots[s];
        REQUIRE(c.k && c.v && aligned(c.k, 16) && aligned(c.v, 16), LUCE_EINVAL,
                "%s: slot %d cache null or not 16-byte aligned", who, s);
        const CommitArgs a{c.len, c.cap, c.n_path, c.row0, c.path, c.acc, c.pos, c.pos0};
        CommitSlot& o = b.slot[s];
        if ((rc = add_commit_slot(o, a, s, heads, scores, n_rows, lds, stats, r, &nr, &any_acc, who))) return rc;
        o.k = reinterpret_cast<__half*>(c.k);
        o.v = reinterpret_cast<__half*>(c.v);
        o.head_step = (int64_t)c.cap * D;
        for (int e = 0; e < 2; ++e) o.span[e] = (int64_t)(c.len / LUCE_PAGE_KEYS + e) * LUCE_PAGE_KEYS * D;
        r[nr++] = range_of(c.k, heads * c.cap * D * 2, s, "K cache", true);
        r[nr++] = range_of(c.v, heads * c.cap * D * 2, s, "V cache", true);
    }
    return run_commit(b, n_layers, Hq, Hkv, scores, n_rows, lds, stats, r, nr, any_acc, stream, who);
}

int luce_tree_commit_paged(const luce_paged_commit_slot* slots, int n_seq, int n_layers, int Hq, int Hkv, int D,
                           const float* scores, int n_rows, int64_t lds, const float* stats, void* stream)
{
    const char* who = "tree_commit_paged";
    int rc = check_commit_call(n_seq, n_layers, Hq, Hkv, D, slots, who);
    if (rc) return rc;
    CommitBatch b{};
    b.n_slot = n_seq;
    ByteRange r[4 * LUCE_MAX_SEQ + 2];
    int nr = 0;
    bool any_acc = false;
    const int64_t heads = (int64_t)n_layers * Hkv, page = heads * LUCE_PAGE_KEYS * D;
    for (int s = 0; s < n_seq; ++s) {
        const luce_paged_commit_slot& c = slots[s];
        REQUIRE(c.k_pool && c.v_pool && aligned(c.k_pool, 16) && aligned(c.v_pool, 16), LUCE_EINVAL,
                "%s: slot %d pool null or not 16-byte aligned", who, s);
        REQUIRE(c.n_pages >= 1 && c.n_table >= 0 && (c.table_host || c.n_path == 0), LUCE_EINVAL,
                "%s: slot %d has no pages or no table", who, s);
        const CommitArgs a{c.len, c.cap, c.n_path, c.row0, c.path, c.acc, c.pos, c.pos0};
        CommitSlot& o = b.slot[s];
        if ((rc = add_commit_slot(o, a, s, heads, scores, n_rows, lds, stats, r, &nr, &any_acc, who))) return rc;
        o.k = reinterpret_cast<__half*>(c.k_pool);
        o.v = reinterpret_cast<__half*>(c.v_pool);
        o.head_step = (int64_t)LUCE_PAGE_KEYS * D;
        add_pool(r, &nr, c.k_pool, page * c.n_pages * 2, s, kPoolK);
        add_pool(r, &nr, c.v_pool, page * c.n_pages * 2, s, kPoolV);
        for (int i = 0; i < c.n_path; ++i)
            for (int to = 0; to < 2; ++to) {
                const int key = c.len + (to ? i : c.path[i]), at = key / LUCE_PAGE_KEYS;
                REQUIRE(at < c.n_table && c.table_host[at] >= 0 && c.table_host[at] < c.n_pages, LUCE_EINVAL,
                        "%s: slot %d key %d has no page in [0, %d)", who, s, key, c.n_pages);
                o.span[at - c.len / LUCE_PAGE_KEYS] = c.table_host[at] * page;
            }
    }
    // a row that one slot writes is no other slot's row
    for (int s = 0; s < n_seq; ++s)
        for (int t = 0; t < n_seq; ++t)
            for (int i = 0; i < b.slot[s].n_path && s != t; ++i)
                for (int j = 0; j < b.slot[t].n_path; ++j) {
                    const CommitSlot &a = b.slot[s], &o = b.slot[t];
                    const int64_t to = a.at(a.len + i);
                    REQUIRE((a.k != o.k && a.v != o.v) || (to != o.at(o.len + j) && to != o.at(o.len + o.path[j])), LUCE_EINVAL,
                            "%s: slots %d and %d share a row", who, s, t);
                }
    return run_commit(b, n_layers, Hq, Hkv, scores, n_rows, lds, stats, r, nr, any_acc, stream, who);
}

// ------------------------------------------------------------ eviction

namespace {

struct EvictArgs {
    const float* acc;
    const int32_t* pos;
    float* acc_out;
    int32_t* pos_out;
    int len, cap, budget, sinks, recent, next_pos;
};

}  // namespace

static int add_evict_slot(EvictSlot& o, const EvictArgs& e, int s, int64_t heads, ByteRange* r, int* nr, bool* any,
                          const char* who)
{
    REQUIRE(e.acc && e.pos && e.acc_out && e.pos_out && aligned(e.acc, 4) && aligned(e.pos, 4) && aligned(e.acc_out, 4) &&
                aligned(e.pos_out, 4),
            LUCE_EINVAL, "%s: slot %d acc or pos null or misaligned", who, s);
    REQUIRE(e.cap >= 1 && e.len >= 0 && e.len <= e.cap, LUCE_EINVAL, "%s: slot %d len=%d outside [0, cap=%d]", who, s, e.len,
            e.cap);
    REQUIRE(e.len <= LUCE_MAX_KEYS, LUCE_EUNSUPPORTED, "%s: slot %d has %d keys (at most %d)", who, s, e.len,
            LUCE_MAX_KEYS);
    REQUIRE(e.budget >= 1 && e.sinks >= 0 && e.recent >= 0 && (int64_t)e.sinks + e.recent <= e.budget, LUCE_EINVAL,
            "%s: slot %d needs 1 <= budget and sinks + recent <= budget (%d, %d, %d)", who, s, e.budget, e.sinks,
            e.recent);
    REQUIRE(e.next_pos >= 0, LUCE_EINVAL, "%s: slot %d next_pos=%d", who, s, e.next_pos);
    o.acc = e.acc;
    o.pos = e.pos;
    o.acc_out = e.acc_out;
    o.pos_out = e.pos_out;
    o.len = e.len;
    o.cap = e.cap;
    o.budget = e.budget;
    o.sinks = e.sinks;
    o.recent = e.recent;
    o.next_pos = e.next_pos;
    const bool copies = e.acc_out != e.acc || e.pos_out != e.pos;
    *any = *any || e.len > e.budget || (copies && e.len > 0);
    r[(*nr)++] = range_of(e.acc, heads * e.cap * 4, s, "acc", false, 1);
    r[(*nr)++] = range_of(e.pos, heads * e.cap * 4, s, "pos", false, 2);
    r[(*nr)++] = range_of(e.acc_out, heads * e.cap * 4, s, "acc_out", true, 1);
    r[(*nr)++] = range_of(e.pos_out, heads * e.cap * 4, s, "pos_out", true, 2);
    return LUCE_OK;
}

int luce_kv_evict(const luce_evict_slot* slots, int n_seq, int n_layers, int Hkv, int D, void* stream)
{
    const char* who = "kv_evict";
    int rc = check_layers(n_seq, n_layers, Hkv, D, slots, who);
    if (rc) return rc;
    EvictBatch b{};
    b.n_slot = n_seq;
    ByteRange r[6 * LUCE_MAX_SEQ];
    int nr = 0;
    bool any = false;
    const int64_t heads = (int64_t)n_layers * Hkv;
    for (int s = 0; s < n_seq; ++s) {
        const luce_evict_slot& e = slots[s];
        REQUIRE(e.k && e.v && aligned(e.k, 16) && aligned(e.v, 16), LUCE_EINVAL,
                "%s: slot %d cache null or not 16-byte aligned", who, s);
        const EvictArgs a{e.acc, e.pos, e.acc_out, e.pos_out, e.len, e.cap, e.budget, e.sinks, e.recent, e.next_pos};
        EvictSlot& o = b.slot[s];
        if ((rc = add_evict_slot(o, a, s, heads, r, &nr, &any, who))) return rc;
        o.k = reinterpret_cast<__half*>(e.k);
        o.v = reinterpret_cast<__half*>(e.v);
        o.head_step = (int64_t)e.cap * D;
        r[nr++] = range_of(e.k, heads * e.cap * D * 2, s, "K cache", true);
        r[nr++] = range_of(e.v, heads * e.cap * D * 2, s, "V cache", true);
    }
    if ((rc = check_apart(r, nr, who))) return rc;
    if (!any) return ok();
    return cuda_status(launch_kv_evict(b, n_layers, Hkv, (cudaStream_t)stream), who);
}

int luce_kv_evict_paged(const luce_paged_evict_slot* slots, int n_seq, int n_layers, int Hkv, int D, void* stream)
{
    const char* who = "kv_evict_paged";
    int rc = check_layers(n_seq, n_layers, Hkv, D, slots, who);
    if (rc) return rc;
    EvictBatch b{};
    b.n_slot = n_seq;
    ByteRange r[6 * LUCE_MAX_SEQ];
    int nr = 0;
    bool any = false;
    const int64_t heads = (int64_t)n_layers * Hkv;
    for (int s = 0; s < n_seq; ++s) {
        const luce_paged_evict_slot& e = slots[s];
        REQUIRE(e.k_pool && e.v_pool && aligned(e.k_pool, 16) && aligned(e.v_pool, 16), LUCE_EINVAL,
                "%s: slot %d pool null or not 16-byte aligned", who, s);
        REQUIRE(e.table && aligned(e.table, 4) && e.n_pages >= 1, LUCE_EINVAL, "%s: slot %d has no pages or no table", who,
                s);
        const EvictArgs a{e.acc, e.pos, e.acc_out, e.pos_out, e.len, e.cap, e.budget, e.sinks, e.recent, e.next_pos};
        EvictSlot& o = b.slot[s];
        if ((rc = add_evict_slot(o, a, s, heads, r, &nr, &any, who))) return rc;
        o.k = reinterpret_cast<__half*>(e.k_pool);
        o.v = reinterpret_cast<__half*>(e.v_pool);
        o.pages = e.table;
        o.n_pages = e.n_pages;
        o.head_step = (int64_t)LUCE_PAGE_KEYS * D;
        REQUIRE(heads * LUCE_PAGE_KEYS * e.n_pages < ((int64_t)1 << 31), LUCE_EUNSUPPORTED,
                "%s: slot %d pool has 2^31 rows or more", who, s);
        o.page_rows = (int32_t)(heads * LUCE_PAGE_KEYS);
        add_pool(r, &nr, e.k_pool, heads * LUCE_PAGE_KEYS * D * 2 * e.n_pages, s, kPoolK);
        add_pool(r, &nr, e.v_pool, heads * LUCE_PAGE_KEYS * D * 2 * e.n_pages, s, kPoolV);
    }
    if ((rc = check_apart(r, nr, who))) return rc;
    if (!any) return ok();
    return cuda_status(launch_kv_evict(b, n_layers, Hkv, (cudaStream_t)stream), who);
}
