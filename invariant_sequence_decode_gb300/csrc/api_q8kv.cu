// api_q8kv.cu - the C ABI over a slot's cache in 8 bits: the pass that norms,
// rotates and appends a projection's rows, sealing, attention (see
// include/luce.h for the contract).
#include <math.h>
#include <stdlib.h>

#include <algorithm>

#include "../../include/luce.h"
#include "api.h"
#include "api_cache.h"
#include "kernels.h"
#include "q8kv.h"

using namespace luce;

static_assert(LUCE_Q8KV_BLOCK == kQ8Block && LUCE_Q8KV_MAX_TAIL == kQ8MaxTail && LUCE_PAGE_KEYS == kQ8Page, "sizes of the cache");

// ------------------------------------------------------------ projection

namespace {

// What a view's rows write of one cache: n rows of D values in each head.
struct CacheRows {
    const __half* at;
    int64_t head_stride, tok_stride;
    int heads, n;
    const char* what;

    ByteRange hull(int slot) const
    {
        return range_of(at, (head_stride * (heads - 1) + tok_stride * (n - 1) + LUCE_HEAD_DIM) * 2, slot, what, true);
    }
};

// Whether two of them share a value.  Slots' caches may lie between one another's heads (slices
// of one pool along its tokens) or rows, so where the strides are alike the rows are compared, not
// what spans them: row (g, i) of a and (h, j) of b lie d + (h - g) head_stride + (j - i) tok_stride
// apart, and as a head's rows fit its stride only the nearest differences can be small.
bool rows_meet(const CacheRows& a, const CacheRows& b)
{
    const ByteRange x = a.hull(0), y = b.hull(0);
    if (x.hi <= y.lo || y.hi <= x.lo) return false;
    if (a.head_stride != b.head_stride || a.tok_stride != b.tok_stride) return true;
    const int64_t d = ((int64_t)(uintptr_t)b.at - (int64_t)(uintptr_t)a.at) / 2;
    const int64_t h0 = a.head_stride ? -d / a.head_stride : 0;
    for (int64_t h = std::max<int64_t>(h0 - 1, 1 - a.heads); h <= std::min<int64_t>(h0 + 1, a.heads - 1); ++h) {
        const int64_t e = d + h * a.head_stride, t0 = -e / a.tok_stride;
        for (int64_t t = std::max<int64_t>(t0 - 1, 1 - a.n); t <= std::min<int64_t>(t0 + 1, b.n - 1); ++t)
            if (std::abs(e + t * a.tok_stride) < LUCE_HEAD_DIM) return true;
    }
    return false;
}

}  // namespace

int luce_qk_norm_rope(const float* qkv, int64_t ld, const luce_seqview* views, int n_seq, int Hq, int Hkv, int D,
                      const float* q_gamma, const float* k_gamma, float eps, const int32_t* pos, int n_axes,
                      const uint8_t* pair_axis, double theta, float* q, void* stream)
{
    const char* who = "qk_norm_rope";
    REQUIRE(qkv && pos && q && views, LUCE_EINVAL, "%s: null qkv/pos/q/views", who);
    REQUIRE(Hkv >= 1 && Hq >= 1 && Hq <= (1 << 16) && Hkv <= (1 << 16), LUCE_EINVAL, "%s: heads %d/%d", who, Hq, Hkv);
    REQUIRE(D == LUCE_HEAD_DIM, LUCE_EUNSUPPORTED, "%s: head_dim %d (only %d)", who, D, LUCE_HEAD_DIM);
    REQUIRE(ld >= (int64_t)(Hq + 2 * Hkv) * D && ld % 4 == 0 && ld <= (1 << 28), LUCE_EINVAL,
            "%s: ld=%lld must be a multiple of 4 that holds %d heads, at most 2^28", who, (long long)ld, Hq + 2 * Hkv);
    REQUIRE(aligned(qkv, 16) && aligned(q, 16) && aligned(q_gamma, 16) && aligned(k_gamma, 16) && aligned(pos, 4), LUCE_EINVAL,
            "%s: qkv, q and the gammas must be 16-byte, pos 4-byte aligned", who);
    REQUIRE(eps >= 0 && isfinite(eps), LUCE_EINVAL, "%s: eps must be finite and >= 0", who);
    REQUIRE(theta > 0 && isfinite(theta), LUCE_EINVAL, "%s: theta must be positive", who);
    REQUIRE(n_axes >= 1 && n_axes <= LUCE_MAX_AXES, LUCE_EINVAL, "%s: n_axes=%d outside 1..%d", who, n_axes, LUCE_MAX_AXES);
    REQUIRE(pair_axis || n_axes == 1, LUCE_EINVAL, "%s: %d axes need pair_axis", who, n_axes);
    REQUIRE(n_seq >= 1 && n_seq <= LUCE_MAX_SEQ, LUCE_EINVAL, "%s: n_seq=%d outside 1..%d (more than %d sequences are refused)",
            who, n_seq, LUCE_MAX_SEQ, LUCE_MAX_SEQ);
    PairAxes axes{};
    for (int i = 0; pair_axis && i < D / 2; ++i) {
        REQUIRE(pair_axis[i] < n_axes, LUCE_EINVAL, "%s: pair %d is on axis %d of %d", who, i, pair_axis[i], n_axes);
        axes.bits[i >> 4] |= (uint32_t)pair_axis[i] << (2 * (i & 15));
    }
    AppendViews to{};
    to.n_view = n_seq;
    int64_t T = 0, rows = 0;
    CacheRows written[2 * LUCE_MAX_SEQ];
    for (int s = 0; s < n_seq; ++s) {
        const luce_seqview& v = views[s];
        REQUIRE(v.k && v.v && aligned(v.k, 16) && aligned(v.v, 16), LUCE_EINVAL, "%s: view %d cache null or not 16-byte aligned",
                who, s);
        REQUIRE(v.n_q >= 1 && v.len >= v.n_q && v.len <= v.cap, LUCE_EINVAL, "%s: view %d needs 1 <= n_q=%d <= len=%d <= cap=%d", who,
                s, v.n_q, v.len, v.cap);
        REQUIRE(v.tok_stride >= D && v.tok_stride % 8 == 0 && v.tok_stride < ((int64_t)1 << 32), LUCE_EINVAL,
                "%s: view %d tok_stride must be a multiple of 8, at least D", who, s);
        REQUIRE((int64_t)v.cap * v.tok_stride < ((int64_t)1 << 38) &&
                    (Hkv == 1 || (v.head_stride % 8 == 0 && v.head_stride >= (int64_t)v.cap * v.tok_stride &&
                                  v.head_stride < ((int64_t)1 << 38))),
                LUCE_EINVAL, "%s: view %d head_stride must be a multiple of 8 and keep the heads apart", who, s);
        REQUIRE(v.row0 >= 0 && v.row0 <= INT32_MAX - v.n_q, LUCE_EINVAL, "%s: view %d rows out of range", who, s);
        for (int e = 0; e < s; ++e)
            REQUIRE(v.row0 >= views[e].row0 + views[e].n_q || views[e].row0 >= v.row0 + v.n_q, LUCE_EINVAL,
                    "%s: views %d and %d claim the same rows", who, e, s);
        T = std::max<int64_t>(T, (int64_t)v.row0 + v.n_q);
        rows += v.n_q;
        AppendView& a = to.view[s];
        a.k = reinterpret_cast<__half*>(v.k);
        a.v = reinterpret_cast<__half*>(v.v);
        a.head_stride = Hkv == 1 ? 0 : v.head_stride;
        a.tok_stride = v.tok_stride;
        a.row0 = v.row0;
        a.n = v.n_q;
        a.at0 = v.len - v.n_q;
        written[2 * s] = CacheRows{a.k + a.at0 * v.tok_stride, a.head_stride, v.tok_stride, Hkv, v.n_q, "K cache"};
        written[2 * s + 1] = CacheRows{a.v + a.at0 * v.tok_stride, a.head_stride, v.tok_stride, Hkv, v.n_q, "V cache"};
        for (int e = 0; e < 2 * s + 2; ++e)
            for (int c = std::max(e + 1, 2 * s); c < 2 * s + 2; ++c)
                REQUIRE(!rows_meet(written[e], written[c]), LUCE_EINVAL, "%s: the %s of slot %d overlaps the %s of slot %d", who,
                        written[c].what, s, written[e].what, e / 2);
    }
    // (rows are apart, so as many of them as the highest number says cover all)
    REQUIRE(rows == T, LUCE_EINVAL, "%s: the views name %lld of %lld rows", who, (long long)rows, (long long)T);
    ByteRange r[5];
    int nr = 0;
    r[nr++] = range_of(qkv, ((T - 1) * ld + (int64_t)(Hq + 2 * Hkv) * D) * 4, -1, "projection", false);
    r[nr++] = range_of(q, T * Hq * D * 4, -1, "q", true);
    r[nr++] = range_of(pos, T * n_axes * 4, -1, "positions", false);
    if (q_gamma) r[nr++] = range_of(q_gamma, D * 4, -1, "q_gamma", false);
    if (k_gamma) r[nr++] = range_of(k_gamma, D * 4, -1, "k_gamma", false);
    int rc = check_apart(r, nr, who);
    for (int c = 0; c < 2 * n_seq && !rc; ++c) {
        const ByteRange h = written[c].hull(c / 2);
        for (int i = 0; i < nr && !rc; ++i) {
            if (h.hi <= r[i].lo || r[i].hi <= h.lo) continue;
            const ByteRange two[2] = {r[i], h};
            rc = check_apart(two, 2, who);
        }
    }
    if (rc) return rc;
    return cuda_status(launch_qk_norm_rope(qkv, ld, (int)T, Hq, Hkv, to, q_gamma, k_gamma, eps, pos, axes, rope_freq(theta), q,
                                           (cudaStream_t)stream),
                       who);
}

// ------------------------------------------------------------ sealing

int luce_q8kv_seal(const luce_q8kv_slot* slots, int n_seq, int n_layers, int Hkv, int D, void* stream)
{
    const char* who = "q8kv_seal";
    int rc = check_layers(n_seq, n_layers, Hkv, D, slots, who);
    if (rc) return rc;
    Q8SealBatch b{};
    b.n_slot = n_seq;
    ByteRange r[6 * LUCE_MAX_SEQ];
    int nr = 0, units = 0;
    const int64_t heads = (int64_t)n_layers * Hkv;
    for (int s = 0; s < n_seq; ++s) {
        const luce_q8kv_slot& c = slots[s];
        REQUIRE(c.k && c.v && aligned(c.k, 32) && aligned(c.v, 32), LUCE_EINVAL, "%s: slot %d tail null or not 32-byte aligned", who,
                s);
        REQUIRE(c.cap >= 1 && c.len >= 0 && c.len <= c.cap, LUCE_EINVAL, "%s: slot %d len=%d outside [0, cap=%d]", who, s, c.len,
                c.cap);
        REQUIRE(c.sealed >= 0 && c.sealed % LUCE_Q8KV_BLOCK == 0, LUCE_EINVAL, "%s: slot %d sealed=%d must be a multiple of %d", who, s,
                c.sealed, LUCE_Q8KV_BLOCK);
        REQUIRE((int64_t)c.sealed + c.len <= LUCE_MAX_KEYS, LUCE_EUNSUPPORTED, "%s: slot %d would hold %lld keys (at most %d)", who, s,
                (long long)c.sealed + c.len, LUCE_MAX_KEYS);
        REQUIRE(c.n_pages >= 0 && c.n_pages * heads < ((int64_t)1 << 40), LUCE_EINVAL, "%s: slot %d n_pages=%d out of range", who, s,
                c.n_pages);
        Q8SealSlot& o = b.slot[s];
        o.k = reinterpret_cast<__half*>(c.k);
        o.v = reinterpret_cast<__half*>(c.v);
        o.n = c.len;
        o.cap = c.cap;
        o.sealed = c.sealed;
        r[nr++] = range_of(c.k, heads * c.cap * D * 2, s, "K tail", true);
        r[nr++] = range_of(c.v, heads * c.cap * D * 2, s, "V tail", true);
        const int whole = c.len / LUCE_Q8KV_BLOCK * LUCE_Q8KV_BLOCK;
        if (whole == 0) continue;
        units += whole / LUCE_Q8KV_BLOCK;
        REQUIRE(c.k_codes && c.v_codes && c.scales && aligned(c.k_codes, 16) && aligned(c.v_codes, 16) && aligned(c.scales, 16),
                LUCE_EINVAL, "%s: slot %d codes or scales null or not 16-byte aligned", who, s);
        REQUIRE(aligned(c.table, 4), LUCE_EINVAL, "%s: slot %d table misaligned", who, s);
        REQUIRE(c.table || (int64_t)c.n_pages * LUCE_PAGE_KEYS >= c.sealed + whole, LUCE_EINVAL,
                "%s: slot %d has %d pages for %d keys", who, s, c.n_pages, c.sealed + whole);
        o.k_codes = c.k_codes;
        o.v_codes = c.v_codes;
        o.scales = c.scales;
        o.table = c.table;
        o.n_pages = c.n_pages;
        // (of slots that share pools, what the host can see: through one table, or none, a key
        // has one place)
        for (int e = 0; e < s; ++e) {
            const luce_q8kv_slot& d = slots[e];
            const int end = d.sealed + d.len / LUCE_Q8KV_BLOCK * LUCE_Q8KV_BLOCK;
            const bool shared = c.table == d.table && (c.k_codes == d.k_codes || c.v_codes == d.v_codes || c.scales == d.scales);
            REQUIRE(!shared || end == d.sealed || c.sealed >= end || d.sealed >= c.sealed + whole, LUCE_EINVAL,
                    "%s: slots %d and %d would write the same blocks of one pool", who, e, s);
        }
        add_pool(r, &nr, c.k_codes, heads * kQ8PageBytes * c.n_pages, s, "K codes");
        add_pool(r, &nr, c.v_codes, heads * kQ8PageBytes * c.n_pages, s, "V codes");
        add_pool(r, &nr, c.scales, heads * kQ8PageScales * 4 * c.n_pages, s, "scales");
        if (c.table) r[nr++] = range_of(c.table, (c.sealed + whole + LUCE_PAGE_KEYS - 1) / LUCE_PAGE_KEYS * 4, s, "table", false);
    }
    if ((rc = check_apart(r, nr, who))) return rc;
    if (units == 0) return ok();
    return cuda_status(launch_q8kv_seal(b, n_layers, Hkv, (cudaStream_t)stream), who);
}

// ------------------------------------------------------------ attention

size_t luce_q8kv_attn_workspace_size(int n_rows, int Hq, int Hkv, int D, int max_sealed)
{
    if (n_rows < 1 || n_rows > LUCE_MAX_ROWS || Hkv < 1 || Hq < Hkv || Hq % Hkv || Hq / Hkv > 8 || Hkv > 4096 ||
        D != LUCE_HEAD_DIM || max_sealed < 0 || max_sealed > LUCE_MAX_KEYS)
        return 0;
    return std::max<size_t>(256, q8kv_part_bytes((int64_t)q8kv_max_chunks(max_sealed, Hkv) * n_rows * Hq));
}

int luce_q8kv_attn(const float* q, const luce_q8kv_view* views, int n_seq, int Hq, int Hkv, int D, float scale, float* out,
                   void* ws, size_t ws_bytes, void* stream)
{
    const char* who = "q8kv_attn";
    REQUIRE(q && out && ws && views, LUCE_EINVAL, "%s: null q/out/ws/views", who);
    REQUIRE(Hkv >= 1 && Hq >= Hkv && Hq % Hkv == 0, LUCE_EINVAL, "%s: Hq=%d must be a multiple of Hkv=%d", who, Hq, Hkv);
    REQUIRE(Hq / Hkv <= 8, LUCE_EUNSUPPORTED, "%s: group size %d > 8", who, Hq / Hkv);
    REQUIRE(Hkv <= 4096, LUCE_EUNSUPPORTED, "%s: %d KV heads > 4096", who, Hkv);
    REQUIRE(D == LUCE_HEAD_DIM, LUCE_EUNSUPPORTED, "%s: head_dim %d (only %d)", who, D, LUCE_HEAD_DIM);
    REQUIRE(isfinite(scale), LUCE_EINVAL, "%s: scale must be finite", who);
    REQUIRE(aligned(q, 16) && aligned(out, 4) && aligned(ws, 256), LUCE_EINVAL, "%s: q must be 16-byte, ws 256-byte aligned", who);
    REQUIRE(n_seq >= 1 && n_seq <= LUCE_MAX_SEQ, LUCE_EINVAL, "%s: n_seq=%d outside 1..%d (more than %d sequences are refused)", who,
            n_seq, LUCE_MAX_SEQ, LUCE_MAX_SEQ);
    Q8Batch b{};
    ByteRange r[6 * LUCE_MAX_SEQ + 3];
    int nr = 0;
    bool covered[LUCE_MAX_ROWS] = {};
    for (int s = 0; s < n_seq; ++s) {
        const luce_q8kv_view& v = views[s];
        const int rc = add_q8kv_view(b, s, v, Hkv, covered, who);
        if (rc) return rc;
        const Q8View& t = b.view[s];
        if (t.sealed > 0) {
            const int64_t pages = t.n_pages - 1;
            r[nr++] = range_of(t.k_codes, pages * t.page_stride + (int64_t)Hkv * kQ8PageBytes, s, "K codes", false);
            r[nr++] = range_of(t.v_codes, pages * t.page_stride + (int64_t)Hkv * kQ8PageBytes, s, "V codes", false);
            r[nr++] = range_of(t.scales, (pages * t.scale_stride + (int64_t)Hkv * kQ8PageScales) * 4, s, "scales", false);
            if (t.table) r[nr++] = range_of(t.table, (t.sealed + LUCE_PAGE_KEYS - 1) / LUCE_PAGE_KEYS * 4, s, "table", false);
        }
        const int64_t elems = t.head_stride * (Hkv - 1) + t.tok_stride * (t.tail + t.n_nodes - 1) + D;
        r[nr++] = range_of(t.k, elems * 2, s, "K tail", false);
        r[nr++] = range_of(t.v, elems * 2, s, "V tail", false);
    }
    for (int i = 0; i < b.n_row; ++i) REQUIRE(covered[i], LUCE_EINVAL, "%s: row %d belongs to no view", who, i);
    const size_t need = std::max<size_t>(256, q8kv_part_bytes(q8kv_chunks(b, Hq, Hkv)));
    REQUIRE(ws_bytes >= need, LUCE_ENOSPACE, "%s: workspace %zu bytes < %zu needed", who, ws_bytes, need);
    const int64_t heads = (int64_t)b.n_row * Hq;
    // (a row's q is read before its out is written)
    r[nr++] = range_of(q, heads * D * 4, -1, "q", false, 1);
    r[nr++] = range_of(out, heads * D * 4, -1, "out", true, 1);
    r[nr++] = range_of(ws, (int64_t)need, -1, "workspace", true);
    const int rc = check_apart(r, nr, who);
    if (rc) return rc;
    return cuda_status(launch_q8kv_attention(q, b, Hq, Hkv, scale, ws, out, (cudaStream_t)stream), who);
}

int luce_test_q8kv_wait_expiry(int64_t limit_ns, void* stream)
{
    REQUIRE(limit_ns >= 1000 && limit_ns <= 1000000000, LUCE_EINVAL,
            "test_q8kv_wait_expiry: limit_ns=%lld outside 1 us .. 1 s", (long long)limit_ns);
    return cuda_status(launch_q8kv_wait_expiry((uint64_t)limit_ns, (cudaStream_t)stream), "test_q8kv_wait_expiry");
}

int luce::add_q8kv_view(Q8Batch& b, int s, const luce_q8kv_view& v, int Hkv, bool* covered, const char* who)
{
    REQUIRE(v.k && v.v && aligned(v.k, 16) && aligned(v.v, 16), LUCE_EINVAL, "%s: view %d tail null or not 16-byte aligned", who, s);
    REQUIRE(v.n_nodes >= 1 && v.n_nodes <= LUCE_MAX_TREE, LUCE_EINVAL, "%s: view %d has %d nodes (1..%d)", who, s, v.n_nodes,
            LUCE_MAX_TREE);
    REQUIRE(v.sealed >= 0 && v.sealed % LUCE_Q8KV_BLOCK == 0 && v.len >= 0, LUCE_EINVAL,
            "%s: view %d sealed=%d must be a multiple of %d, len=%d not negative", who, s, v.sealed, LUCE_Q8KV_BLOCK, v.len);
    REQUIRE(v.len <= LUCE_Q8KV_MAX_TAIL, LUCE_EUNSUPPORTED, "%s: view %d has %d keys in its tail (at most %d: seal them)", who, s, v.len,
            LUCE_Q8KV_MAX_TAIL);
    REQUIRE((int64_t)v.sealed + v.len + v.n_nodes <= LUCE_MAX_KEYS, LUCE_EUNSUPPORTED, "%s: view %d has %lld keys (at most %d)", who, s,
            (long long)v.sealed + v.len + v.n_nodes, LUCE_MAX_KEYS);
    REQUIRE(v.len + v.n_nodes <= v.cap, LUCE_EINVAL, "%s: view %d len=%d + nodes=%d exceeds cap=%d", who, s, v.len, v.n_nodes, v.cap);
    REQUIRE(v.window >= 0 && v.sinks >= 0, LUCE_EINVAL, "%s: view %d window=%d and sinks=%d must not be negative", who, s, v.window,
            v.sinks);
    REQUIRE(v.tok_stride >= LUCE_HEAD_DIM && v.tok_stride % 8 == 0 && v.tok_stride < ((int64_t)1 << 32), LUCE_EINVAL,
            "%s: view %d tok_stride must be a multiple of 8, at least D", who, s);
    REQUIRE((int64_t)v.cap * v.tok_stride < ((int64_t)1 << 38) &&
                (Hkv == 1 || (v.head_stride % 8 == 0 && v.head_stride >= (int64_t)v.cap * v.tok_stride &&
                              v.head_stride < ((int64_t)1 << 38))),
            LUCE_EINVAL, "%s: view %d head_stride must be a multiple of 8 and keep the heads apart", who, s);
    REQUIRE(v.row0 >= 0 && v.row0 <= LUCE_MAX_ROWS - v.n_nodes, LUCE_EINVAL, "%s: view %d rows out of range", who, s);
    for (int j = 0; j < v.n_nodes; ++j) {
        REQUIRE(!covered[v.row0 + j], LUCE_EINVAL, "%s: row %d claimed twice", who, v.row0 + j);
        covered[v.row0 + j] = true;
    }
    const int rc = tree_path(v.parent, v.n_nodes, b.row, s, v.row0, who);
    if (rc) return rc;
    Q8View& t = b.view[s];
    if (v.sealed > 0) {
        REQUIRE(v.k_codes && v.v_codes && v.scales && aligned(v.k_codes, 16) && aligned(v.v_codes, 16) && aligned(v.scales, 16),
                LUCE_EINVAL, "%s: view %d codes or scales null or not 16-byte aligned", who, s);
        REQUIRE(aligned(v.table, 4), LUCE_EINVAL, "%s: view %d table misaligned", who, s);
        REQUIRE(v.n_pages >= 1 && (v.table || (int64_t)v.n_pages * LUCE_PAGE_KEYS >= v.sealed), LUCE_EINVAL,
                "%s: view %d has %d pages for %d keys", who, s, v.n_pages, v.sealed);
        const int64_t page = (int64_t)Hkv * kQ8PageBytes;
        REQUIRE(v.page_stride == 0 || (v.page_stride >= page && v.page_stride % kQ8PageBytes == 0 && v.page_stride < ((int64_t)1 << 38)),
                LUCE_EINVAL, "%s: view %d page_stride must be a multiple of %d and keep the pages apart", who, s, kQ8PageBytes);
        REQUIRE(v.n_pages <= ((int64_t)1 << 46) / std::max(v.page_stride, page), LUCE_EINVAL, "%s: view %d n_pages=%d out of range", who,
                s, v.n_pages);
        t.k_codes = v.k_codes;
        t.v_codes = v.v_codes;
        t.scales = v.scales;
        t.table = v.table;
        t.n_pages = v.n_pages;
        t.page_stride = v.page_stride ? v.page_stride : page;
        t.scale_stride = t.page_stride / kQ8PageBytes * kQ8PageScales;
    }
    t.k = reinterpret_cast<const __half*>(v.k);
    t.v = reinterpret_cast<const __half*>(v.v);
    t.head_stride = Hkv == 1 ? 0 : v.head_stride;
    t.tok_stride = v.tok_stride;
    t.sealed = v.sealed;
    t.tail = v.len;
    t.n_nodes = v.n_nodes;
    t.row0 = v.row0;
    t.window = v.window;
    t.sinks = v.sinks;
    b.n_view = s + 1;
    b.n_row = std::max(b.n_row, v.row0 + v.n_nodes);
    return LUCE_OK;
}
