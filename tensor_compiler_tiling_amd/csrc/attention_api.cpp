// C entry points of the key-value cache and of attention over it
// (include/convtile.h): argument checks, the choice of kernel and the launch.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cstdint>

#include "../../include/convtile.h"
#include "attention_kernels.hpp"
#include "ct_kernels.hpp"

namespace ct {

namespace {

constexpr long long kMaxPlaces = 1LL << 30;   // a sequence's
constexpr long long kMaxRows = (1LL << 26) - 1;    // tokens x heads: 64 threads each in a launch of fewer than 2^32
constexpr long long kMaxGroups = (1LL << 23) - 1;  // workgroups of 512 threads
constexpr long long kMaxStride = 1LL << 40;   // elements

bool plain_dtype(int dt) { return dt == CT_F32 || dt == CT_F16 || dt == CT_BF16; }
int elem_bytes(int dt) { return dt == CT_F32 ? 4 : dt == CT_E4M3 ? 1 : 2; }

bool misaligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

// Strides of [outer][middle][inner] rows of `dim` elements: any order of the
// axes, no two rows on one place.
bool apart(long long a, long long na, long long b, long long nb, long long c, long long nc, long long dim) {
    long long st[3] = {a, b, c}, n[3] = {na, nb, nc};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (st[j] < st[i]) {
                const long long s = st[i], m = n[i];
                st[i] = st[j], n[i] = n[j], st[j] = s, n[j] = m;
            }
    __int128 reach = dim;  // elements that the axes so far span
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;  // an axis of one has no stride to speak of
        if (st[i] < reach) return false;
        reach += (__int128)st[i] * (n[i] - 1);
    }
    return true;
}

int check_cache(const ct_kv_cache* c, KvPages* out) {
    if (!c) return fail(CT_ERR_INVALID_ARG, "cache must not be NULL");
    if (c->dtype != CT_F16 && c->dtype != CT_BF16 && c->dtype != CT_E4M3)
        return fail(CT_ERR_INVALID_ARG, "cache: unknown dtype %d", c->dtype);
    if (c->pages < 1 || c->heads < 1 || c->page < 1 || c->dim < 1)
        return fail(CT_ERR_INVALID_ARG, "cache: pages, heads, page and dim must be positive");
    if (c->dim % 16 || c->dim > 256)
        return fail(CT_ERR_UNSUPPORTED, "cache: rows of %d elements (whole multiples of 16 up to 256)", c->dim);
    if (c->heads > 1 << 16) return fail(CT_ERR_UNSUPPORTED, "cache: more than 2^16 heads");
    if (!c->k || !c->v) return fail(CT_ERR_INVALID_ARG, "cache: k and v must not be NULL");
    const int es = elem_bytes(c->dtype);
    if (misaligned(c->k, 16) || misaligned(c->v, 16)) return fail(CT_ERR_INVALID_ARG, "cache: k and v must be 16-byte aligned");
    const long long ld[3] = {c->ld_page, c->ld_head, c->ld_token}, n[3] = {c->pages, c->heads, c->page};
    const long long lds[3] = {c->lds_page, c->lds_head, c->lds_token};
    const bool q8 = c->dtype == CT_E4M3;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (ld[i] < 1 || ld[i] > kMaxStride || (q8 && (lds[i] < 1 || lds[i] > kMaxStride)))
            return fail(CT_ERR_INVALID_ARG, "cache: strides must be positive (at most 2^40)");
        if (ld[i] * es % 16) return fail(CT_ERR_INVALID_ARG, "cache: rows must be whole multiples of 16 bytes apart");
    }
    if (!apart(ld[0], n[0], ld[1], n[1], ld[2], n[2], c->dim)) return fail(CT_ERR_INVALID_ARG, "cache: rows must not overlap");
    if (q8) {
        if (!c->k_scale || !c->v_scale) return fail(CT_ERR_INVALID_ARG, "cache: 8-bit rows have scales");
        if (misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4))
            return fail(CT_ERR_INVALID_ARG, "cache: scales are not aligned to their elements");
        if (!apart(lds[0], n[0], lds[1], n[1], lds[2], n[2], 1)) return fail(CT_ERR_INVALID_ARG, "cache: scales must not overlap");
    } else if (c->k_scale || c->v_scale) {
        return fail(CT_ERR_INVALID_ARG, "cache: scales belong to CT_E4M3");
    }
    KvPages p{};
    p.k = static_cast<char*>(c->k);
    p.v = static_cast<char*>(c->v);
    p.ks = c->k_scale;
    p.vs = c->v_scale;
    p.pages = c->pages, p.heads = c->heads, p.page = c->page, p.dim = c->dim;
    p.ld_page = n[0] > 1 ? ld[0] * es : 0, p.ld_head = n[1] > 1 ? ld[1] * es : 0, p.ld_token = n[2] > 1 ? ld[2] * es : 0;
    if (q8) p.lds_page = n[0] > 1 ? lds[0] : 0, p.lds_head = n[1] > 1 ? lds[1] : 0, p.lds_token = n[2] > 1 ? lds[2] : 0;
    page_magic(p);
    *out = p;
    return CT_OK;
}

int check_batch(const ct_kv_batch* b, const KvPages& c, KvBatch* out) {
    if (!b) return fail(CT_ERR_INVALID_ARG, "batch must not be NULL");
    if (b->tokens < 0 || b->sequences < 0) return fail(CT_ERR_INVALID_ARG, "tokens and sequences must not be negative");
    if (b->tokens == 0) return CT_OK;
    if (b->sequences < 1) return fail(CT_ERR_INVALID_ARG, "%d tokens of no sequence", b->tokens);
    if (!b->lens) return fail(CT_ERR_INVALID_ARG, "lens must not be NULL");
    if (misaligned(b->lens, 4) || misaligned(b->starts, 4) || misaligned(b->table, 4))
        return fail(CT_ERR_INVALID_ARG, "lens, starts and table must be aligned to their elements");
    if (!b->starts && b->tokens % b->sequences)
        return fail(CT_ERR_INVALID_ARG, "%d tokens of %d sequences need starts", b->tokens, b->sequences);
    if (b->table) {
        if (b->width < 1) return fail(CT_ERR_INVALID_ARG, "the table must have columns");
        if (b->sequences > 1 && (b->ldt < b->width || b->ldt > kMaxStride))
            return fail(CT_ERR_INVALID_ARG, "table: row stride %lld for %d columns", b->ldt, b->width);
    } else if (b->sequences > c.pages) {
        return fail(CT_ERR_INVALID_ARG, "%d sequences of a page each need as many pages (got %d)", b->sequences, c.pages);
    }
    KvBatch o{};
    o.width = b->table ? b->width : 1;
    if ((long long)o.width * c.page > kMaxPlaces) return fail(CT_ERR_UNSUPPORTED, "more than 2^30 places a sequence");
    if ((long long)b->tokens * c.heads > kMaxRows) return fail(CT_ERR_UNSUPPORTED, "2^26 rows or more in a call");
    if (b->sequences > 1 << 24) return fail(CT_ERR_UNSUPPORTED, "more than 2^24 sequences");
    // attention's workgroups count through the starts
    if (b->starts && b->sequences > 1 << 16) return fail(CT_ERR_UNSUPPORTED, "more than 2^16 sequences with starts");
    o.lens = b->lens, o.starts = b->starts, o.table = b->table;
    o.ldt = b->sequences > 1 ? b->ldt : 0;
    o.tokens = b->tokens, o.sequences = b->sequences;
    o.even = b->tokens / b->sequences;
    *out = o;
    return CT_OK;
}

// [tokens][heads] rows of `dim` elements.  `written`: no two on one place.
int check_rows(const char* name, const void* p, long long token, long long head, int tokens, int heads, int dim, int dt, bool written) {
    if (!p) return fail(CT_ERR_INVALID_ARG, "%s must not be NULL", name);
    if (misaligned(p, elem_bytes(dt))) return fail(CT_ERR_INVALID_ARG, "%s is not aligned to its elements", name);
    if ((tokens > 1 && (token < 0 || token > kMaxStride)) || (heads > 1 && (head < 0 || head > kMaxStride)))
        return fail(CT_ERR_INVALID_ARG, "%s: strides must not be negative (at most 2^40)", name);
    if (written && !apart(token, tokens, head, heads, 0, 1, dim)) return fail(CT_ERR_INVALID_ARG, "%s: rows must not overlap", name);
    return CT_OK;
}

int rows_call(const ct_kv_cache* cache, const ct_kv_batch* batch, const void* k, long long k_token, long long k_head, const void* v,
              long long v_token, long long v_head, int dtype, bool write, void* stream) {
    KvRowsParams p{};
    int st = check_cache(cache, &p.c);
    if (st == CT_OK) st = check_batch(batch, p.c, &p.b);
    if (st != CT_OK) return st;
    if (!plain_dtype(dtype)) return fail(CT_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    const int n = batch->tokens, es = elem_bytes(dtype);
    if (n == 0) return CT_OK;
    st = check_rows("k", k, k_token, k_head, n, p.c.heads, p.c.dim, dtype, !write);
    if (st == CT_OK) st = check_rows("v", v, v_token, v_head, n, p.c.heads, p.c.dim, dtype, !write);
    if (st == CT_OK && write && cache->k == cache->v) return fail(CT_ERR_INVALID_ARG, "cache: k and v must not be the same");
    if (st == CT_OK && write && cache->dtype == CT_E4M3 && cache->k_scale == cache->v_scale)
        return fail(CT_ERR_INVALID_ARG, "cache: k_scale and v_scale must not be the same");
    if (st == CT_OK && !write && k == v) return fail(CT_ERR_INVALID_ARG, "k and v must not be the same");
    if (st == CT_OK && (k == cache->k || k == cache->v || v == cache->k || v == cache->v))
        return fail(CT_ERR_INVALID_ARG, "k and v must not be the cache's own");
    if (st != CT_OK) return st;
    p.k = static_cast<char*>(const_cast<void*>(k));
    p.v = static_cast<char*>(const_cast<void*>(v));
    p.k_token = n > 1 ? k_token * es : 0, p.v_token = n > 1 ? v_token * es : 0;
    p.k_head = p.c.heads > 1 ? k_head * es : 0, p.v_head = p.c.heads > 1 ? v_head * es : 0;
    const hipError_t e = write ? launch_kv_write(p, cache->dtype, dtype, static_cast<hipStream_t>(stream))
                               : launch_kv_read(p, cache->dtype, dtype, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? CT_OK : hip_fail(e, write ? "kv_write launch" : "kv_read launch");
}

// The sizes of a call, whose plan goes to `plan` (not for no tokens).
int check_sizes(int tokens, int sequences, int heads, int kv_heads, int dim, long long max_len, int window, int sinks,
                int cache_dtype, AttendPlan* plan) {
    if (tokens < 0 || sequences < 0 || heads < 1 || kv_heads < 1 || dim < 1 || max_len < 0)
        return fail(CT_ERR_INVALID_ARG, "counts must not be negative, heads and dim must be positive");
    if (heads % kv_heads) return fail(CT_ERR_INVALID_ARG, "%d heads of q for %d of the cache", heads, kv_heads);
    if (cache_dtype != CT_F16 && cache_dtype != CT_BF16 && cache_dtype != CT_E4M3)
        return fail(CT_ERR_INVALID_ARG, "cache: unknown dtype %d", cache_dtype);
    if (window < 0 || sinks < 0) return fail(CT_ERR_INVALID_ARG, "window and sinks must not be negative");
    if (sinks && !window) return fail(CT_ERR_INVALID_ARG, "sinks belong to a window");
    if (dim % 16 || dim > 256) return fail(CT_ERR_UNSUPPORTED, "rows of %d elements (whole multiples of 16 up to 256)", dim);
    if ((long long)tokens * heads > kMaxRows) return fail(CT_ERR_UNSUPPORTED, "2^26 rows or more of q");
    if (sequences > 1 << 24 || heads > 1 << 16) return fail(CT_ERR_UNSUPPORTED, "more than 2^24 sequences or 2^16 heads");
    if (tokens == 0) return CT_OK;
    if (sequences < 1) return fail(CT_ERR_INVALID_ARG, "%d tokens of no sequence", tokens);
    const long long most = max_len && max_len < kMaxPlaces ? max_len : kMaxPlaces;
    *plan = attend_plan(tokens, sequences, kv_heads, heads / kv_heads, dim, most, window ? window : kNoWindow, sinks,
                        cache_dtype == CT_E4M3);
    return CT_OK;
}

}  // namespace
}  // namespace ct

extern "C" {

int ct_kv_write(const ct_kv_cache* cache, const ct_kv_batch* batch, const void* k, long long k_token, long long k_head,
                const void* v, long long v_token, long long v_head, int dtype, void* stream) {
    return ct::rows_call(cache, batch, k, k_token, k_head, v, v_token, v_head, dtype, true, stream);
}

int ct_kv_read(const ct_kv_cache* cache, const ct_kv_batch* batch, void* k, long long k_token, long long k_head, void* v,
               long long v_token, long long v_head, int dtype, void* stream) {
    return ct::rows_call(cache, batch, k, k_token, k_head, v, v_token, v_head, dtype, false, stream);
}

int ct_kv_attention_fwd(const ct_kv_cache* cache, const ct_kv_batch* batch, const ct_kv_mask* mask, const void* q,
                        long long q_token, long long q_head, void* y, long long y_token, long long y_head, int heads, int dtype,
                        float scale, long long max_len, void* workspace, long long workspace_bytes, void* stream) {
    using namespace ct;
    AttendParams p{};
    int st = check_cache(cache, &p.c);
    if (st == CT_OK) st = check_batch(batch, p.c, &p.b);
    if (st != CT_OK) return st;
    const ct_kv_mask none{0, 0, nullptr, 0};
    const ct_kv_mask& mk = mask ? *mask : none;
    const int n = batch->tokens;
    AttendPlan plan{};
    st = check_sizes(n, batch->sequences, heads, cache->heads, cache->dim, max_len, mk.window, mk.sinks, cache->dtype, &plan);
    if (st != CT_OK) return st;
    if (dtype != CT_F16 && dtype != CT_BF16) return fail(CT_ERR_INVALID_ARG, "q must be CT_F16 or CT_BF16, got %d", dtype);
    if (cache->dtype != CT_E4M3 && cache->dtype != dtype)
        return fail(CT_ERR_INVALID_ARG, "q of dtype %d over a cache of %d", dtype, cache->dtype);
    if (!(scale > 0.0f && scale <= FLT_MAX)) return fail(CT_ERR_INVALID_ARG, "scale must be positive and finite");
    // 8-bit rows widen to half their value in fp16
    p.scale = scale * 1.44269504f * (cache->dtype == CT_E4M3 && dtype == CT_F16 ? 2.0f : 1.0f);
    if (!(p.scale > 0.0f && p.scale <= FLT_MAX)) return fail(CT_ERR_UNSUPPORTED, "scale %g leaves the range of fp32", (double)scale);
    if (mk.tree ? mk.words < 1 || mk.words > 1 << 20 : mk.words != 0)
        return fail(CT_ERR_INVALID_ARG, "a tree has rows of 1 to 2^20 words, and words belong to a tree");
    if (misaligned(mk.tree, 8)) return fail(CT_ERR_INVALID_ARG, "tree is not aligned to its elements");
    if (n == 0) return CT_OK;
    st = check_rows("q", q, q_token, q_head, n, heads, cache->dim, dtype, false);
    if (st == CT_OK) st = check_rows("y", y, y_token, y_head, n, heads, cache->dim, dtype, true);
    if (st != CT_OK) return st;
    if (y == q || y == cache->k || y == cache->v) return fail(CT_ERR_INVALID_ARG, "y must not be q or the cache");
    const long long need = attend_workspace_bytes(plan, n, heads, cache->dim);
    if (need > 0) {
        if (!workspace || workspace_bytes < need)
            return fail(CT_ERR_INVALID_ARG, "this call needs a workspace of %lld bytes (got %lld)", need,
                        workspace ? workspace_bytes : 0LL);
        if (misaligned(workspace, 16)) return fail(CT_ERR_INVALID_ARG, "workspace is not 16-byte aligned");
    }
    p.q = static_cast<const char*>(q);
    p.y = static_cast<char*>(y);
    p.q_token = n > 1 ? q_token * 2 : 0, p.y_token = n > 1 ? y_token * 2 : 0;
    p.q_head = heads > 1 ? q_head * 2 : 0, p.y_head = heads > 1 ? y_head * 2 : 0;
    p.tree = mk.tree;
    p.words = mk.words;
    p.group = heads / cache->heads;
    p.window = mk.window && mk.window < kNoWindow ? mk.window : kNoWindow;
    p.sinks = mk.sinks < kNoWindow ? mk.sinks : kNoWindow;
    const long long tiles = attend_tiles(plan, p.b, p.group);
    if (tiles * plan.parts * p.c.heads > kMaxGroups) return fail(CT_ERR_UNSUPPORTED, "more workgroups than one launch takes");
    p.tiles = (int)tiles;
    p.parts = plan.parts;
    if (p.parts > 1) {
        // the sums first: their rows are whole multiples of 16 bytes
        p.part_o = static_cast<float*>(workspace);
        p.part_ml = p.part_o + (long long)p.parts * n * heads * cache->dim;
    }
    const hipError_t e = launch_attend(plan, p, cache->dtype, dtype, static_cast<hipStream_t>(stream));
    return e == hipSuccess ? CT_OK : hip_fail(e, "attention launch");
}

long long ct_kv_attention_workspace_bytes(int tokens, int sequences, int heads, int kv_heads, int dim, long long max_len,
                                          int window, int sinks, int cache_dtype) {
    ct::AttendPlan plan{};
    const int st = ct::check_sizes(tokens, sequences, heads, kv_heads, dim, max_len, window, sinks, cache_dtype, &plan);
    if (st != CT_OK) return st;
    return tokens == 0 ? 0 : ct::attend_workspace_bytes(plan, tokens, heads, dim);
}

}  // extern "C"
