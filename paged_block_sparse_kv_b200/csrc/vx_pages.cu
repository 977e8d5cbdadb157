// vx_pages.cu -- C ABI of the page calls (include/vx.h): validation, workspace layout, launches.
#include <algorithm>
#include <cstdio>

#include "vx_internal.h"

namespace {

using vx::set_error;

#define VX_TRY(x)                   \
    do {                            \
        vx_status _s = (x);         \
        if (_s != VX_OK) return _s; \
    } while (0)

constexpr int32_t MAX_ROWS = 4096;

vx_status bad(vx_status s, const char *what) { return set_error(s, what); }

vx_status check_word_ptr(const void *p, const char *name, bool can_be_null = false) {
    char msg[96];
    if (!p && can_be_null) return VX_OK;
    if (!p || (reinterpret_cast<uintptr_t>(p) & 3u)) {
        snprintf(msg, sizeof msg, "%s is NULL or not 4-byte aligned", name);
        return set_error(VX_ERR_INVALID_ARG, msg);
    }
    return VX_OK;
}

vx_status check_pool(const vx_geometry *g, const vx_page_pool *p) {
    if (!p) return bad(VX_ERR_INVALID_ARG, "page pool is NULL");
    if (p->elem_bytes != 1 && p->elem_bytes != 2) return bad(VX_ERR_INVALID_ARG, "elem_bytes must be 1 or 2");
    if (p->num_pages < 1 || p->num_pages > INT32_MAX / g->num_kv_heads)
        return bad(VX_ERR_INVALID_ARG, "num_pages must be >= 1, and num_pages * num_kv_heads fit int32");
    VX_TRY(vx::validate_ptr(p->k_cache, "pool k_cache", false));
    if (!g->mla_shared_kv) VX_TRY(vx::validate_ptr(p->v_cache, "pool v_cache", false));
    else if (p->v_cache) return bad(VX_ERR_INVALID_ARG, "an MLA pool has no v_cache");
    VX_TRY(vx::validate_ptr(p->centroids, "pool centroids", true));
    if ((p->k_scale == nullptr) != (p->v_scale == nullptr))
        return bad(VX_ERR_INVALID_ARG, "a pool has both scales or none");
    if (p->k_scale && p->elem_bytes != 1) return bad(VX_ERR_INVALID_ARG, "only 8-bit pools have scales");
    VX_TRY(check_word_ptr(p->k_scale, "pool k_scale", true));
    return check_word_ptr(p->v_scale, "pool v_scale", true);
}

vx::PoolArrays arrays(const vx_page_pool *p) {
    return {static_cast<uint8_t *>(p->k_cache), static_cast<uint8_t *>(p->v_cache),
            static_cast<uint8_t *>(p->centroids), p->k_scale, p->v_scale};
}

vx::PageArgs page_args(const vx_geometry *g, const vx_page_pool *src, const vx_page_pool *dst) {
    vx::PageArgs a{};
    a.src = arrays(src);
    a.dst = arrays(dst);
    const int32_t heads = g->num_kv_heads * g->page_size * dst->elem_bytes;
    a.kb = heads * g->head_dim_qk;
    a.vb = g->mla_shared_kv ? 0 : heads * g->head_dim_v;
    a.cb = dst->centroids ? g->num_kv_heads * g->head_dim_qk * 2 : 0;
    a.Hkv = g->num_kv_heads;
    a.P = g->page_size;
    a.src_pages = src->num_pages;
    a.num_pages = dst->num_pages;
    return a;
}

void table_args(vx::PageArgs *a, const vx_geometry *g, const vx_page_table *t) {
    a->page_ptr = t->page_ptr;
    a->page_indices = t->page_indices;
    a->seq_lens = t->seq_lens;
    a->B = g->batch;
    a->max_pages = t->max_pages;
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Workspace: head words, a word per page (the copy's claims) or per 32 pages (flags, whole segments
// of 1024 pages), a count per segment, four words per new row, one per old row (of the largest batch:
// the size depends on the pool and the new rows alone, and a workspace serves as the batch changes),
// two per possible move.
struct PageWs {
    size_t a, b, c, d, e, f, total;
};
PageWs page_ws(const vx_geometry *g, int32_t rows) {
    const size_t n = (size_t)g->num_pool_pages, segs = (n + 1023) / 1024;
    PageWs w;
    w.a = 256;
    w.b = w.a + up256(std::max(n, segs * 32) * sizeof(int32_t));
    w.c = w.b + up256(segs * sizeof(int32_t));
    w.d = w.c + up256((size_t)rows * 4 * sizeof(int32_t));
    w.e = w.d + up256((size_t)MAX_ROWS * sizeof(int32_t));
    w.f = w.e + up256((n / 2 + 1) * sizeof(int32_t));
    w.total = w.f + up256((n / 2 + 1) * sizeof(int32_t));
    return w;
}

vx_status set_ws(vx::PageArgs *a, const vx_geometry *g, int32_t rows, void *ws, size_t ws_bytes) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 15u))
        return bad(VX_ERR_WORKSPACE, "workspace is NULL or not 16-byte aligned");
    const PageWs w = page_ws(g, rows);
    if (ws_bytes < w.total) {
        char msg[96];
        snprintf(msg, sizeof msg, "workspace of %zu bytes < %zu needed", ws_bytes, w.total);
        return set_error(VX_ERR_WORKSPACE, msg);
    }
    char *p = static_cast<char *>(ws);
    a->head = reinterpret_cast<int32_t *>(p);
    a->list_a = reinterpret_cast<int32_t *>(p + w.a);
    a->list_b = reinterpret_cast<int32_t *>(p + w.b);
    a->list_c = reinterpret_cast<int32_t *>(p + w.c);
    a->list_d = reinterpret_cast<int32_t *>(p + w.d);
    a->list_e = reinterpret_cast<int32_t *>(p + w.e);
    a->list_f = reinterpret_cast<int32_t *>(p + w.f);
    return VX_OK;
}

vx_status launched(cudaError_t e, const char *where) {
    if (e == cudaSuccess) return VX_OK;
    char msg[160];
    snprintf(msg, sizeof msg, "%s: %s", where, cudaGetErrorString(e));
    return set_error(VX_ERR_CUDA, msg);
}

// The kernels index their work with 31 bits: pieces of 16 KB of a page, spans of 256 table entries.
int64_t pieces_of(const vx::PageArgs &a) { return (((int64_t)a.kb + a.vb + a.cb) / 16 + 1023) / 1024; }
vx_status check_work(int64_t units) {
    return units <= INT32_MAX ? VX_OK : bad(VX_ERR_UNSUPPORTED, "more than 2^31 units of work in one call");
}

// [a, a + an) and [b, b + bn) share a byte
bool overlap(const void *a, size_t an, const void *b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + bn && y < x + an;
}

// Any array of one pool shares memory with any array of the other
bool pools_overlap(const vx_page_pool *p, const vx_page_pool *q, const vx::PageArgs &a) {
    const size_t bytes[5] = {(size_t)a.kb, (size_t)a.vb, (size_t)a.cb, p->k_scale ? (size_t)a.Hkv * 4 : 0,
                             p->k_scale ? (size_t)a.Hkv * 4 : 0};  // of a page, in both pools
    const void *x[5] = {p->k_cache, p->v_cache, p->centroids, p->k_scale, p->v_scale};
    const void *y[5] = {q->k_cache, q->v_cache, q->centroids, q->k_scale, q->v_scale};
    for (int i = 0; i < 5; ++i)
        for (int j = 0; j < 5; ++j)
            if (bytes[i] && bytes[j] &&
                overlap(x[i], (size_t)p->num_pages * bytes[i], y[j], (size_t)q->num_pages * bytes[j]))
                return true;
    return false;
}

}  // namespace

extern "C" {

size_t vx_page_workspace_size(const vx_geometry *geo, int32_t rows) {
    if (vx::validate_geometry(geo) != VX_OK) return 0;
    if (rows < 1 || rows > MAX_ROWS) {
        bad(VX_ERR_INVALID_ARG, "rows must be in [1, 4096]");
        return 0;
    }
    return page_ws(geo, rows).total;
}

vx_status vx_copy_pages(const vx_geometry *geo, const vx_page_pool *src, const vx_page_pool *dst,
                        const int32_t *src_pages, const int32_t *dst_pages, int32_t num_copies, void *ws,
                        size_t ws_bytes, int32_t *err, void *stream) {
    VX_TRY(vx::validate_geometry(geo));
    VX_TRY(check_pool(geo, src));
    VX_TRY(check_pool(geo, dst));
    if (dst->num_pages != geo->num_pool_pages)
        return bad(VX_ERR_INVALID_ARG, "the destination pool must have num_pool_pages pages");
    if (src->elem_bytes != dst->elem_bytes || !src->centroids != !dst->centroids || !src->k_scale != !dst->k_scale)
        return bad(VX_ERR_INVALID_ARG, "the pools must have the same arrays and element size");
    if (num_copies < 0) return bad(VX_ERR_INVALID_ARG, "num_copies < 0");
    VX_TRY(check_word_ptr(err, "err", true));
    vx::PageArgs a = page_args(geo, src, dst);
    const bool one = src->k_cache == dst->k_cache;
    if (one && (src->v_cache != dst->v_cache || src->centroids != dst->centroids || src->k_scale != dst->k_scale ||
                src->v_scale != dst->v_scale || src->num_pages != dst->num_pages))
        return bad(VX_ERR_INVALID_ARG, "pools that share k_cache must be the same pool");
    if (!one && pools_overlap(src, dst, a)) return bad(VX_ERR_INVALID_ARG, "two pools must not overlap in memory");
    if (num_copies == 0) return VX_OK;
    VX_TRY(check_word_ptr(src_pages, "src_pages"));
    VX_TRY(check_word_ptr(dst_pages, "dst_pages"));
    VX_TRY(set_ws(&a, geo, 1, ws, ws_bytes));
    a.copy_src = src_pages;
    a.copy_dst = dst_pages;
    a.num_copies = num_copies;
    a.one_pool = one ? 1 : 0;
    a.err = err;
    VX_TRY(check_work(num_copies * pieces_of(a)));
    return launched(vx::launch_copy_pages(a, static_cast<cudaStream_t>(stream)), "page copy launch");
}

vx_status vx_update_table(const vx_geometry *geo, const vx_page_pool *pool, const vx_page_table *table,
                          const int32_t *ref_in, const int32_t *parent, const int32_t *grow, int32_t new_rows,
                          const int32_t *new_page_ptr, int32_t *new_page_indices, int64_t num_indices,
                          int32_t *new_seq_lens, int32_t new_max_pages, int32_t *ref_out, void *ws, size_t ws_bytes,
                          int32_t *err, void *stream) {
    VX_TRY(vx::validate_table(geo, table));
    VX_TRY(check_pool(geo, pool));
    if (pool->num_pages != geo->num_pool_pages)
        return bad(VX_ERR_INVALID_ARG, "the pool must have num_pool_pages pages");
    if (new_rows < 1 || new_rows > MAX_ROWS) return bad(VX_ERR_INVALID_ARG, "new_rows must be in [1, 4096]");
    if (new_max_pages < 1 || (int64_t)new_max_pages * geo->page_size > INT32_MAX)
        return bad(VX_ERR_INVALID_ARG, "new_max_pages must be >= 1, and its tokens fit int32");
    if (num_indices < 1 || num_indices > INT32_MAX) return bad(VX_ERR_INVALID_ARG, "num_indices must be in [1, 2^31)");
    VX_TRY(check_word_ptr(parent, "parent"));
    VX_TRY(check_word_ptr(grow, "grow"));
    VX_TRY(check_word_ptr(new_page_ptr, "new_page_ptr"));
    VX_TRY(check_word_ptr(new_page_indices, "new_page_indices"));
    VX_TRY(check_word_ptr(new_seq_lens, "new_seq_lens"));
    VX_TRY(vx::validate_ptr(ref_in, "ref_in", false));
    VX_TRY(vx::validate_ptr(ref_out, "ref_out", false));
    VX_TRY(check_word_ptr(err, "err", true));
    const size_t pool_words = (size_t)pool->num_pages * 4;
    if (ref_in != ref_out && overlap(ref_in, pool_words, ref_out, pool_words))
        return bad(VX_ERR_INVALID_ARG, "ref_out must be ref_in itself or apart from it");
    if (overlap(new_page_indices, (size_t)num_indices * 4, table->page_indices, 4) ||
        overlap(new_seq_lens, (size_t)new_rows * 4, table->seq_lens, (size_t)geo->batch * 4))
        return bad(VX_ERR_INVALID_ARG, "the new rows must not lie in the old table's memory");
    vx::PageArgs a = page_args(geo, pool, pool);
    table_args(&a, geo, table);
    VX_TRY(set_ws(&a, geo, new_rows, ws, ws_bytes));
    a.ref_in = ref_in;
    a.ref_out = ref_out;
    a.parent = parent;
    a.grow = grow;
    a.new_rows = new_rows;
    a.new_ptr = new_page_ptr;
    a.new_indices = new_page_indices;
    a.num_indices = num_indices;
    a.new_lens = new_seq_lens;
    a.new_max_pages = new_max_pages;
    a.err = err;
    VX_TRY(check_work(8 * (new_rows * pieces_of(a) + 4) + pool->num_pages / 256 +
                      ((int64_t)new_rows + geo->batch + 2) * (table->max_pages / 256 + 1)));
    return launched(vx::launch_update_table(a, static_cast<cudaStream_t>(stream)), "table update launch");
}

vx_status vx_compact_pages(const vx_geometry *geo, const vx_page_pool *pool, const vx_page_table *table,
                           const int32_t *ref_in, int32_t *page_indices_out, int32_t *ref_out, int32_t *remap,
                           int32_t *num_live, void *ws, size_t ws_bytes, int32_t *err, void *stream) {
    VX_TRY(vx::validate_table(geo, table));
    VX_TRY(check_pool(geo, pool));
    if (pool->num_pages != geo->num_pool_pages)
        return bad(VX_ERR_INVALID_ARG, "the pool must have num_pool_pages pages");
    VX_TRY(vx::validate_ptr(ref_in, "ref_in", false));
    VX_TRY(check_word_ptr(page_indices_out, "page_indices_out"));
    VX_TRY(vx::validate_ptr(ref_out, "ref_out", false));  // written in 16-byte stores
    VX_TRY(check_word_ptr(remap, "remap"));
    VX_TRY(check_word_ptr(num_live, "num_live"));
    VX_TRY(check_word_ptr(err, "err", true));
    const size_t pool_words = (size_t)pool->num_pages * 4;
    if (ref_in != ref_out && overlap(ref_in, pool_words, ref_out, pool_words))
        return bad(VX_ERR_INVALID_ARG, "ref_out must be ref_in itself or apart from it");
    if (overlap(remap, pool_words, ref_in, pool_words) || overlap(remap, pool_words, ref_out, pool_words))
        return bad(VX_ERR_INVALID_ARG, "remap must be apart from the reference counts");
    vx::PageArgs a = page_args(geo, pool, pool);
    table_args(&a, geo, table);
    VX_TRY(set_ws(&a, geo, 1, ws, ws_bytes));
    a.ref_in = ref_in;
    a.ref_out = ref_out;
    a.indices_out = page_indices_out;
    a.remap = remap;
    a.num_live = num_live;
    a.err = err;
    VX_TRY(check_work(pool->num_pages * pieces_of(a) + ((int64_t)geo->batch + 2) * (table->max_pages / 256 + 1) + (1 << 20)));
    return launched(vx::launch_compact_pages(a, static_cast<cudaStream_t>(stream)), "page compaction launch");
}

}  // extern "C"
