// k_pages.cu -- pages of a pool: copy, new table rows (fork, free, grow), compaction.
//
// Each call is a planning kernel and an applying kernel.  The planner is one thread-block
// cluster: its CTAs split the pool's reference counts, exchange their totals through
// distributed shared memory and give every free (or live) page its rank by prefix sums, so
// that the pages handed out depend on the counts alone, never on timing.  The applier fills
// the GPU: page data moves in pieces of PG_PIECE 16-byte chunks, table rows and reference
// counts in spans of PG_SPAN entries.  Bound: HBM for the page data (read and written once),
// latency of a few dependent loads for the planner.
#include <cooperative_groups.h>

#include <algorithm>

#include "vx_internal.h"

namespace cg = cooperative_groups;

namespace vx {

namespace {

constexpr int PG_CTAS = 8;        // CTAs of the planning cluster
constexpr int PG_THREADS = 1024;  // threads of a planning CTA
constexpr int PG_WARPS = PG_THREADS / 32;
constexpr int PG_MAX_ROWS = 4096;
constexpr int PG_PIECE = 1024;    // 16-byte chunks of a page moved by one block at a time
constexpr int PG_SPAN = 1024;     // table entries handled by one block at a time
constexpr int PG_BLOCK = 256;     // threads of an applying block

// ------------------------------------------------------------------ ranks over the pool

// Warp w of the cluster (of PG_CTAS * PG_WARPS) owns pages [w * span, (w + 1) * span), span a
// multiple of 128: 32 lanes x 4 consecutive pages per step.
__device__ __forceinline__ int64_t warp_span(int64_t n) {
    const int64_t w = PG_CTAS * PG_WARPS;
    return ((n + w - 1) / w + 127) / 128 * 128;
}

__device__ __forceinline__ int4 load4(const int32_t *p, int64_t at, int64_t n, int fill) {
    if (at + 4 <= n) return *reinterpret_cast<const int4 *>(p + at);
    int4 v = make_int4(fill, fill, fill, fill);
    if (at < n) v.x = p[at];
    if (at + 1 < n) v.y = p[at + 1];
    if (at + 2 < n) v.z = p[at + 2];
    return v;
}

// Flags of a lane's 4 pages (bit e: page at + e has ref > 0 when LIVE, == 0 otherwise; none past n)
template <bool LIVE>
__device__ __forceinline__ uint32_t flags4(const int4 &v, int64_t at, int64_t n) {
    const int r[4] = {v.x, v.y, v.z, v.w};
    uint32_t f = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (at + e < n && (LIVE ? r[e] > 0 : r[e] == 0)) f |= 1u << e;
    return f;
}

// Exclusive rank of the calling lane's first flag among the warp's (lane-major order), and the
// warp's total.
__device__ __forceinline__ int lane_rank(uint32_t f, int lane, int &total) {
    int before = 0;
    total = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t b = __ballot_sync(FULL, (f >> e) & 1u);
        before += __popc(b & ((1u << lane) - 1u));
        total += __popc(b);
    }
    return before;
}

// Count the flagged pages of every warp of the cluster and give each its exclusive base.
// `s_warp` [PG_WARPS] and `s_total` are shared; each(at, v) sees every lane's loads.
template <bool LIVE, typename Each>
__device__ int64_t cluster_base(const int32_t *ref, int64_t n, int32_t *s_warp, int32_t *s_total, int64_t &all,
                                Each each) {
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t span = warp_span(n), p0 = ((int64_t)cl.block_rank() * PG_WARPS + warp) * span;
    int count = 0;
#pragma unroll 4
    for (int64_t o = 0; o < span; o += 128) {
        const int64_t at = p0 + o + lane * 4;
        const int4 v = load4(ref, at, n, -1);
        count += __popc(flags4<LIVE>(v, at, n));
        each(at, v);
    }
    count = __reduce_add_sync(FULL, count);
    if (lane == 0) s_warp[warp] = count;
    __syncthreads();
    if (warp == 0) {
        const int c = s_warp[lane];
        int x = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(FULL, x, off);
            if (lane >= off) x += y;
        }
        s_warp[lane] = x - c;
        if (lane == 31) *s_total = x;
    }
    cl.sync();
    int64_t base = s_warp[warp];
    all = 0;
    for (int c = 0; c < PG_CTAS; ++c) {
        const int t = *cl.map_shared_rank(s_total, c);
        if (c < (int)cl.block_rank()) base += t;
        all += t;
    }
    return base;
}

// ------------------------------------------------------------------ page data

// 16-byte chunks of one page over all arrays, and its pieces
__device__ __forceinline__ int page_chunks(const PageArgs &a) { return (a.kb + a.vb + a.cb) >> 4; }
__device__ __forceinline__ int page_pieces(const PageArgs &a) { return ceil_div(page_chunks(a), PG_PIECE); }

__device__ __forceinline__ void copy_piece(const PageArgs &a, int64_t src, int64_t dst, int piece) {
    const int nk = a.kb >> 4, nv = a.vb >> 4, nc = a.cb >> 4;
    constexpr int U = PG_PIECE / PG_BLOCK;
    uint4 v[U];
    uint8_t *to[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        int c = piece * PG_PIECE + u * PG_BLOCK + (int)threadIdx.x;
        const uint8_t *from = nullptr;
        to[u] = nullptr;
        if (c < nk) {
            from = a.src.k + src * a.kb + (int64_t)c * 16;
            to[u] = a.dst.k + dst * a.kb + (int64_t)c * 16;
        } else if ((c -= nk) < nv) {
            from = a.src.v + src * a.vb + (int64_t)c * 16;
            to[u] = a.dst.v + dst * a.vb + (int64_t)c * 16;
        } else if ((c -= nv) < nc) {
            from = a.src.cen + src * a.cb + (int64_t)c * 16;
            to[u] = a.dst.cen + dst * a.cb + (int64_t)c * 16;
        }
        if (from) v[u] = *reinterpret_cast<const uint4 *>(from);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (to[u]) *reinterpret_cast<uint4 *>(to[u]) = v[u];
    if (piece == 0 && a.src.ks && (int)threadIdx.x < a.Hkv) {
        a.dst.ks[dst * a.Hkv + threadIdx.x] = a.src.ks[src * a.Hkv + threadIdx.x];
        a.dst.vs[dst * a.Hkv + threadIdx.x] = a.src.vs[src * a.Hkv + threadIdx.x];
    }
}

// ------------------------------------------------------------------ copy

// list_a[p], for every page p a copy names as a destination: the lowest index of such a copy,
// or -1 when the page is also a source (one pool).  Entries of other pages are not read.
__global__ void __cluster_dims__(PG_CTAS) __launch_bounds__(PG_THREADS) k_plan_copy(const PageArgs a) {
    pdl_wait();
    pdl_trigger();
    cg::cluster_group cl = cg::this_cluster();
    const int t0 = (int)cl.block_rank() * PG_THREADS + threadIdx.x;
    for (int64_t i = t0; i < a.num_copies; i += PG_CTAS * PG_THREADS) {
        const int32_t d = a.copy_dst[i];
        if (d >= 0 && d < a.num_pages) a.list_a[d] = INT32_MAX;
    }
    cl.sync();
    for (int64_t i = t0; i < a.num_copies; i += PG_CTAS * PG_THREADS) {
        const int32_t d = a.copy_dst[i], s = a.copy_src[i];
        if (d >= 0 && d < a.num_pages) atomicMin(a.list_a + d, (int32_t)i);
        if (a.one_pool && s >= 0 && s < a.num_pages) atomicMin(a.list_a + s, -1);
    }
}

__global__ void __launch_bounds__(PG_BLOCK) k_apply_copy(const PageArgs a) {
    pdl_wait();
    const int pieces = page_pieces(a);
    for (int64_t it = blockIdx.x; it < (int64_t)a.num_copies * pieces; it += gridDim.x) {
        const int i = (int)(it / pieces), piece = (int)(it % pieces);
        const int32_t s = a.copy_src[i], d = a.copy_dst[i];
        unsigned bad = 0;
        if (s < 0 || s >= a.src_pages || d < 0 || d >= a.num_pages) bad = VX_DATA_BAD_PAGE_ID;
        else if (a.list_a[d] != i) bad = VX_DATA_BAD_COPY;
        if (bad) {
            if (piece == 0 && threadIdx.x == 0) set_err(a.err, bad);
            continue;
        }
        copy_piece(a, s, d, piece);
    }
}

// ------------------------------------------------------------------ new rows

// Shared arrays of the planner, PG_MAX_ROWS ints each
struct UpdateShared {
    int32_t *first;  // [old rows] lowest child, INT32_MAX: none
    int32_t *kids;   // [old rows] children
    int32_t *off;    // [new rows] rank of the row's first fresh page
    int32_t *held;   // [new rows] pages taken over from the parent (its last one excluded when copied)
};

// What the applier needs: head[0] 1 (apply) or 0 (refused); list_a[i] the fresh page that takes
// the copy of new row i's last page, or -1; list_b[b] the change of the references to old row
// b's whole pages, list_c[b] to its partly filled last page.
__global__ void __cluster_dims__(PG_CTAS) __launch_bounds__(PG_THREADS) k_plan_update(const PageArgs a) {
    extern __shared__ int32_t s_rows[];
    __shared__ int32_t s_warp[PG_WARPS], s_total;
    __shared__ long long s_scan[PG_WARPS];
    __shared__ unsigned s_bad;
    pdl_wait();
    pdl_trigger();
    cg::cluster_group cl = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool lead = cl.block_rank() == 0;
    const UpdateShared s{s_rows, s_rows + PG_MAX_ROWS, s_rows + 2 * PG_MAX_ROWS, s_rows + 3 * PG_MAX_ROWS};
    if (tid == 0) s_bad = 0;
    for (int b = tid; b < a.B; b += PG_THREADS) {
        s.first[b] = INT32_MAX;
        s.kids[b] = 0;
    }
    __syncthreads();
    // ---- rows (every CTA does all of them: each needs the offsets)
    unsigned bad = 0;
    for (int i = tid; i < a.new_rows; i += PG_THREADS) {
        const int32_t p = a.parent[i];
        if (p < -1 || p >= a.B) bad |= VX_DATA_BAD_ROW;
        else if (p >= 0) {
            atomicMin(s.first + p, i);
            atomicAdd(s.kids + p, 1);
        }
    }
    for (int b = tid; b < a.B; b += PG_THREADS) {
        const int32_t L = a.seq_lens[b];
        if (L < 0 || L > a.max_pages * a.P) bad |= VX_DATA_BAD_SEQ_LEN;
    }
    if (bad) atomicOr(&s_bad, bad);
    __syncthreads();
    const bool sound = s_bad == 0;
    // rows in order: thread t takes rows [t * per, (t + 1) * per)
    const int per = ceil_div(a.new_rows, PG_THREADS);
    long long mine = 0;
    bad = 0;
    if (sound) {
        for (int i = tid * per; i < min(a.new_rows, (tid + 1) * per); ++i) {
            const int32_t p = a.parent[i], g = a.grow[i];
            const int32_t L = p >= 0 ? a.seq_lens[p] : 0;
            const int32_t n = ceil_div(L, a.P);
            bool copy = false;
            if (L % a.P) {
                const int32_t tail = a.page_indices[a.page_ptr[p] + n - 1];
                if (tail < 0 || tail >= a.num_pages) bad |= VX_DATA_BAD_PAGE_ID;
                else copy = !(s.first[p] == i && a.ref_in[tail] == 1);
            }
            const int64_t L2 = (int64_t)L + g;
            if (g < 0 || L2 > (int64_t)a.new_max_pages * a.P) {
                bad |= VX_DATA_BAD_SEQ_LEN;
                continue;
            }
            const int32_t n2 = (int32_t)((L2 + a.P - 1) / a.P);
            const int32_t to = a.new_ptr[i];
            if (to < 0 || (int64_t)to + n2 > a.num_indices) bad |= VX_DATA_BAD_ROW;
            s.off[i] = (n2 - n + (copy ? 1 : 0));
            s.held[i] = n - (copy ? 1 : 0);
            mine += s.off[i];
            if (lead) {
                a.list_a[i] = -1;
                if (p >= 0 && s.first[p] == i) a.list_c[p] = copy ? -1 : 0;
            }
        }
    }
    if (bad) atomicOr(&s_bad, bad);
    // exclusive prefix of the rows' fresh pages
    long long x = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long y = __shfl_up_sync(FULL, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    long long before = x - mine, need = 0;
    for (int w = 0; w < PG_WARPS; ++w) {
        if (w < warp) before += s_scan[w];
        need += s_scan[w];
    }
    const unsigned rows_bad = s_bad;
    if (!rows_bad) {
        for (int i = tid * per; i < min(a.new_rows, (tid + 1) * per); ++i) {
            const int c = s.off[i];
            s.off[i] = (int32_t)min(before, (long long)INT32_MAX);
            before += c;
        }
    }
    // ---- the pool: copy the counts, find the free pages
    int64_t nfree = 0;
    int64_t rank0 = cluster_base<false>(a.ref_in, a.num_pages, s_warp, &s_total, nfree, [&](int64_t at, const int4 &v) {
        if (a.ref_out == a.ref_in) return;
        if (at + 4 <= a.num_pages) *reinterpret_cast<int4 *>(a.ref_out + at) = v;
        else {
            if (at < a.num_pages) a.ref_out[at] = v.x;
            if (at + 1 < a.num_pages) a.ref_out[at + 1] = v.y;
            if (at + 2 < a.num_pages) a.ref_out[at + 2] = v.z;
        }
    });
    const unsigned all_bad = rows_bad | (!rows_bad && need > nfree ? VX_DATA_NO_PAGES : 0u);
    if (lead) {
        if (tid == 0) {
            a.head[0] = all_bad ? 0 : 1;
            if (all_bad) set_err(a.err, all_bad);
        }
        for (int i = tid; i < a.new_rows; i += PG_THREADS) {
            const int32_t p = a.parent[i];
            a.new_lens[i] = all_bad ? 0 : (p >= 0 ? a.seq_lens[p] : 0) + a.grow[i];
        }
        for (int b = tid; b < a.B; b += PG_THREADS) {
            a.list_b[b] = s.kids[b] - 1;
            if (s.kids[b] == 0) a.list_c[b] = -1;
        }
    }
    if (!all_bad) {
        // ---- hand the lowest `need` free pages to the rows
        const int64_t span = warp_span(a.num_pages), p0 = ((int64_t)cl.block_rank() * PG_WARPS + warp) * span;
        for (int64_t o = 0; o < span && rank0 < need; o += 128) {
            const int64_t at = p0 + o + lane * 4;
            const uint32_t f = flags4<false>(load4(a.ref_in, at, a.num_pages, -1), at, a.num_pages);
            int total;
            int64_t r = rank0 + lane_rank(f, lane, total);
            rank0 += total;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!((f >> e) & 1u)) continue;
                if (r < need) {
                    const int32_t id = (int32_t)(at + e);
                    int lo = 0, hi = a.new_rows - 1;  // the last row with off <= r
                    while (lo < hi) {
                        const int mid = (lo + hi + 1) >> 1;
                        if (s.off[mid] <= r) lo = mid;
                        else hi = mid - 1;
                    }
                    const int32_t k = (int32_t)r - s.off[lo], p = a.parent[lo];
                    a.new_indices[a.new_ptr[lo] + s.held[lo] + k] = id;
                    if (k == 0 && p >= 0 && s.held[lo] < ceil_div(a.seq_lens[p], a.P)) a.list_a[lo] = id;
                    a.ref_out[id] = 1;
                }
                ++r;
            }
        }
    }
    cl.sync();  // no CTA leaves while another may still read its total
}

__global__ void __launch_bounds__(PG_BLOCK) k_apply_update(const PageArgs a) {
    pdl_wait();
    if (a.head[0] == 0) return;
    const int pieces = page_pieces(a);
    const int spans = ceil_div(a.max_pages, PG_SPAN);
    const int64_t copies = (int64_t)a.new_rows * pieces, rows = (int64_t)a.new_rows * spans,
                  refs = (int64_t)a.B * spans;
    for (int64_t it = blockIdx.x; it < copies + rows + refs; it += gridDim.x) {
        if (it < copies) {  // the copy of a forked row's last page
            const int i = (int)(it / pieces);
            const int32_t d = a.list_a[i];
            if (d < 0) continue;
            const int32_t p = a.parent[i];
            const int32_t src = a.page_indices[a.page_ptr[p] + a.seq_lens[p] / a.P];
            copy_piece(a, src, d, (int)(it % pieces));
        } else if (it < copies + rows) {  // entries taken over from the parent
            const int i = (int)((it - copies) / spans), j0 = (int)((it - copies) % spans) * PG_SPAN;
            const int32_t p = a.parent[i];
            if (p < 0) continue;
            const int held = ceil_div(a.seq_lens[p], a.P) - (a.list_a[i] >= 0 ? 1 : 0);
            const int32_t *from = a.page_indices + a.page_ptr[p];
            int32_t *to = a.new_indices + a.new_ptr[i];
            for (int j = j0 + threadIdx.x; j < min(held, j0 + PG_SPAN); j += PG_BLOCK) to[j] = from[j];
        } else {  // references of an old row's pages
            const int b = (int)((it - copies - rows) / spans), j0 = (int)((it - copies - rows) % spans) * PG_SPAN;
            const int32_t L = a.seq_lens[b], whole = L / a.P, n = ceil_div(L, a.P);
            const int dw = a.list_b[b], dt = a.list_c[b];
            if (dw == 0 && (dt == 0 || n == whole)) continue;
            const int32_t *from = a.page_indices + a.page_ptr[b];
            for (int j = j0 + threadIdx.x; j < min(n, j0 + PG_SPAN); j += PG_BLOCK) {
                const int32_t id = from[j];
                if (id < 0 || id >= a.num_pages) set_err(a.err, VX_DATA_BAD_PAGE_ID);
                else if (const int d = j < whole ? dw : dt) atomicAdd(a.ref_out + id, d);
            }
        }
    }
}

// ------------------------------------------------------------------ compaction

// list_a[i]: the i-th free page below n; list_b[r], list_c[r]: id and references of the r-th
// live page (r >= head[0] only: those with id >= n); head[1]: moves.  Move i takes page
// list_b[head[0] + i] to list_a[i].
__global__ void __cluster_dims__(PG_CTAS) __launch_bounds__(PG_THREADS) k_plan_compact(const PageArgs a) {
    __shared__ int32_t s_warp[PG_WARPS], s_total;
    pdl_wait();
    pdl_trigger();
    cg::cluster_group cl = cg::this_cluster();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t n = 0;
    int64_t rank0 = cluster_base<true>(a.ref_in, a.num_pages, s_warp, &s_total, n, [](int64_t, const int4 &) {});
    const int64_t span = warp_span(a.num_pages), p0 = ((int64_t)cl.block_rank() * PG_WARPS + warp) * span;
#pragma unroll 2
    for (int64_t o = 0; o < span; o += 128) {
        const int64_t at = p0 + o + lane * 4;
        const int4 v = load4(a.ref_in, at, a.num_pages, 0);
        const int ref[4] = {v.x, v.y, v.z, v.w};
        const uint32_t f = flags4<true>(v, at, a.num_pages);
        int total;
        int64_t r = rank0 + lane_rank(f, lane, total);  // live pages before this one
        rank0 += total;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int64_t p = at + e;
            if (p >= a.num_pages) break;
            const bool live = (f >> e) & 1u;
            if (p == n) a.head[0] = (int32_t)r;
            if (p >= n) {
                if (live) {
                    a.list_b[r] = (int32_t)p;
                    a.list_c[r] = ref[e];
                } else {
                    a.remap[p] = -1;
                }
                a.ref_out[p] = 0;
            } else if (live) {
                a.remap[p] = (int32_t)p;
                a.ref_out[p] = ref[e];
            } else {
                a.list_a[p - r] = (int32_t)p;
                a.remap[p] = -1;
            }
            r += live;
        }
    }
    if (n == a.num_pages && cl.block_rank() == 0 && threadIdx.x == 0) a.head[0] = (int32_t)n;
    cl.sync();
    const int32_t low = *reinterpret_cast<volatile int32_t *>(a.head), moves = (int32_t)n - low;
    if (cl.block_rank() == 0 && threadIdx.x == 0) {
        a.head[1] = moves;
        *a.num_live = (int32_t)n;
    }
    for (int i = (int)cl.block_rank() * PG_THREADS + threadIdx.x; i < moves; i += PG_CTAS * PG_THREADS) {
        const int32_t d = a.list_a[i];
        a.remap[a.list_b[low + i]] = d;
        a.ref_out[d] = a.list_c[low + i];
    }
    cl.sync();
}

__global__ void __launch_bounds__(PG_BLOCK) k_apply_compact(const PageArgs a) {
    pdl_wait();
    const int pieces = page_pieces(a);
    const int spans = ceil_div(a.max_pages, PG_SPAN);
    const int32_t low = a.head[0], moves = a.head[1];
    const int64_t copies = (int64_t)moves * pieces, rows = (int64_t)a.B * spans;
    for (int64_t it = blockIdx.x; it < copies + rows; it += gridDim.x) {
        if (it < copies) {
            const int i = (int)(it / pieces);
            copy_piece(a, a.list_b[low + i], a.list_a[i], (int)(it % pieces));
        } else {
            const int b = (int)((it - copies) / spans), j0 = (int)((it - copies) % spans) * PG_SPAN;
            const int32_t L = a.seq_lens[b];
            if (L < 0 || L > a.max_pages * a.P) {
                if (j0 == 0 && threadIdx.x == 0) set_err(a.err, VX_DATA_BAD_SEQ_LEN);
                continue;
            }
            const int n = ceil_div(L, a.P);
            const int64_t at = a.page_ptr[b];
            for (int j = j0 + threadIdx.x; j < min(n, j0 + PG_SPAN); j += PG_BLOCK) {
                const int32_t id = a.page_indices[at + j];
                int32_t to = id >= 0 && id < a.num_pages ? a.remap[id] : -1;
                if (to < 0) {
                    set_err(a.err, VX_DATA_BAD_PAGE_ID);
                    to = id;
                }
                a.indices_out[at + j] = to;
            }
        }
    }
}

// blocks of an applying grid: every item, at most 8 blocks per SM
cudaError_t apply_grid(int64_t items, unsigned *grid) {
    const int sms = current_sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    *grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(items, (int64_t)sms * 8));
    return cudaSuccess;
}

template <typename Plan, typename Apply>
cudaError_t launch_pages(Plan plan, Apply apply, size_t smem, int64_t items, const PageArgs &a, cudaStream_t s) {
    unsigned grid = 0;
    cudaError_t e = apply_grid(items, &grid);
    if (e == cudaSuccess) e = launch_k(plan, dim3(PG_CTAS), dim3(PG_THREADS), smem, s, true, a);
    if (e == cudaSuccess) e = launch_k(apply, dim3(grid), dim3(PG_BLOCK), 0, s, true, a);
    return e;
}

int64_t host_pieces(const PageArgs &a) { return (((int64_t)a.kb + a.vb + a.cb) / 16 + PG_PIECE - 1) / PG_PIECE; }

}  // namespace

cudaError_t launch_copy_pages(const PageArgs &a, cudaStream_t s) {
    return launch_pages(k_plan_copy, k_apply_copy, 0, (int64_t)a.num_copies * host_pieces(a), a, s);
}

cudaError_t launch_update_table(const PageArgs &a, cudaStream_t s) {
    constexpr int smem = 4 * PG_MAX_ROWS * (int)sizeof(int32_t);
    static std::atomic<unsigned long long> done;
    const cudaError_t e = ensure_smem_limit(k_plan_update, smem, done);
    if (e != cudaSuccess) return e;
    const int64_t spans = (a.max_pages + PG_SPAN - 1) / PG_SPAN;
    return launch_pages(k_plan_update, k_apply_update, smem, a.new_rows * host_pieces(a) + (a.new_rows + a.B) * spans, a, s);
}

cudaError_t launch_compact_pages(const PageArgs &a, cudaStream_t s) {
    const int64_t spans = (a.max_pages + PG_SPAN - 1) / PG_SPAN;
    return launch_pages(k_plan_compact, k_apply_compact, 0, a.num_pages / 2 * host_pieces(a) + a.B * spans, a, s);
}

}  // namespace vx
