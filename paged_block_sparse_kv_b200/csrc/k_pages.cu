// k_pages.cu -- pages of a pool: copy, new table rows (fork, free, grow), compaction.
//
// The first kernel of an update or a compaction reads the pool's reference counts once, over the
// whole GPU: a bit per page (free, or live) and the count of each segment of PG_SEG pages.  A
// block of the next kernel takes the segments' prefix sums into shared memory, so a warp that
// looks at a segment's 32 words of bits knows the rank of each of its pages: what is handed out
// or moved depends on the counts alone, never on timing, and no single block has to scan the
// pool (a cluster of 8 blocks that did took 23 us over 290,000 pages).  Every block has one small
// job: these kernels run a few microseconds, and instructions are fetched cold.
// Page data moves in pieces of PG_PIECE 16-byte chunks.  Bound: HBM for page data (read and
// written once), a few dependent loads for the rest.
// Measured on one B200: 8,192 pages of 67.6 KB from pool to pool 179 us (6.2 TB/s, 0.95 of the copy
// peak), a half empty pool of 32,768 such pages compacted in 188 us (5.9 TB/s); 5 pages 3.7 us; new
// rows of 256 requests over 290,000 pages 9.2 us, of 64 beams 7.4 us; 500 latent pages compacted in
// 6.9 us.  Measured and not kept: bulk copies through shared memory (185-189 us in 2-4 blocks of 3 x 16 KB
// per SM, where plain loads took 183), one flat list of all chunks (187), pieces of 1,280 to 2,304
// chunks (179-190 us).
#include <cooperative_groups.h>

#include <algorithm>

#include "vx_internal.h"

namespace cg = cooperative_groups;

namespace vx {

namespace {

constexpr int PG_CTAS = 8;       // CTAs of the copy planner's cluster
constexpr int PG_THREADS = 1024; // threads of a planning block
constexpr int PG_SEG = 1024;     // pages of a segment: 32 words of bits, one 128-byte line
constexpr int PG_GROUPS = 1024;  // prefix sums a block keeps (a segment each in pools of 2^20 pages)
constexpr int PG_MAX_ROWS = 4096;
constexpr int PG_PIECE = 1024;   // 16-byte chunks of a page moved by one block at a time
constexpr int PG_SPAN = 256;     // table entries handled by one warp, 8 per lane
constexpr int PG_BLOCK = 256;    // threads of an applying block
constexpr int PG_RANKS = PG_BLOCK / 32 / 4 * PG_SEG;  // pages that a block handing out fresh ones looks at
// Copies up to which every block checks its own pair (k_copy_few) instead of a planner checking all:
// us with and without the planner: 5 pages of 35 KB 4.3 and 2.4, 256 6.4 and 5.3, 512 10.8 and 9.9, 1,024
// 18.3 and 18.6, 4,096 55.7 and 81.6.
constexpr int PG_FEW = 512;

// ------------------------------------------------------------------ flags and ranks

// Flags of a planning block's 4 * PG_THREADS pages from p0: ref > 0 when LIVE, ref == 0 otherwise,
// none past the pool; list_a[p / 32] holds the bits, list_b[p / PG_SEG] the segments' counts.  With
// `out` the reference counts are copied there.
template <bool LIVE>
__device__ __forceinline__ void flag_pages(const PageArgs &a, int64_t p0, int32_t *out) {
    __shared__ int32_t s_count[PG_THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t at = p0 + (int64_t)tid * 4, n = a.num_pages;
    int4 v = make_int4(-1, -1, -1, -1);
    if (at + 4 <= n) {
        v = *reinterpret_cast<const int4 *>(a.ref_in + at);
        if (out) *reinterpret_cast<int4 *>(out + at) = v;
    } else {
        int32_t *w[3] = {&v.x, &v.y, &v.z};
#pragma unroll
        for (int e = 0; e < 3; ++e)
            if (at + e < n) {
                *w[e] = a.ref_in[at + e];
                if (out) out[at + e] = *w[e];
            }
    }
    const int r[4] = {v.x, v.y, v.z, v.w};
    uint32_t f = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) f |= (LIVE ? r[e] > 0 : r[e] == 0) ? 1u << e : 0u;
    const int count = __reduce_add_sync(FULL, __popc(f));
    f <<= 4 * (lane & 7);
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) f |= __shfl_xor_sync(FULL, f, off);
    if ((lane & 7) == 0 && at < (n + PG_SEG - 1) / PG_SEG * PG_SEG) a.list_a[at / 32] = (int32_t)f;
    if (lane == 0) s_count[tid >> 5] = count;
    __syncthreads();
    constexpr int PER = PG_SEG / 128;  // warps of a segment
    if (tid < PG_THREADS / 32 / PER && p0 + (int64_t)tid * PG_SEG < n) {
        int c = 0;
#pragma unroll
        for (int w = 0; w < PER; ++w) c += s_count[tid * PER + w];
        a.list_b[p0 / PG_SEG + tid] = c;
    }
}

// A block's view of the flags: prefix sums of groups of `g` segments in shared memory.
struct PoolRanks {
    const int32_t *bits, *counts;
    const uint32_t *pre;  // [groups + 1], shared
    int32_t segs, g, groups;

    __device__ __forceinline__ PoolRanks(const PageArgs &a, const uint32_t *s_pre)
        : bits(a.list_a), counts(a.list_b), pre(s_pre) {
        segs = (int)((a.num_pages + PG_SEG - 1) / PG_SEG);
        g = segs <= PG_GROUPS ? 1 : ceil_div(segs, PG_GROUPS);
        groups = g == 1 ? segs : ceil_div(segs, g);
    }
    // the prefix sums, by the whole block
    __device__ __forceinline__ void sum(uint32_t *s_pre, uint32_t *s_warp) const {
        // thread t sums groups [t * per, (t + 1) * per)
        const int per = ceil_div(groups, PG_BLOCK), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        const int k0 = min(groups, (int)threadIdx.x * per), k1 = min(groups, k0 + per);
        uint32_t mine = 0;
#pragma unroll 1
        for (int k = k0; k < k1; ++k) {
            s_pre[k] = mine;
#pragma unroll 1
            for (int s = k * g; s < min(segs, (k + 1) * g); ++s) mine += (uint32_t)counts[s];
        }
        uint32_t x = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(FULL, x, off);
            if (lane >= off) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        uint32_t before = x - mine;
#pragma unroll 1
        for (int w = 0; w < warp; ++w) before += s_warp[w];
#pragma unroll 1
        for (int k = k0; k < k1; ++k) s_pre[k] += before;
        if (threadIdx.x == PG_BLOCK - 1) s_pre[groups] = before + mine;
        __syncthreads();
    }
    __device__ __forceinline__ uint32_t total() const { return pre[groups]; }
    // flagged pages before segment `seg`
    __device__ __forceinline__ uint32_t before_segment(int seg) const {
        const int k = g == 1 ? seg : seg / g;
        uint32_t r = pre[k];
#pragma unroll 1
        for (int s = k * g; s < seg; ++s) r += (uint32_t)counts[s];
        return r;
    }
    // By a whole warp: lane l's word of segment `seg` and the flagged pages before that word
    __device__ __forceinline__ uint32_t segment_word(int seg, int lane, uint32_t &rank) const {
        const uint32_t w = (uint32_t)bits[(int64_t)seg * 32 + lane], c = __popc(w);
        uint32_t x = c;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const uint32_t y = __shfl_up_sync(FULL, x, off);
            if (lane >= off) x += y;
        }
        rank = before_segment(seg) + x - c;
        return w;
    }
    // By a whole warp: the flagged page of rank r (below the total)
    __device__ __forceinline__ uint32_t page_of(uint32_t r, int lane) const {
        int lo = 0, hi = groups - 1;  // the last group with at most r before it
#pragma unroll 1
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (pre[mid] <= r) lo = mid;
            else hi = mid - 1;
        }
        int seg = lo * g;
        if (g > 1) {
#pragma unroll 1
            while (before_segment(seg) + (uint32_t)counts[seg] <= r) ++seg;
        }
        uint32_t rank;
        uint32_t w = segment_word(seg, lane, rank);
        const bool mine = r >= rank && r - rank < (uint32_t)__popc(w);
        const int src = __ffs(__ballot_sync(FULL, mine)) - 1;
        w = __shfl_sync(FULL, w, src);
#pragma unroll 1
        for (rank = r - __shfl_sync(FULL, rank, src); rank > 0; --rank) w &= w - 1;
        return (uint32_t)seg * PG_SEG + src * 32 + __ffs(w) - 1;
    }
};

// ------------------------------------------------------------------ page data

// 16-byte chunks of one page over all arrays, and its pieces
__device__ __forceinline__ int page_chunks(const PageArgs &a) { return (a.kb + a.vb + a.cb) >> 4; }
__device__ __forceinline__ int page_pieces(const PageArgs &a) { return ceil_div(page_chunks(a), PG_PIECE); }

__device__ __forceinline__ void copy_piece(const PageArgs &a, int64_t src, int64_t dst, int piece) {
    const int nk = a.kb >> 4, nv = a.vb >> 4, nc = a.cb >> 4;
    constexpr int U = PG_PIECE / PG_BLOCK;
    uint4 v[U];
    uint8_t *to[U];
    // equal pieces (to a warp's 32 chunks): a short last one would cost a block as much as a whole one
    const int size = (ceil_div(page_chunks(a), page_pieces(a)) + 31) & ~31;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int k = u * PG_BLOCK + (int)threadIdx.x;
        int c = k < size ? piece * size + k : INT32_MAX;
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
    const uint32_t pieces = page_pieces(a);
    for (uint32_t it = blockIdx.x; it < (uint32_t)a.num_copies * pieces; it += gridDim.x) {
        const int i = it / pieces, piece = it - i * pieces;
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

// Few copies: every block looks for its own pair's rivals itself, and the planner is saved.
__global__ void __launch_bounds__(PG_BLOCK) k_copy_few(const PageArgs a) {
    pdl_wait();
    const uint32_t pieces = page_pieces(a);
    for (uint32_t it = blockIdx.x; it < (uint32_t)a.num_copies * pieces; it += gridDim.x) {
        const int i = it / pieces, piece = it - i * pieces;
        const int32_t s = a.copy_src[i], d = a.copy_dst[i];
        bool rival = false;
        for (int j = threadIdx.x; j < a.num_copies; j += PG_BLOCK)
            rival |= (j < i && a.copy_dst[j] == d) || (a.one_pool && a.copy_src[j] == d);
        rival = __syncthreads_or(rival);
        unsigned bad = 0;
        if (s < 0 || s >= a.src_pages || d < 0 || d >= a.num_pages) bad = VX_DATA_BAD_PAGE_ID;
        else if (rival) bad = VX_DATA_BAD_COPY;
        if (bad) {
            if (piece == 0 && threadIdx.x == 0) set_err(a.err, bad);
            continue;
        }
        copy_piece(a, s, d, piece);
    }
}

// ------------------------------------------------------------------ new rows

// Block 0 plans the rows, the others flag the free pages.  What the rows' plan leaves: head[0] the
// error bits found, head[1] the pages needed (at most 2^31 - 1); list_d[b] 2 * (children of old
// row b) + (1 when its first child keeps its partly filled last page); for new row i its length
// and list_c[i]:
struct RowPlan {
    int32_t off;   // rank of its first fresh page among the free ones
    int32_t held;  // entries taken over from the parent
    int32_t from;  // where they start in page_indices
    int32_t tail;  // the page that its first fresh page takes a copy of, or -1
};
__global__ void __launch_bounds__(PG_THREADS) k_plan_update(const PageArgs a) {
    pdl_wait();
    pdl_trigger();
    if (blockIdx.x > 0) {
        flag_pages<false>(a, (int64_t)(blockIdx.x - 1) * PG_THREADS * 4, a.ref_out != a.ref_in ? a.ref_out : nullptr);
        return;
    }
    __shared__ int32_t s_first[PG_MAX_ROWS];  // [old rows] lowest child, INT32_MAX: none
    __shared__ int32_t s_kids[PG_MAX_ROWS];   // [old rows] as list_d
    __shared__ long long s_scan[PG_THREADS / 32];
    __shared__ unsigned s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int log2_p = __ffs(a.P) - 1;
    const int per = ceil_div(a.new_rows, PG_THREADS);  // rows [tid * per, (tid + 1) * per) are this thread's
    const int row0 = tid * per, row1 = min(a.new_rows, row0 + per);
    struct Row {
        int32_t p, g, to, L, n, from, tail, tail_ref;
    };
    auto load_row = [&](int i) {
        Row r{a.parent[i], a.grow[i], a.new_ptr[i], 0, 0, 0, -1, 0};
        if (r.p >= 0 && r.p < a.B) {
            r.L = a.seq_lens[r.p];
            if (r.L < 0 || r.L > a.max_pages * a.P) r.L = 0;  // refused below
            r.from = a.page_ptr[r.p];
            r.n = (r.L + a.P - 1) >> log2_p;
            if (r.L & (a.P - 1)) {
                r.tail = a.page_indices[r.from + r.n - 1];
                if (r.tail >= 0 && r.tail < a.num_pages) r.tail_ref = a.ref_in[r.tail];
            }
        }
        return r;
    };
    Row first_row{};
    if (row0 < row1) first_row = load_row(row0);
    if (tid == 0) s_bad = 0;
    unsigned bad = 0;
    for (int b = tid; b < a.B; b += PG_THREADS) {
        s_first[b] = INT32_MAX;
        s_kids[b] = 0;
        const int32_t L = a.seq_lens[b];
        if (L < 0 || L > a.max_pages * a.P) bad |= VX_DATA_BAD_SEQ_LEN;
    }
    __syncthreads();
    for (int i = row0; i < row1; ++i) {
        const int32_t p = i == row0 ? first_row.p : a.parent[i];
        if (p < -1 || p >= a.B) bad |= VX_DATA_BAD_ROW;
        else if (p >= 0) {
            atomicMin(s_first + p, i);
            atomicAdd(s_kids + p, 2);
        }
    }
    __syncthreads();
    auto fresh = [&](int i, const Row &r, bool &copy) -> int32_t {  // pages new row i needs
        copy = r.tail >= 0 && !(s_first[r.p] == i && r.tail_ref == 1);
        const int64_t L2 = (int64_t)r.L + r.g;
        if (r.g < 0 || L2 > (int64_t)a.new_max_pages * a.P) {
            bad |= VX_DATA_BAD_SEQ_LEN;
            return 0;
        }
        const int32_t n2 = (int32_t)((L2 + a.P - 1) >> log2_p);
        if (r.to < 0 || (int64_t)r.to + n2 > a.num_indices) bad |= VX_DATA_BAD_ROW;
        // (a last page that is free would be handed out while its row still holds it)
        if (r.L & (a.P - 1) && r.tail_ref < 1) bad |= VX_DATA_BAD_PAGE_ID;
        return n2 - r.n + (copy ? 1 : 0);
    };
    long long mine = 0;
    bool first_copy = false;
    int32_t first_need = 0;
    for (int i = row0; i < row1; ++i) {
        const Row r = i == row0 ? first_row : load_row(i);
        bool copy;
        const int32_t c = fresh(i, r, copy);
        if (i == row0) {
            first_copy = copy;
            first_need = c;
        }
        mine += c;
        if (r.tail >= 0 && !copy) s_kids[r.p] |= 1;  // the first child alone
    }
    if (bad) atomicOr(&s_bad, bad);
    // exclusive prefix of the rows' fresh pages
    auto scan = [&](long long v) {  // inclusive, over a warp
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long y = __shfl_up_sync(FULL, v, off);
            if (lane >= off) v += y;
        }
        return v;
    };
    const long long x = scan(mine);
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    const long long w = scan(s_scan[lane]);  // every warp for itself: PG_THREADS is 32 warps
    const long long need = __shfl_sync(FULL, w, 31), warp_before = __shfl_sync(FULL, w, (warp + 31) & 31);
    long long before = x - mine + (warp > 0 ? warp_before : 0);
    if (tid == 0) {
        a.head[0] = (int32_t)s_bad;
        a.head[1] = (int32_t)min(need, (long long)INT32_MAX);
    }
    for (int i = row0; i < row1; ++i) {
        const Row r = i == row0 ? first_row : load_row(i);
        bool copy = first_copy;
        const int32_t c = i == row0 ? first_need : fresh(i, r, copy);
        reinterpret_cast<RowPlan *>(a.list_c)[i] = {(int32_t)before, r.n - (copy ? 1 : 0), r.from, copy ? r.tail : -1};
        a.new_lens[i] = r.L + r.g;  // zeroed by the applier when the call is refused
        before += c;
    }
    for (int b = tid; b < a.B; b += PG_THREADS) a.list_d[b] = s_kids[b];
}

// Blocks of the second kernel by job, in this order, and what one of them is divided into (32-bit:
// a 64-bit division costs as much as the rest of a block's address arithmetic)
struct UpdateJobs {
    uint32_t copies, fresh, rows, refs;
    uint32_t spans, pieces;
};
// false: more blocks or warps than 2^31
__host__ __forceinline__ bool update_jobs(const PageArgs &a, UpdateJobs *j) {
    constexpr int64_t W = PG_BLOCK / 32;
    const int64_t segs = (a.num_pages + PG_SEG - 1) / PG_SEG;
    const int64_t spans = (a.max_pages + PG_SPAN - 1) / PG_SPAN;
    const int64_t pieces = (((int64_t)a.kb + a.vb + a.cb) / 16 + PG_PIECE - 1) / PG_PIECE;
    const int64_t n[4] = {a.new_rows * pieces, (segs * 4 + W - 1) / W, (a.new_rows * spans + W - 1) / W,
                          (a.B * spans + W - 1) / W};
    *j = {(uint32_t)n[0], (uint32_t)n[1], (uint32_t)n[2], (uint32_t)n[3], (uint32_t)spans, (uint32_t)pieces};
    return (n[0] + n[1] + n[2] + n[3]) * W <= INT32_MAX;
}

__global__ void __launch_bounds__(PG_BLOCK) k_apply_update(const PageArgs a, const UpdateJobs jobs) {
    __shared__ uint32_t s_pre[PG_GROUPS + 1], s_warp[PG_BLOCK / 32];
    __shared__ int32_t s_row[PG_RANKS];  // fresh pages: the new row of a rank
    extern __shared__ int32_t s_to[];    // [new_rows]
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    const RowPlan *plans = reinterpret_cast<const RowPlan *>(a.list_c);
    // the block's job, and what its warp works on: a quarter of a segment, a span of a new or an old
    // row, or a piece of a page.  What can be loaded is on its way before the ranks are summed.
    uint32_t job = blockIdx.x;
    const bool is_copy = job < jobs.copies, is_fresh = !is_copy && (job -= jobs.copies) < jobs.fresh,
               is_row = !is_copy && !is_fresh && (job -= jobs.fresh) < jobs.rows;
    if (!is_copy && !is_fresh && !is_row) job -= jobs.rows;
    const uint32_t unit = job * (PG_BLOCK / 32) + (tid >> 5);
    RowPlan plan{0, 0, 0, -1};
    int at = 0, item = 0, j0 = 0, kids = 0, L = 0;
    if (is_copy) {
        item = job / jobs.pieces;
        plan = plans[item];
    } else if (is_row) {
        item = unit / jobs.spans;
        j0 = (unit - item * jobs.spans) * PG_SPAN;
        if (item < a.new_rows) {
            plan = plans[item];
            at = a.new_ptr[item];
        }
    } else if (!is_fresh) {
        item = unit / jobs.spans;
        j0 = (unit - item * jobs.spans) * PG_SPAN;
        if (item < a.B) {
            L = a.seq_lens[item];
            at = a.page_ptr[item];
            kids = a.list_d[item];
        }
    }
    const uint32_t need = (uint32_t)a.head[1];
    const unsigned row_bad = (unsigned)a.head[0];
    PoolRanks free_pages(a, s_pre);
    uint32_t total;
    if (is_copy || is_fresh) {
        free_pages.sum(s_pre, s_warp);
        total = free_pages.total();
    } else {  // the total alone, without a barrier
        uint32_t c = 0;
        for (int s = lane; s < free_pages.segs; s += 32) c += (uint32_t)free_pages.counts[s];
        total = __reduce_add_sync(FULL, c);
    }
    const unsigned bad = row_bad ? row_bad : need > total ? VX_DATA_NO_PAGES : 0u;
    if (bad) {
        for (uint32_t i = blockIdx.x * PG_BLOCK + tid; i < (uint32_t)a.new_rows; i += gridDim.x * PG_BLOCK) a.new_lens[i] = 0;
        if (blockIdx.x == 0 && tid == 0) set_err(a.err, bad);
        return;
    }
    if (is_copy) {  // of a forked row's last page
        if (plan.tail >= 0)
            copy_piece(a, plan.tail, free_pages.page_of((uint32_t)plan.off, lane), job - item * jobs.pieces);
    } else if (is_row) {  // entries taken over from the parent
        int32_t id[PG_SPAN / 32];
        bool bad_id = false;
#pragma unroll
        for (int u = 0; u < PG_SPAN / 32; ++u) {
            const int j = j0 + 32 * u + lane;
            id[u] = j < plan.held ? a.page_indices[plan.from + j] : 0;
            bad_id |= id[u] < 0 || id[u] >= a.num_pages;
        }
        if (bad_id) set_err(a.err, VX_DATA_BAD_PAGE_ID);
#pragma unroll
        for (int u = 0; u < PG_SPAN / 32; ++u) {
            const int j = j0 + 32 * u + lane;
            if (j < plan.held) a.new_indices[at + j] = id[u];
        }
    } else if (!is_fresh) {  // references of an old row's pages
        const int log2_p = __ffs(a.P) - 1;
        const int32_t whole = L >> log2_p, n = (L + a.P - 1) >> log2_p;
        const int dw = (kids >> 1) - 1, dt = (kids & 1) - 1;
        if (j0 >= n || (dw == 0 && (dt == 0 || n == whole))) return;
#pragma unroll 4
        for (int j = j0 + lane; j < min(n, j0 + PG_SPAN); j += 32) {
            const int32_t id = a.page_indices[at + j];
            if (id < 0 || id >= a.num_pages) set_err(a.err, VX_DATA_BAD_PAGE_ID);
            else if (const int d = j < whole ? dw : dt) atomicAdd(a.ref_out + id, d);
        }
    } else {  // the lowest `need` free pages to the rows in order
        // this block's segments have ranks [r0, r0 + PG_RANKS); which row each belongs to: every row
        // marks its first rank, and a running maximum fills the rest
        const int first = (int)(job * (PG_BLOCK / 32) / 4);
        const uint32_t r0 = free_pages.before_segment(min(first, free_pages.segs - 1));
        if (r0 >= need) return;
        for (int e = tid; e < PG_RANKS; e += PG_BLOCK) s_row[e] = 0;
        __syncthreads();
        for (int i = tid; i < a.new_rows; i += PG_BLOCK) {
            const RowPlan p = plans[i];
            s_to[i] = a.new_ptr[i] + p.held - p.off;  // place of rank 0 in new_indices
            const int64_t d = (int64_t)p.off - r0;
            if (d < PG_RANKS) atomicMax(&s_row[d > 0 ? d : 0], i);
        }
        __syncthreads();
        constexpr int PER = PG_RANKS / PG_BLOCK;
        int32_t top[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) top[e] = max(s_row[tid * PER + e], e > 0 ? top[e - 1] : 0);
        int32_t x = top[PER - 1];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t y = __shfl_up_sync(FULL, x, off);
            if (lane >= off) x = max(x, y);
        }
        if (lane == 31) s_warp[tid >> 5] = (uint32_t)x;
        x = __shfl_up_sync(FULL, x, 1);
        if (lane == 0) x = 0;
        __syncthreads();
        for (int w = 0; w < (tid >> 5); ++w) x = max(x, (int32_t)s_warp[w]);
#pragma unroll
        for (int e = 0; e < PER; ++e) s_row[tid * PER + e] = max(top[e], x);
        __syncthreads();
        const int seg = (int)(unit / 4), w0 = (int)(unit % 4) * 8;
        if (seg >= free_pages.segs) return;
        uint32_t rank0;
        const uint32_t words = free_pages.segment_word(seg, lane, rank0);
#pragma unroll 1
        for (int w = w0; w < w0 + 8; ++w) {
            const uint32_t f = __shfl_sync(FULL, words, w);
            const uint32_t r = __shfl_sync(FULL, rank0, w) + __popc(f & ((1u << lane) - 1u));
            if (!((f >> lane) & 1u) || r >= need) continue;
            const int32_t page = seg * PG_SEG + w * 32 + lane;
            a.new_indices[s_to[s_row[r - r0]] + (int32_t)r] = page;
            a.ref_out[page] = 1;
        }
    }
}

// ------------------------------------------------------------------ compaction

__global__ void __launch_bounds__(PG_THREADS) k_plan_compact(const PageArgs a) {
    pdl_wait();
    pdl_trigger();
    flag_pages<true>(a, (int64_t)blockIdx.x * PG_THREADS * 4, a.ref_out != a.ref_in ? a.ref_out : nullptr);
}

// With n live pages, `low` of them below page n: move i takes the live page of rank low + i to the
// free page of rank i.  list_e[i] is the one, list_f[i] the other; remap[p] of a page that moves is
// -2 - i until the move writes its new id; head[0] the moves.
__global__ void __launch_bounds__(PG_BLOCK) k_list_compact(const PageArgs a) {
    __shared__ uint32_t s_pre[PG_GROUPS + 1], s_warp[PG_BLOCK / 32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    PoolRanks live(a, s_pre);
    live.sum(s_pre, s_warp);
    const uint32_t n = live.total();
    // live pages below page n
    uint32_t low = n;
    if (n < a.num_pages) {
        uint32_t rank;
        const uint32_t w = live.segment_word((int)(n / PG_SEG), lane, rank);
        low = __shfl_sync(FULL, rank + __popc(w & ((1u << (n & 31)) - 1u)), (int)(n / 32) & 31);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.head[0] = (int32_t)(n - low);
        *a.num_live = (int32_t)n;
    }
    const int64_t q = (int64_t)blockIdx.x * (PG_BLOCK / 32) + (threadIdx.x >> 5);
    const int seg = (int)(q / 4), w0 = (int)(q % 4) * 8;
    if (seg >= live.segs) return;
    uint32_t rank0;
    const uint32_t words = live.segment_word(seg, lane, rank0);
#pragma unroll 1
    for (int w = w0; w < w0 + 8; ++w) {
        const uint32_t f = __shfl_sync(FULL, words, w);
        const uint32_t r = __shfl_sync(FULL, rank0, w) + __popc(f & ((1u << lane) - 1u));
        const uint32_t p = (uint32_t)seg * PG_SEG + w * 32 + lane;
        if (p >= a.num_pages) return;
        const bool is_live = (f >> lane) & 1u;
        if (is_live && p >= n) a.list_e[r - low] = (int32_t)p;
        if (!is_live && p < n) a.list_f[p - r] = (int32_t)p;
        a.remap[p] = !is_live ? -1 : p < n ? (int32_t)p : -2 - (int32_t)(r - low);
    }
}

// The lists of k_plan_compact and k_list_compact for pools of at most 4 * PG_THREADS pages, by one
// block and in one launch.
__global__ void __launch_bounds__(PG_THREADS) k_list_small(const PageArgs a) {
    __shared__ int32_t s_sum[PG_THREADS / 32];
    __shared__ int32_t s_low;
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pages = (int)a.num_pages, p0 = tid * 4;
    int32_t ref[4];
    int live = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        ref[e] = p0 + e < pages ? a.ref_in[p0 + e] : 0;
        live += ref[e] > 0;
    }
    auto scan = [&](int v) {  // inclusive, over a warp
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(FULL, v, off);
            if (lane >= off) v += y;
        }
        return v;
    };
    const int x = scan(live);
    if (lane == 31) s_sum[warp] = x;
    __syncthreads();
    const int w = scan(s_sum[lane]);  // every warp for itself: PG_THREADS is 32 warps
    const int n = __shfl_sync(FULL, w, 31);
    const int r0 = x - live + (warp > 0 ? __shfl_sync(FULL, w, (warp + 31) & 31) : 0);
    if (tid == 0 && n == pages) s_low = n;
    int r = r0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (p0 + e == n && n < pages) s_low = r;  // live pages below page n
        r += ref[e] > 0;
    }
    __syncthreads();
    const int low = s_low;
    if (tid == 0) {
        a.head[0] = n - low;
        *a.num_live = n;
    }
    r = r0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int p = p0 + e;
        if (p >= pages) break;
        const bool is_live = ref[e] > 0;
        if (a.ref_out != a.ref_in) a.ref_out[p] = ref[e];
        if (is_live && p >= n) a.list_e[r - low] = p;
        if (!is_live && p < n) a.list_f[p - r] = p;
        a.remap[p] = !is_live ? -1 : p < n ? p : -2 - (r - low);
        r += is_live;
    }
}

// Blocks [0, rows): tables, a warp to PG_SPAN entries; the others: pieces of the moves
__global__ void __launch_bounds__(PG_BLOCK) k_apply_compact(const PageArgs a, const int rows) {
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31;
    if ((int)blockIdx.x < rows) {
        const uint32_t spans = ceil_div(a.max_pages, PG_SPAN);
        const uint32_t it = blockIdx.x * (PG_BLOCK / 32) + (tid >> 5);
        const int b = it / spans, j0 = (it - b * spans) * PG_SPAN;
        if (b >= a.B) return;
        const int32_t L = a.seq_lens[b];
        if (L < 0 || L > a.max_pages * a.P) {
            if (j0 == 0 && lane == 0) set_err(a.err, VX_DATA_BAD_SEQ_LEN);
            return;
        }
        const int n = ceil_div(L, a.P);
        const int64_t at = a.page_ptr[b];
#pragma unroll 4
        for (int j = j0 + lane; j < min(n, j0 + PG_SPAN); j += 32) {
            const int32_t id = a.page_indices[at + j];
            int32_t to = id >= 0 && id < a.num_pages ? a.remap[id] : -1;
            if (to < -1) to = a.list_f[-2 - to];  // not written by its move yet
            if (to < 0) {
                set_err(a.err, VX_DATA_BAD_PAGE_ID);
                to = id;
            }
            a.indices_out[at + j] = to;
        }
        return;
    }
    const uint32_t pieces = page_pieces(a), copies = (uint32_t)a.head[0] * pieces;
    for (uint32_t it = blockIdx.x - rows; it < copies; it += gridDim.x - rows) {
        const int i = it / pieces, piece = it - i * pieces;
        const int32_t from = a.list_e[i], to = a.list_f[i];
        if (piece == 0 && tid == 0) {
            a.ref_out[to] = a.ref_in[from];
            a.ref_out[from] = 0;
            a.remap[from] = to;
        }
        copy_piece(a, from, to, piece);
    }
}

// blocks of an applying grid: every item, at most 8 blocks per SM
cudaError_t apply_grid(int64_t items, unsigned *grid) {
    const int sms = current_sm_count();
    if (sms < 1) return cudaErrorInvalidDevice;
    *grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(items, (int64_t)sms * 8));
    return cudaSuccess;
}

int64_t plan_blocks(const PageArgs &a) { return (a.num_pages + 4 * PG_THREADS - 1) / (4 * PG_THREADS); }
int64_t host_pieces(const PageArgs &a) { return (((int64_t)a.kb + a.vb + a.cb) / 16 + PG_PIECE - 1) / PG_PIECE; }

}  // namespace

cudaError_t launch_copy_pages(const PageArgs &a, cudaStream_t s) {
    unsigned grid = 0;
    if (a.num_copies * host_pieces(a) > INT32_MAX) return cudaErrorInvalidValue;
    cudaError_t e = apply_grid((int64_t)a.num_copies * host_pieces(a), &grid);
    if (e == cudaSuccess && a.num_copies <= PG_FEW)
        return launch_k(k_copy_few, dim3(grid), dim3(PG_BLOCK), 0, s, true, a);
    if (e == cudaSuccess) e = launch_k(k_plan_copy, dim3(PG_CTAS), dim3(PG_THREADS), 0, s, true, a);
    if (e == cudaSuccess) e = launch_k(k_apply_copy, dim3(grid), dim3(PG_BLOCK), 0, s, true, a);
    return e;
}

cudaError_t launch_update_table(const PageArgs &a, cudaStream_t s) {
    UpdateJobs j;
    if (!update_jobs(a, &j)) return cudaErrorInvalidValue;
    const uint32_t blocks = j.fresh + j.rows + j.refs + j.copies;
    cudaError_t e = launch_k(k_plan_update, dim3((unsigned)(1 + plan_blocks(a))), dim3(PG_THREADS), 0, s, true, a);
    const size_t smem = (size_t)a.new_rows * sizeof(int32_t);
    if (e == cudaSuccess) e = launch_k(k_apply_update, dim3((unsigned)blocks), dim3(PG_BLOCK), smem, s, true, a, j);
    return e;
}

cudaError_t launch_compact_pages(const PageArgs &a, cudaStream_t s) {
    constexpr int W = PG_BLOCK / 32;
    const int64_t lists = ((a.num_pages + PG_SEG - 1) / PG_SEG * 4 + W - 1) / W;
    const int64_t rows = (a.B * (int64_t)((a.max_pages + PG_SPAN - 1) / PG_SPAN) + W - 1) / W;
    unsigned grid = 0;
    cudaError_t e = apply_grid(std::max<int64_t>(1, a.num_pages / 2 * host_pieces(a)), &grid);
    if ((rows + grid) * W > INT32_MAX || a.num_pages * host_pieces(a) > INT32_MAX) e = cudaErrorInvalidValue;
    if (plan_blocks(a) == 1) {  // (500 latent pages: 8.7 us in three launches, 7.0 in two)
        if (e == cudaSuccess) e = launch_k(k_list_small, dim3(1), dim3(PG_THREADS), 0, s, true, a);
    } else {
        if (e == cudaSuccess) e = launch_k(k_plan_compact, dim3((unsigned)plan_blocks(a)), dim3(PG_THREADS), 0, s, true, a);
        if (e == cudaSuccess) e = launch_k(k_list_compact, dim3((unsigned)lists), dim3(PG_BLOCK), 0, s, true, a);
    }
    if (e == cudaSuccess)
        e = launch_k(k_apply_compact, dim3((unsigned)(rows + grid)), dim3(PG_BLOCK), 0, s, true, a, (int)rows);
    return e;
}

}  // namespace vx
