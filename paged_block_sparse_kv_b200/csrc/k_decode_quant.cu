// k_decode_quant.cu -- exact softmax attention over the selected pages of an 8-bit cache (GQA).
//
// For query head g of KV head h, over the valid tokens t of the selected pages p:
//   x_t = sm_scale * k_scale[p][h] * (q_g . kc_t),  out = sum_t softmax(x)_t v_scale[p][h] vc_t
// with kc, vc the codes (int8 or e4m3).  The work split (flat list of 16-token tiles, pieces,
// one partial per (row, piece), merge) is that of k_decode.cu, and so is a merge kernel.  Partials
// are divided by their own sums here: a sum of weighted values, undivided, leaves fp32's range when
// the values are near its end (a thousand of 2^119 do), their mean does not.
//
// Both code types are exact in fp16 (int8: integers up to 128; e4m3: 4 significant bits,
// 2^-9 .. 448), so the products run as fp16 mma with fp32 sums and the scales stay outside:
// k_scale multiplies a tile's logits, v_scale a tile's P.V product.  The query is bf16, whose
// range fp16 lacks: each query head is first scaled by a power of two that puts its largest
// element into [2^14, 2^15), exact for every element down to 2^-29 of the largest (smaller
// ones keep an absolute error of 2^-40 of it), and the factor goes into the logits' scale.  P
// is rounded to fp16, to half a step of 2^-10 where bf16's is 2^-7; it is taken relative to
// 2^-DQ_PSHIFT of the running maximum of weight times v_scale, so that what is down to 2^-29 of it is
// a normal number.
//
// Fragments straight from 8-bit tiles, no transposition of bytes:
//  * K (A operand, tokens x dims): the order of the contracted dims is free as long as Q has
//    the same one, so a lane takes 16 consecutive dims of its two token rows with one 16-byte
//    shared load each and feeds 4 mma steps from them (bytes 4s, 4s+1 and 4s+2, 4s+3 are the
//    two k halves of step s).
//  * V (A operand, dims x tokens): ldmatrix.trans moves byte pairs, so a lane gets two dims
//    of two tokens per register: bytes 0, 2 are dim 2g of both tokens, bytes 1, 3 dim 2g + 1.
//    Row g of the fragment is dim 2g of the 16, row g + 8 dim 2g + 1; nothing else changes.
// Value codes past the request's length are zeroed in registers, logits there are -inf.
//
// Bound: HBM (2 bytes read per token, KV head and dim for 4 G operations).  Measured on one B200,
// whole call: 256 requests of 64 pages (543 MB) 103-107 us by the GPU, 5.1-5.3 TB/s, the decode kernel alone 5.5 TB/s;
// 32 requests of 128 pages (135 MB) 33.5 us, 4.0 TB/s: 3 us until the first copies leave (selection,
// then page table, both from DRAM), warps that end over 9 us (22 to 31 us), the merge.  The
// conversions are hidden: with none at all (a timing copy) 256 requests took 0.5% and 32 requests 0.3%
// less.  16 warps per SM because a tile is a chain of short steps: 8 warps took 137 us where 16 took
// 108; the ring then holds 3 tiles per warp, the same 192 KB.  Units that follow the weights (see
// attend_codes) and partials divided by their sums cost 256 requests 0.6 to 1.8% (by the GPU) and 32
// requests 1.2%, in turn with the largest v_scale as the unit; an integer exponent as the unit cost 2.8%,
// weights computed ahead of the maximum 3%.
// Measured and not kept: the block joining its warps' partials itself (its loads of fresh partials
// cost 4-5 us at the block's end: 37.5 and 33.0 us), the first two tiles issued before the rest (33.3
// and 32.7), the selection's lines prefetched before the dependency wait (34.9 and 32.7).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <type_traits>

#include "vx_attend.cuh"

namespace vx {

namespace {

// Partials per row above which the merge takes a block per row and head (k_merge_many).  Against
// k_merge, us per call: 61 partials per row 18.3 and 19.8, 128 12.2 and 15.5, 256 13.1 and 19.3, 512 21.3
// and 32.2; but 16 per row 22.4 and 21.8, 32 9.0 and 8.6.
constexpr int DQ_MANY = 32;
constexpr int DQ_FEW = 4;            // at most this many: k_merge_few
constexpr float DQ_PSHIFT = 15.f;       // weights are at most 2^15, fp16's largest number is 65504
constexpr float DQ_PUNIT = 0x1p-15f;    // the output leaves the tiles without that factor
constexpr float DQ_MLAG = 16.f;         // the softmax's reference may stay this far below the largest logit (log2 units)
// 16-token tiles in flight per warp (4 KB each at head_dim 128): about 192 KB per SM
constexpr int dq_stages(int warps) { return warps > 8 ? 48 / warps : 6; }

struct __align__(16) QuantMeta {
    int32_t row, nvalid;
    float ks, vs;
};

__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }

// D = A(16x16, row) * B(16x8, col) + D, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four codes to fp16: bytes (0, 1) and (2, 3) of w, or (0, 2) and (1, 3) when SPLIT.
template <int FMT, bool SPLIT>
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == VX_QUANT_INT8) {
        // u = code + 128 as the low byte of fp16 1024 + u; less 1152 gives the code, exactly
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
        const uint32_t a = __byte_perm(u, 0x64646464u, SPLIT ? 0x4240 : 0x4140);
        const uint32_t b = __byte_perm(u, 0x64646464u, SPLIT ? 0x4341 : 0x4342);
        lo = half2_bits(__hsub2(*reinterpret_cast<const __half2 *>(&a), off));
        hi = half2_bits(__hsub2(*reinterpret_cast<const __half2 *>(&b), off));
    } else {
        const uint32_t v = SPLIT ? __byte_perm(w, 0u, 0x3120) : w;
        const __half2_raw a = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v & 0xffffu), __NV_E4M3);
        const __half2_raw b = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v >> 16), __NV_E4M3);
        lo = half2_bits(__half2(a));
        hi = half2_bits(__half2(b));
    }
}

// Byte offset of 16-byte chunk `chunk` of token row `row` in a tile: rows of D bytes, swizzled
// by TMA over 128 bytes (D = 128) or 64 bytes (D = 64, where the pattern repeats every 8 rows).
template <int D>
__device__ __forceinline__ uint32_t code_off(int row, int chunk) {
    if constexpr (D == 128) return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
    return static_cast<uint32_t>(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

// 4 bytes global -> shared, asynchronously; cp_async_arrive: one arrival on `bar` once the thread's
// copies so far have landed
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

// A tile as the consumer sees it: where its codes are, its valid tokens and its page's scales.
struct Tile {
    uint32_t k, v;
    int32_t nvalid;
    float ks, vs;
};

// How the value scales of two tiles, and of a row's tiles so far, lie to one another.
struct Spread {
    float low = INFINITY;  // the smallest of the row

    // with the next one or two tiles: may they go as a pair, and is `far` needed?
    __device__ __forceinline__ void next(float a, float b, bool &pair, bool &far) {
        const float lo = fminf(fabsf(a), fabsf(b)), hi = fmaxf(fabsf(a), fabsf(b));
        low = fminf(low, lo);
        far = !(hi <= low * 0x1p60f) || low < 0x1p-100f;
        pair = hi <= lo * 16.f && !far;
    }
};

// T 16-token tiles of one row.  qf: the query heads as mma B fragments in the dims order above; hs:
// the logits' scale of heads 2 q4, 2 q4 + 1 (log2 units).  Weights are exp2(logit - m_run) and l_run is
// their sum; m_run stays up to DQ_MLAG behind the largest logit.  acc: the output, unnormalised, in
// units of 2^(m_run + d_run - DQ_PSHIFT), where m_run + d_run is the largest logit + log2 of v_scale
// met (kept as the difference d_run: beside a logit of 2^24 the sum would be off by whole powers of
// two, and P out of fp16's range).  P is multiplied by v_scale * unit, unit = 2^(DQ_PSHIFT - d_run),
// before it is rounded to fp16, so acc needs no multiplication per tile.  What that rounding loses is at
// most 2^-35 of the largest weight times v_scale met, whatever the scales of the row's pages are: in
// units of the largest v_scale alone, all of a page was lost that carries the weight under a scale 2^-42
// of another's.  (Of a pair, d_run follows the larger scale: 4 bits of 2^-40, and the scale's rounding to
// a power of two one.)  far: a weight or the unit may leave fp32's range, because the row's scales differ
// by more than 2^60 or one is below 2^-100: then weight and scale share one exponent.  Two tiles at a
// time share the maximum's shuffles and give the scheduler two independent chains.
template <int D, int NT, int FMT, int T>
__device__ __forceinline__ void attend_codes(const Tile (&tile)[T], const uint32_t (&qf)[NT][D / 16][2],
                                             const float (&hs)[NT][2], float (&acc)[NT][D / 16][4],
                                             float (&m_run)[NT][2], float (&l_run)[NT][2], float (&d_run)[NT][2],
                                             float (&unit)[NT][2], bool far, int lane) {
    constexpr int MT = D / 16;
    constexpr int HALVES = D / 64;  // 16-byte chunks a lane takes of a token row
    const int g4 = lane >> 2, q4 = lane & 3;
    float s[T][NT][4];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[t][nt][e] = 0.f;
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            // chunk HALVES * q4 + h: the 8 lanes of a quarter warp cover all 32 banks
            const uint4 r0 = lds_v4(tile[t].k + code_off<D>(g4, HALVES * q4 + h));
            const uint4 r1 = lds_v4(tile[t].k + code_off<D>(g4 + 8, HALVES * q4 + h));
            const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
            for (int st = 0; st < 4; ++st) {
                uint32_t a0, a1, a2, a3;
                codes_to_half<FMT, false>(w0[st], a0, a2);
                codes_to_half<FMT, false>(w1[st], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma_f16_16816(s[t][nt], a0, a1, a2, a3, qf[nt][h * 4 + st][0], qf[nt][h * 4 + st][1]);
            }
        }
    }
    // 2^(ve - 1) < |v_scale| <= 2^ve of the tile with the largest
    float vs_top = fabsf(tile[0].vs);
#pragma unroll
    for (int t = 1; t < T; ++t) vs_top = fmaxf(vs_top, fabsf(tile[t].vs));
    const float ve = __uint_as_float(0x4b000000u + ((__float_as_uint(vs_top) + 0x7fffffu) >> 23)) - 8388735.f;
    // online softmax (base 2), tokens >= nvalid masked
    uint32_t pb[T][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        float x[T][4], most[2];
        bool change = false;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const float f[2] = {hs[nt][0] * tile[t].ks, hs[nt][1] * tile[t].ks};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[t][e] = g4 + 8 * (e >> 1) < tile[t].nvalid ? s[t][nt][e] * f[e & 1] : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float mx = fmaxf(x[0][i], x[0][i + 2]);
#pragma unroll
            for (int t = 1; t < T; ++t) mx = fmaxf(mx, fmaxf(x[t][i], x[t][i + 2]));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 16));
            most[i] = mx;
            const float above = mx - m_run[nt][i];
            change |= above > DQ_MLAG || above + ve > d_run[nt][i];
        }
        if (__any_sync(FULL, change)) {  // rare after a row's first tiles
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float m = most[i] - m_run[nt][i] > DQ_MLAG ? most[i] : m_run[nt][i];
                const float by = m_run[nt][i] - m;  // 0, or -inf at a row's first tiles
                const float d = fmaxf(d_run[nt][i] + by, most[i] - m + ve);
                const float alpha = exp2f(d_run[nt][i] + by - d);
                l_run[nt][i] *= exp2f(by);
                unit[nt][i] = exp2f(DQ_PSHIFT - d);
                m_run[nt][i] = m;
                d_run[nt][i] = d;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    acc[nt][mt][i] *= alpha;
                    acc[nt][mt][i + 2] *= alpha;
                }
            }
        }
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const float r[2] = {tile[t].vs * unit[nt][0], tile[t].vs * unit[nt][1]};
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = exp2f(x[t][e] - m_run[nt][e & 1]);
#pragma unroll
            for (int i = 0; i < 2; ++i) l_run[nt][i] += p[i] + p[i + 2];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] *= r[e & 1];
            if (T == 1 && far) {
                const uint32_t bits = __float_as_uint(tile[t].vs), field = (bits >> 23) & 0xffu;
                float mant = __uint_as_float((bits & 0x807fffffu) | 0x3f800000u);
                if (field == 0u) mant = tile[t].vs * 0x1p126f;
                if (field == 255u) mant = tile[t].vs;  // an infinite scale or a NaN shows in the output
                const float by = static_cast<float>(static_cast<int>(max(field, 1u)) - 127) + DQ_PSHIFT;
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = exp2f(x[t][e] - m_run[nt][e & 1] + (by - d_run[nt][e & 1])) * mant;
            }
            pb[t][nt][0] = movmatrix_t(half2_bits(__floats2half2_rn(p[0], p[1])));
            pb[t][nt][1] = movmatrix_t(half2_bits(__floats2half2_rn(p[2], p[3])));
        }
    }
    // O^T[dim][head] += codes . P^T
    const int mi = lane >> 3, tok = (lane & 7) + 8 * (mi & 1);
#pragma unroll
    for (int t = 0; t < T; ++t) {
        const int nvalid = tile[t].nvalid;
        const bool tail = nvalid < DEC_TILE;
        const int t_lo = 2 * q4, t_hi = 8 + 2 * q4;  // tokens of this lane's A halves
        const uint32_t mlo = (t_lo < nvalid ? 0x0000ffffu : 0u) | (t_lo + 1 < nvalid ? 0xffff0000u : 0u);
        const uint32_t mhi = (t_hi < nvalid ? 0x0000ffffu : 0u) | (t_hi + 1 < nvalid ? 0xffff0000u : 0u);
#pragma unroll
        for (int c = 0; c < MT; c += 2) {
            uint32_t r[4];
            ldsm_x4_t(tile[t].v + code_off<D>(tok, c + (mi >> 1)), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t lo = r[2 * u], hi = r[2 * u + 1];
                if (tail) {
                    lo &= mlo;
                    hi &= mhi;
                }
                uint32_t a0, a1, a2, a3;
                codes_to_half<FMT, true>(lo, a0, a1);
                codes_to_half<FMT, true>(hi, a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16_16816(acc[nt][c + u], a0, a1, a2, a3, pb[t][nt][0], pb[t][nt][1]);
            }
        }
    }
}

// The group's query heads (row-major from qb, G of them) as mma B fragments in the dims order above,
// each scaled into fp16's range, and the logits' scale (log2 units) that undoes it.
template <int D, int NT>
__device__ __forceinline__ void load_query(const __nv_bfloat16 *qb, int G, float scale_log2, uint32_t (&qf)[NT][D / 16][2],
                                           float (&hs)[NT][2], int lane) {
    constexpr int MT = D / 16, HALVES = D / 64;
    const int g4 = lane >> 2, q4 = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int head = nt * 8 + g4;
        uint2 w[MT];  // dims (HALVES q4 + half) 16 + 4 st .. + 3 of step half * 4 + st
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            w[i] = make_uint2(0u, 0u);
            if (head < G)
                w[i] = *reinterpret_cast<const uint2 *>(qb + (size_t)head * D + (HALVES * q4 + i / 4) * 16 + (i & 3) * 4);
            top = __vmaxu2(top, __vmaxu2(w[i].x & 0x7fff7fffu, w[i].y & 0x7fff7fffu));
        }
        uint32_t amax = max(top & 0xffffu, top >> 16);
        amax = max(amax, __shfl_xor_sync(FULL, amax, 1));
        amax = max(amax, __shfl_xor_sync(FULL, amax, 2));
        // 2^(14 - exponent of the largest element), at most 2^113: that takes bf16's smallest number to 2^-20,
        // still exact in fp16, and leaves its inverse 13 bits above fp32's smallest normal number for sm_scale
        const uint32_t ef = min(268u - (amax >> 7), 240u);
        const float mul = __uint_as_float(ef << 23);
        const float inv = __uint_as_float((254u - ef) << 23) * scale_log2;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            qf[nt][i][0] = half2_bits(__floats2half2_rn(__uint_as_float(w[i].x << 16) * mul,
                                                        __uint_as_float(w[i].x & 0xffff0000u) * mul));
            qf[nt][i][1] = half2_bits(__floats2half2_rn(__uint_as_float(w[i].y << 16) * mul,
                                                        __uint_as_float(w[i].y & 0xffff0000u) * mul));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) hs[nt][i] = __shfl_sync(FULL, inv, (2 * q4 + i) * 4);
    }
}

// LATE: the split has late pieces (see k_decode.cu).
template <int D, int NT, int FMT, bool LATE>
__global__ void __launch_bounds__(quant_warps(NT * 8) * 32, 1)
    k_decode_quant(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const DecodeArgs a, const float *__restrict__ k_scale, const float *__restrict__ v_scale) {
    constexpr int TILE_BYTES = DEC_TILE * D;
    constexpr int STAGE_BYTES = 2 * TILE_BYTES;  // K tile + V tile
    constexpr int MT = D / 16;
    constexpr int WARPS = quant_warps(NT * 8), DQ_STAGES = dq_stages(WARPS);

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;  // 128-byte swizzle wants 1 KB alignment
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g4 = lane >> 2, q4 = lane & 3;
    const uint32_t stage0 = base + (uint32_t)(warp * DQ_STAGES) * STAGE_BYTES;
    const uint32_t bar0 = base + (uint32_t)(WARPS * DQ_STAGES) * STAGE_BYTES + (uint32_t)(warp * DQ_STAGES) * 8u;
    QuantMeta *meta = reinterpret_cast<QuantMeta *>(smem_raw + (base - raw) + WARPS * DQ_STAGES * STAGE_BYTES +
                                                    WARPS * DQ_STAGES * 8);
    int32_t *pieces = reinterpret_cast<int32_t *>(meta + WARPS * DQ_STAGES) + warp * DQ_STAGES;  // of the stages' tiles
    meta += warp * DQ_STAGES;

    if (lane == 0) {
        // two arrivals complete a stage: the one that announces its bytes, and its scales' copies
        for (int s = 0; s < DQ_STAGES; ++s) mbar_init(bar0 + 8u * s, 2);
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    __syncwarp();

    const int64_t wid = (int64_t)warp * gridDim.x + blockIdx.x;  // few chunks still reach every SM
    if (wid >= a.static_chunks) return;

    uint32_t qf[NT][MT][2];
    float hs[NT][2];
    float acc[NT][MT][4];
    float m_run[NT][2], l_run[NT][2], d_run[NT][2], unit[NT][2];

    // partial of row `r` (at least one tile attended) for piece `c`: slot r + c.  The output is divided
    // by its sum before its unit goes in: no number is then larger than the largest value
    auto write_partial = [&](int64_t r, int64_t c) {
        const int64_t slot = r + c;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int head = nt * 8 + 2 * q4 + i;
                float v = l_run[nt][i];
                v += __shfl_xor_sync(FULL, v, 4);
                v += __shfl_xor_sync(FULL, v, 8);
                v += __shfl_xor_sync(FULL, v, 16);
                if (head < a.G) {
                    float *o = a.o_part + (slot * a.G + head) * D + 2 * g4;
                    const float inv = v > 0.f ? __fdividef(DQ_PUNIT, v) : 0.f;
                    const float half = exp2f(0.5f * d_run[nt][i]);  // the unit can be 2^128
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
                        *reinterpret_cast<float2 *>(o + mt * 16) = make_float2(acc[nt][mt][i] * inv * half * half,
                                                                               acc[nt][mt][2 + i] * inv * half * half);
                    if (g4 == 0) {
                        float *ml = a.ml_part + (slot * a.G + head) * 2;
                        ml[0] = m_run[nt][i];
                        ml[1] = v;
                    }
                }
            }
    };
    Spread spread;
    auto start_row = [&](int64_t r) {
        spread = Spread();
        const int b = static_cast<int>((uint32_t)r / (uint32_t)a.Hkv), h = static_cast<int>((uint32_t)r % (uint32_t)a.Hkv);
        const __nv_bfloat16 *qb = a.q + ((size_t)b * a.Hq + (size_t)h * a.G) * D;
        load_query<D, NT>(qb, a.G, a.scale_log2, qf, hs, lane);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m_run[nt][i] = d_run[nt][i] = -INFINITY;
                l_run[nt][i] = unit[nt][i] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
        }
    };
    auto p_start = [&](int64_t c) -> int64_t {
        if constexpr (LATE) return piece_start<true>(c, a.units, a.static_units, a.static_chunks, a.chunks);
        return chunk_start<true>(c, a.units, a.chunks);
    };
    // the next piece this warp takes after its static one (warp-uniform): from the counter, or
    // round robin over the warps; a.chunks or more: none left
    int64_t rr_next = a.static_chunks + wid;
    auto next_piece = [&]() -> int64_t {
        if constexpr (!LATE) return a.chunks;
        if (a.piece_ctr) {
            unsigned v = 0;
            if (lane == 0) v = atomicAdd(a.piece_ctr, 1u);
            return a.static_chunks + (int64_t)__shfl_sync(FULL, v, 0);
        }
        const int64_t c = rr_next;
        rr_next += a.static_chunks;
        return c;
    };
    // every row that a piece touches starts with an empty partial (max -inf, sum 0); rows with
    // attended tiles get theirs overwritten later by this same warp
    auto empty_piece = [&](int64_t c) {
        const int64_t u0 = p_start(c), u1 = p_start(c + 1);
        for (int64_t r = div64(u0, a.units_per_row); r <= div64(u1 - 1, a.units_per_row); ++r)
            if (lane < a.G) {
                float *ml = a.ml_part + ((r + c) * a.G + lane) * 2;
                ml[0] = -INFINITY;
                ml[1] = 0.f;
            }
        __syncwarp();
    };

    int64_t fc = wid, batch = p_start(wid), f_end = p_start(wid + 1);
    int64_t cur_row = -1, cur_pc = -1;  // (row, piece) being accumulated
    bool attended = false;              // it has a tile
    // nothing is read before the wait: the first row's query is loaded and scaled while its first
    // tiles are on their way
    pdl_wait();

    Resolved rs;
    auto resolve = [&]() {
        rs = resolve_unit<true>(a, batch + lane, f_end);
        return __ballot_sync(FULL, rs.valid);
    };
    uint32_t pending = resolve();
    uint32_t issued = 0, consumed = 0;
    bool fill_done = false, started = false;

    for (;;) {
        // issue loads until the ring is full or no piece is left
        while (!fill_done && issued - consumed < DQ_STAGES) {
            if (pending == 0) {
                batch += 32;
                if (batch >= f_end) {
                    const int64_t c = next_piece();
                    if (c >= a.chunks) {
                        fill_done = true;
                        break;
                    }
                    fc = c;
                    batch = p_start(c);
                    f_end = p_start(c + 1);
                    empty_piece(c);
                }
                pending = resolve();
                continue;
            }
            const int src = __ffs(pending) - 1;
            pending &= pending - 1;
            const int st = static_cast<int>(issued % DQ_STAGES);
            if (lane == src) {
                const uint32_t bar = bar0 + 8u * st;
                const uint32_t dst = stage0 + (uint32_t)st * STAGE_BYTES;
                // no proxy fence: this stage's earlier shared-memory reads have completed, their
                // values were consumed before the __syncwarp that released the stage
                mbar_arrive_expect_tx(bar, STAGE_BYTES);
                tma_load_3d(dst, &tmK, 0, rs.y, rs.z, bar);
                tma_load_3d(dst + TILE_BYTES, &tmV, 0, rs.y, rs.z, bar);
                // the page's scales straight into the stage's metadata: no thread waits for them
                cp_async_4(smem_u32(&meta[st].ks), k_scale + rs.z);
                cp_async_4(smem_u32(&meta[st].vs), v_scale + rs.z);
                cp_async_arrive(bar);
                *reinterpret_cast<int2 *>(&meta[st]) = make_int2(rs.row, rs.nvalid);
                if constexpr (LATE) pieces[st] = static_cast<int32_t>(fc);
            }
            __syncwarp();
            ++issued;
        }
        if (!started) {
            empty_piece(wid);
            started = true;
        }
        // next tile, or the end (row -1); with the one after it, when that is of the same row and piece
        int64_t row = -1, pc = -1;
        int count = 1;
        const int st = static_cast<int>(consumed % DQ_STAGES), st1 = static_cast<int>((consumed + 1) % DQ_STAGES);
        if (consumed != issued) {
            row = meta[st].row;
            pc = wid;
            if constexpr (LATE) pc = pieces[st];
            if (consumed + 1 != issued && meta[st1].row == row && (!LATE || pieces[st1] == pc)) count = 2;
        }
        if (row < 0 || row != cur_row || pc != cur_pc) {
            if (attended) write_partial(cur_row, cur_pc);
            if (row < 0) break;  // also of a warp that had no tile at all
            if (row != cur_row || attended) start_row(row);
            attended = false;
            cur_row = row;
            cur_pc = pc;
        }
        bool landed = mbar_wait_sleep(bar0 + 8u * st, (consumed / DQ_STAGES) & 1u);
        if (count == 2) landed &= mbar_wait_sleep(bar0 + 8u * st1, ((consumed + 1) / DQ_STAGES) & 1u);
        if (!__all_sync(FULL, landed)) {
            // a load did not arrive in time: report, let every issued load land, drop the partial in
            // progress (its slot keeps its empty partial) and give every piece this warp would
            // still have taken its empty partials
            if (lane == 0) set_err(a.err, VX_DATA_TIMEOUT);
            for (uint32_t i = consumed; i < issued; ++i)
                (void)mbar_wait_bounded(bar0 + 8u * (i % DQ_STAGES), (i / DQ_STAGES) & 1u);
            while (!fill_done) {
                const int64_t c = next_piece();
                if (c >= a.chunks) fill_done = true;
                else empty_piece(c);
            }
            break;
        }
        Tile tile[2];
        auto take = [&](int k, int s) {
            const QuantMeta m = meta[s];
            const uint32_t at = stage0 + (uint32_t)s * STAGE_BYTES;
            tile[k] = {at, at + TILE_BYTES, m.nvalid, m.ks, m.vs};
        };
        take(0, st);
        tile[1] = tile[0];
        if (count == 2) take(1, st1);
        bool pair, far;
        spread.next(tile[0].vs, tile[1].vs, pair, far);
        if (!pair) count = 1;  // the second one waits for the next round
        if (count == 2) {
            attend_codes<D, NT, FMT, 2>(tile, qf, hs, acc, m_run, l_run, d_run, unit, false, lane);
        } else {
            const Tile one[1] = {tile[0]};
            attend_codes<D, NT, FMT, 1>(one, qf, hs, acc, m_run, l_run, d_run, unit, far, lane);
        }
        attended = true;
        __syncwarp();  // every lane is done with these stages before they are refilled
        consumed += count;
    }
}

// Partials (output, maximum in log2 units, sum) of one row and query head, joined in order by a warp;
// D / 32 dims per lane.  Outputs are divided by their sums, here as in the partials.
template <int D>
struct Joined {
    static constexpr int PER = D / 32;
    using Vec = typename std::conditional<PER == 4, float4, float2>::type;
    float o[PER], m = -INFINITY, l = 0.f;

    __device__ __forceinline__ Joined() {
#pragma unroll
        for (int d = 0; d < PER; ++d) o[d] = 0.f;
    }
    // n partials, `stride` heads apart: the maximum of all and the sum first, then the outputs by their
    // shares of it; an empty one (maximum -inf) left no output.  Lane i reads partial i's maximum and
    // sum, and the first 8 outputs are on their way meanwhile.
    __device__ __forceinline__ void add_all(const float *op, const float *ml, int64_t stride, int n, int lane) {
        auto pair = [&](int i) {
            return i < n ? make_float2(ml[i * stride * 2], ml[i * stride * 2 + 1]) : make_float2(-INFINITY, 0.f);
        };
        auto load = [&](Vec (&v)[8], int i0) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                v[u] = *reinterpret_cast<const Vec *>(op + min(i0 + u, n - 1) * stride * D + lane * PER);
        };
        Vec v[8];
        load(v, 0);
        const float2 first = pair(lane);
        m = first.x;
        for (int i = lane + 32; i < n; i += 32) m = fmaxf(m, ml[i * stride * 2]);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, off));
        if (m == -INFINITY) return;
        // exp2(x - m) as a square: the product with a partial's output is taken in two steps, so that a weight
        // below fp32's smallest number still counts beside a large output
        auto root = [&](float x) { return x == -INFINITY ? 0.f : exp2f(0.5f * (x - m)); };
        float h = root(first.x), hl = h * first.y;
        l = h * hl;
        for (int i = lane + 32; i < n; i += 32) {
            const float2 x = pair(i);
            const float r = root(x.x);
            l += r * r * x.y;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(FULL, l, off);
        const float share = l > 0.f ? __fdividef(1.f, l) : 0.f;
#pragma unroll 1
        for (int i0 = 0;;) {
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float f = __shfl_sync(FULL, h, u), g = __shfl_sync(FULL, hl, u) * share;
                const float *x = reinterpret_cast<const float *>(&v[u]);
                if (f != 0.f) {
#pragma unroll
                    for (int d = 0; d < PER; ++d) o[d] += x[d] * f * g;
                }
            }
            if ((i0 += 8) >= n) break;
            load(v, i0);
            const float2 x = pair(i0 + lane);
            h = root(x.x);
            hl = h * x.y;
        }
    }
    __device__ __forceinline__ void store(float *op, float *ml, int lane) const {
        *reinterpret_cast<Vec *>(op + lane * PER) = *reinterpret_cast<const Vec *>(o);
        if (lane == 0) {
            ml[0] = m;
            ml[1] = l;
        }
    }
    __device__ __forceinline__ void finish(const DecodeArgs &a, int64_t r, int g, int lane) const {
        const int b = static_cast<int>((uint32_t)r / (uint32_t)a.Hkv), h = static_cast<int>((uint32_t)r % (uint32_t)a.Hkv);
        const size_t head = (size_t)b * a.Hq + (size_t)h * a.G + g;
        uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + head * D + lane * PER);
#pragma unroll
        for (int d = 0; d < PER; d += 2) dst[d / 2] = pack_bf16x2(o[d], o[d + 1]);
        if (a.lse && lane == 0) a.lse[head] = l > 0.f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
};

// Merge of rows with many partials: a block per (row, query head), whose 8 warps take the partials in
// turn and meet in shared memory, in warp order.
template <int D>
__global__ void __launch_bounds__(256) k_merge_many(const DecodeArgs a) {
    __shared__ __align__(16) float s_o[8][D];
    __shared__ float s_ml[8][2];
    pdl_wait();
    pdl_trigger();  // the next grid may land; it waits for this grid's end
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r = blockIdx.x;
    const int g = blockIdx.y;
    auto piece = [&](int64_t u) { return piece_of<true>(u, a.units, a.static_units, a.static_chunks, a.chunks); };
    const int64_t lo = piece(r * a.units_per_row);
    const int n = static_cast<int>(piece((r + 1) * a.units_per_row - 1) - lo + 1);
    Joined<D> j;
    if (warp < n)
        j.add_all(a.o_part + ((r + lo + warp) * a.G + g) * D, a.ml_part + ((r + lo + warp) * a.G + g) * 2, a.G * 8,
                  (n - warp + 7) / 8, lane);
    j.store(s_o[warp], s_ml[warp], lane);
    __syncthreads();
    if (warp > 0) return;
    Joined<D> all;
    all.add_all(s_o[0], s_ml[0], 1, min(n, 8), lane);
    all.finish(a, r, g, lane);
}

// Merge of rows with at most DQ_FEW partials: a warp per (row, query head), every load issued at once.
template <int D>
__global__ void __launch_bounds__(256, 6) k_merge_few(const DecodeArgs a) {
    pdl_wait();
    pdl_trigger();  // the next grid may land; it waits for this grid's end
    const int lane = threadIdx.x & 31;
    const uint32_t item = blockIdx.x * 8 + (threadIdx.x >> 5);
    const uint32_t r = item / (uint32_t)a.G, g = item - r * (uint32_t)a.G;
    if (r >= (uint32_t)a.B * (uint32_t)a.Hkv) return;
    auto piece = [&](int64_t u) { return piece_of<true>(u, a.units, a.static_units, a.static_chunks, a.chunks); };
    const int64_t lo = piece((int64_t)r * a.units_per_row);
    const int n = static_cast<int>(piece(((int64_t)r + 1) * a.units_per_row - 1) - lo + 1);
    using J = Joined<D>;
    const float *op = a.o_part + ((r + lo) * a.G + g) * D + lane * J::PER, *ml = a.ml_part + ((r + lo) * a.G + g) * 2;
    typename J::Vec v[DQ_FEW];
    float2 s[DQ_FEW];
#pragma unroll
    for (int i = 0; i < DQ_FEW; ++i) {
        s[i] = make_float2(-INFINITY, 0.f);
        if (i < n) {
            s[i] = *reinterpret_cast<const float2 *>(ml + (int64_t)i * a.G * 2);
            v[i] = *reinterpret_cast<const typename J::Vec *>(op + (int64_t)i * a.G * D);
        }
    }
    J j;
#pragma unroll
    for (int i = 0; i < DQ_FEW; ++i) j.m = fmaxf(j.m, s[i].x);
    float h[DQ_FEW];  // as in Joined
#pragma unroll
    for (int i = 0; i < DQ_FEW; ++i) {
        h[i] = s[i].x == -INFINITY ? 0.f : exp2f(0.5f * (s[i].x - j.m));
        j.l += h[i] * h[i] * s[i].y;
    }
    const float share = j.l > 0.f ? __fdividef(1.f, j.l) : 0.f;
#pragma unroll
    for (int i = 0; i < DQ_FEW; ++i) {
        if (s[i].x == -INFINITY) continue;  // an empty partial left no output
        const float f = h[i] * s[i].y * share;
        const float *x = reinterpret_cast<const float *>(&v[i]);
#pragma unroll
        for (int d = 0; d < J::PER; ++d) j.o[d] += x[d] * h[i] * f;
    }
    j.finish(a, r, (int)g, lane);
}

// One block of WARPS warps per (request, KV head) row of at most WARPS * SLOTS tiles: warp w attends
// tiles 2 w and 2 w + 1 (and 2 (w + WARPS), ...), and the warps' partials meet in shared memory, in
// warp order: no partial goes through memory and no merge kernel follows.
template <int D, int NT, int FMT, int WARPS, int SLOTS>
__global__ void __launch_bounds__(WARPS * 32, quant_warps(NT * 8) / WARPS)
    k_decode_quant_row(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                       const DecodeArgs a, const float *__restrict__ k_scale, const float *__restrict__ v_scale) {
    constexpr int TILE_BYTES = DEC_TILE * D, MT = D / 16;
    static_assert(SLOTS % 2 == 0, "tiles go in pairs");
    __shared__ uint64_t s_bar[WARPS];
    __shared__ float s_ml[WARPS][NT * 8][2];
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    float *s_o = reinterpret_cast<float *>(smem_raw + (base - raw));  // [warp][head][dim], after the tiles
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g4 = lane >> 2, q4 = lane & 3;
    const uint32_t bar = smem_u32(&s_bar[warp]);
    if (lane == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    __syncwarp();
    pdl_wait();
    pdl_trigger();  // this grid's dependent waits for its end; it may land now
    const int64_t r = blockIdx.x;
    // lane s < SLOTS: this warp's tile s, which is tile (s / 2 * WARPS + warp) * 2 + s % 2 of the row
    const int64_t u = (int64_t)((lane >> 1) * WARPS + warp) * 2 + (lane & 1);
    Resolved rs{0, 0, 0, 0, false};
    if (lane < SLOTS && u < a.units_per_row)
        rs = resolve_unit<true>(a, r * a.units_per_row + u, (r + 1) * a.units_per_row);
    const uint32_t valid = __ballot_sync(FULL, rs.valid);
    float ks = 0.f, vs = 0.f;
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(valid) * 2 * TILE_BYTES);
    __syncwarp();
    const uint32_t tiles = base + (uint32_t)(warp * SLOTS) * 2 * TILE_BYTES;
    if (rs.valid) {
        const uint32_t dst = tiles + (uint32_t)lane * 2 * TILE_BYTES;
        tma_load_3d(dst, &tmK, 0, rs.y, rs.z, bar);
        tma_load_3d(dst + TILE_BYTES, &tmV, 0, rs.y, rs.z, bar);
        ks = __ldg(k_scale + rs.z);
        vs = __ldg(v_scale + rs.z);
    }
    const int b = static_cast<int>((uint32_t)r / (uint32_t)a.Hkv), h = static_cast<int>((uint32_t)r % (uint32_t)a.Hkv);
    uint32_t qf[NT][MT][2];
    float hs[NT][2], acc[NT][MT][4], m_run[NT][2], l_run[NT][2], d_run[NT][2], unit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m_run[nt][i] = d_run[nt][i] = -INFINITY;
            l_run[nt][i] = unit[nt][i] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
    }
    bool landed = true;
    if (valid) {
        load_query<D, NT>(a.q + ((size_t)b * a.Hq + (size_t)h * a.G) * D, a.G, a.scale_log2, qf, hs, lane);
        landed = __all_sync(FULL, mbar_wait_bounded(bar, 0));
        if (!landed) {  // report, and let the loads land before shared memory is used for the partials
            if (lane == 0) set_err(a.err, VX_DATA_TIMEOUT);
            (void)mbar_wait_bounded(bar, 0);
        }
    }
    uint32_t left = landed ? valid : 0u;
    Spread spread;
    auto next_tile = [&]() -> Tile {  // the lowest of `left`
        const int s = __ffs(left) - 1;
        left &= left - 1;
        const uint32_t at = tiles + (uint32_t)s * 2 * TILE_BYTES;
        return {at, at + TILE_BYTES, __shfl_sync(FULL, rs.nvalid, s), __shfl_sync(FULL, ks, s), __shfl_sync(FULL, vs, s)};
    };
#pragma unroll 1
    while (left) {
        const Tile t0 = next_tile();
        const uint32_t others = left;
        const Tile two[2] = {t0, left ? next_tile() : t0};
        bool pair, far;
        spread.next(t0.vs, two[1].vs, pair, far);
        if (others && pair) {
            attend_codes<D, NT, FMT, 2>(two, qf, hs, acc, m_run, l_run, d_run, unit, false, lane);
        } else {
            const Tile one[1] = {t0};
            attend_codes<D, NT, FMT, 1>(one, qf, hs, acc, m_run, l_run, d_run, unit, far, lane);
            left = others;  // the second one waits for the next round
        }
    }
    __syncthreads();  // every warp is done with its tiles (after a timeout: with its bounded wait)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int head = nt * 8 + 2 * q4 + i;
            float v = l_run[nt][i];
            v += __shfl_xor_sync(FULL, v, 4);
            v += __shfl_xor_sync(FULL, v, 8);
            v += __shfl_xor_sync(FULL, v, 16);
            if (g4 == 0) {
                s_ml[warp][head][0] = m_run[nt][i];
                s_ml[warp][head][1] = v;
            }
            if (head < a.G && valid) {  // divided by its sum, as in k_decode_quant
                float *o = s_o + (warp * a.G + head) * D + 2 * g4;
                const float inv = v > 0.f ? __fdividef(DQ_PUNIT, v) : 0.f, half = exp2f(0.5f * d_run[nt][i]);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
                    *reinterpret_cast<float2 *>(o + mt * 16) = make_float2(acc[nt][mt][i] * inv * half * half,
                                                                           acc[nt][mt][2 + i] * inv * half * half);
            }
        }
    __syncthreads();
    // two dims per thread; a warp without a tile has the maximum -inf and left no output
    for (int e = threadIdx.x; e < a.G * (D / 2); e += WARPS * 32) {
        const int head = e / (D / 2), dim = (e % (D / 2)) * 2;
        float M = -INFINITY, l = 0.f;
        float2 o = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_ml[w][head][0]);
        float f[WARPS];  // roots of the weights, as in Joined
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float m = s_ml[w][head][0];
            f[w] = m == -INFINITY ? 0.f : exp2f(0.5f * (m - M));
            l += f[w] * f[w] * s_ml[w][head][1];
        }
        const float share = l > 0.f ? __fdividef(1.f, l) : 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (s_ml[w][head][0] == -INFINITY) continue;
            const float2 x = *reinterpret_cast<const float2 *>(s_o + (w * a.G + head) * D + dim);
            const float g = f[w] * s_ml[w][head][1] * share;
            o.x += x.x * f[w] * g;
            o.y += x.y * f[w] * g;
        }
        const size_t at = (size_t)b * a.Hq + (size_t)h * a.G + head;
        *reinterpret_cast<uint32_t *>(a.out + at * D + dim) = pack_bf16x2(o.x, o.y);
        if (a.lse && dim == 0) a.lse[at] = l > 0.f ? (M + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
}

template <int D, int NT, int FMT, int WARPS, int SLOTS>
cudaError_t launch_row(const DecodeArgs &a, const QuantArgs &qa, const CUtensorMap &tmK, const CUtensorMap &tmV,
                       cudaStream_t s, bool pdl) {
    constexpr size_t tiles = (size_t)WARPS * SLOTS * 2 * DEC_TILE * D, parts = (size_t)WARPS * NT * 8 * D * 4;
    constexpr size_t smem = 1024 + (tiles > parts ? tiles : parts);
    auto kern = k_decode_quant_row<D, NT, FMT, WARPS, SLOTS>;
    static std::atomic<unsigned long long> done;
    const cudaError_t e = ensure_smem_limit(kern, (int)smem, done);
    if (e != cudaSuccess) return e;
    return launch_k(kern, dim3((unsigned)((int64_t)a.B * a.Hkv)), dim3(WARPS * 32), smem, s, pdl, tmK, tmV, a,
                    (const float *)qa.k_scale, (const float *)qa.v_scale);
}

template <int D, int NT, int FMT>
cudaError_t launch_dnf(const DecodeArgs &a, const QuantArgs &qa, const CUtensorMap &tmK, const CUtensorMap &tmV,
                       int grid, cudaStream_t s, bool pdl) {
    constexpr int WARPS = quant_warps(NT * 8);
    const size_t smem = 1024 + (size_t)WARPS * dq_stages(WARPS) * (2 * DEC_TILE * D + 8 + sizeof(QuantMeta) + sizeof(int32_t));
    if (a.chunks == 0) {  // a block per row, of the fewest warps that hold its tiles
        if (a.units_per_row <= 8) return launch_row<D, NT, FMT, 4, 2>(a, qa, tmK, tmV, s, pdl);
        if (a.units_per_row <= 16) return launch_row<D, NT, FMT, WARPS / 2, 32 / WARPS>(a, qa, tmK, tmV, s, pdl);
        return launch_row<D, NT, FMT, WARPS, DQ_ROW_TILES / WARPS>(a, qa, tmK, tmV, s, pdl);
    }
    const bool late = a.chunks > a.static_chunks;
    auto kern = late ? k_decode_quant<D, NT, FMT, true> : k_decode_quant<D, NT, FMT, false>;
    static std::atomic<unsigned long long> done[2];
    cudaError_t e = ensure_smem_limit(kern, (int)smem, done[late ? 1 : 0]);
    if (e != cudaSuccess) return e;
    e = launch_k(kern, dim3(grid), dim3(WARPS * 32), smem, s, pdl, tmK, tmV, a, (const float *)qa.k_scale,
                 (const float *)qa.v_scale);
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)a.B * a.Hkv, per_row = a.chunks / rows;
    if (per_row > DQ_MANY) return launch_k(k_merge_many<D>, dim3((unsigned)rows, a.G), dim3(256), 0, s, true, a);
    // pieces that a row can span: of the even or static part, and of the late one
    int64_t most = div64(a.units_per_row * a.static_chunks + a.static_units - 1, a.static_units) + 1;
    if (late) most += div64(a.units_per_row * (a.chunks - a.static_chunks) + a.units - a.static_units - 1, a.units - a.static_units) + 1;
    if (most <= DQ_FEW)
        return launch_k(k_merge_few<D>, dim3((unsigned)((rows * a.G + 7) / 8)), dim3(256), 0, s, true, a);
    return launch_merge_normalised(a, s, true);
}

template <int D, int NT>
cudaError_t launch_dn(const DecodeArgs &a, const QuantArgs &qa, const CUtensorMap &tmK, const CUtensorMap &tmV,
                      int grid, cudaStream_t s, bool pdl) {
    return qa.format == VX_QUANT_INT8 ? launch_dnf<D, NT, VX_QUANT_INT8>(a, qa, tmK, tmV, grid, s, pdl)
                                      : launch_dnf<D, NT, VX_QUANT_E4M3>(a, qa, tmK, tmV, grid, s, pdl);
}

}  // namespace

cudaError_t launch_decode_quant(const DecodeArgs &a, const QuantArgs &qa, const CUtensorMap &tmK,
                                const CUtensorMap &tmV, int grid, cudaStream_t s, bool pdl) {
    const int nt = (a.G + 7) / 8;
    if (a.Dqk == 128 && nt == 1) return launch_dn<128, 1>(a, qa, tmK, tmV, grid, s, pdl);
    if (a.Dqk == 128 && nt == 2) return launch_dn<128, 2>(a, qa, tmK, tmV, grid, s, pdl);
    if (a.Dqk == 64 && nt == 1) return launch_dn<64, 1>(a, qa, tmK, tmV, grid, s, pdl);
    if (a.Dqk == 64 && nt == 2) return launch_dn<64, 2>(a, qa, tmK, tmV, grid, s, pdl);
    return cudaErrorInvalidValue;
}

}  // namespace vx
