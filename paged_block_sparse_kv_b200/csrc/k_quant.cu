// k_quant.cu -- cache stage of an 8-bit cache: new tokens quantised into their pages, with the
// pages' scales and centroids, in one pass (decode append and prefill write).
//
// Scale of a (page, KV head), K and V apart: the smallest power of two s >= 2^-126 with
// |x| <= qmax s for every token written into the page; code = rn(x / s).  With s = 2^e the
// division is exact, so a code depends on x and s alone; when a later token raises the scale
// the page's older codes become rn(code * s_old / s).  Centroid: bf16(s * sum(codes) / m), the
// sum of up to 64 codes exact in fp32 (int8: integers; e4m3: multiples of 2^-9 below 2^15),
// product and quotient in fp64, one rounding.
//
// One unit is the keys or the values of one (page, KV head).
//  * A page that holds new tokens alone (all but the first page of a prefill chunk): the unit's
//    page_size / 16 warps keep 16 token rows each in registers (a lane: 16-byte chunks of rows),
//    take the largest magnitude with a warp reduction (and through shared memory when the unit
//    has several warps), convert, store; nothing is read twice.  HBM bound: 2 bytes read and 1
//    written per element.
//  * A page that holds older tokens too: the same warps with its codes in registers as well.
//  * Append: a warp per unit; the one new row, and for the centroid the page's key codes in
//    16-byte chunks.  Value codes are read only when the scale grows.  Latency bound (length ->
//    table -> codes).
// Measured on one B200: prefill of 8 ragged requests, 16-token pages, head_dim 128, e4m3 (833 MB): 144 us
// warm and alone (0.88 of the copy peak), 151 in turn with other work (0.84).  Shortest of four graph
// replays, which flatters: e4m3 139 us, int8 144, 64-token pages 154; head_dim 64 0.58-0.66 of the copy
// peak (a unit is half as long and its fixed part the same).  Four blocks per SM (64 registers): three
// took 156 us where four took 147 and two 174.  A grid of requests by pages, whose blocks past a short
// request's end do nothing, took 151 us where this list takes 144 (and 486 where this one takes 507 for
// 256 of equal length).  Append of 256 requests, 8 KV heads 5.7 us.  The bound of four blocks costs
// spills at head_dim 128: 44-48 bytes in k_quant_prefill, 364-380 in quant_unit (a chunk's first page).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "vx_internal.h"

namespace vx {

namespace {

constexpr int QZ_WARPS = 8;
constexpr int QZ_MAX_STEPS = 16;  // prefill: units a warp takes one after the other, at most

template <int FMT>
__device__ __forceinline__ float code_to_float(uint8_t c) {
    if constexpr (FMT == VX_QUANT_INT8) return static_cast<float>(static_cast<int8_t>(c));
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(__half(h));
}

// nearest code, ties to even; |x| <= qmax up to the rounding of another program's scale
template <int FMT>
__device__ __forceinline__ uint32_t float_to_code(float x) {
    if constexpr (FMT == VX_QUANT_INT8) {
        const int v = __float2int_rn(fminf(fmaxf(x, -127.f), 127.f));
        return static_cast<uint32_t>(v) & 0xffu;
    }
    return __nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3);
}

// the smallest power of two s >= 2^-126 with amax <= qmax * s; amax: bits of a finite bf16 >= 0
template <int FMT>
__device__ __forceinline__ float scale_of(uint32_t amax) {
    // qmax = f 2^n with f in [1, 2): int8 127 = 1.984375 * 2^6, e4m3 448 = 1.75 * 2^8.  A bf16
    // mantissa m (of 128) is above f when m > 126 or m > 96
    constexpr uint32_t n = FMT == VX_QUANT_INT8 ? 6 : 8, mant = FMT == VX_QUANT_INT8 ? 126 : 96;
    const uint32_t e = (amax >> 7) + ((amax & 0x7f) > mant ? 1 : 0);
    return __uint_as_float((e > n ? e - n : 1u) << 23);  // fp32 exponent field, 1 at least
}

// Four new elements (floats x0..x3, |x * inv| <= qmax) to code bytes; int8: `bits` of the sums are
// added up for the centroid, see below.
template <int FMT>
__device__ __forceinline__ uint32_t four_codes(float x0, float x1, float x2, float x3, float inv, uint32_t (&b)[4]) {
    if constexpr (FMT == VX_QUANT_INT8) {
        // 1.5 * 2^23 + x rounds x to an integer, ties to even, in the low bits: 0x4b400000 + code
        b[0] = __float_as_uint(fmaf(x0, inv, 12582912.f));
        b[1] = __float_as_uint(fmaf(x1, inv, 12582912.f));
        b[2] = __float_as_uint(fmaf(x2, inv, 12582912.f));
        b[3] = __float_as_uint(fmaf(x3, inv, 12582912.f));
        return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
    } else {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0 * inv, x1 * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2 * inv, x3 * inv), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
}

// bf16(s * sum / m), rounded once.  Under a power-of-two scale of ordinary size (`plain`) fp32 will
// do, as scaling by s is exact: a whole page (m a power of two) needs no division; else the
// quotient is cut off, its last bit set when a remainder was lost (so that nothing looks like a
// tie that is none), and rounded to bf16.
__device__ __forceinline__ bool plain_scale(float s) {
    return (__float_as_uint(s) & 0x7fffffu) == 0 && s >= 0x1p-80f && s <= 0x1p80f;
}
__device__ __noinline__ uint32_t centroid_f64(float s, float sum, int m) { return f64_to_bf16_rne((double)s * sum / m); }
__device__ __forceinline__ uint32_t centroid_bits(bool plain, float s, float sum, int m) {
    if (!plain) return centroid_f64(s, sum, m);
    if ((m & (m - 1)) == 0) return __bfloat16_as_ushort(__float2bfloat16_rn(sum * (s / static_cast<float>(m))));
    const float d = static_cast<float>(m), q = __fdiv_rz(sum, d);
    const uint32_t lost = __fmaf_rn(-q, d, sum) != 0.f ? 1u : 0u;
    const __nv_bfloat16 c = __float2bfloat16_rn(__uint_as_float(__float_as_uint(q) | lost));
    return __float_as_uint(__bfloat162float(c) * s) >> 16;
}

// An infinity becomes the largest finite value of its sign, a NaN zero; returns the new largest
// magnitude.
template <int NR>
__device__ __noinline__ uint32_t make_finite(uint4 (&x)[NR]) {
    uint32_t amax = 0;
    for (int i = 0; i < NR; ++i) {
        uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        for (int j = 0; j < 4; ++j) {
            uint32_t h[2] = {w[j] & 0xffffu, w[j] >> 16};
            for (int u = 0; u < 2; ++u) {
                const uint32_t mag = h[u] & 0x7fffu;
                if (mag > 0x7f80u) h[u] = 0;
                else if (mag == 0x7f80u) h[u] = (h[u] & 0x8000u) | 0x7f7fu;
                amax = max(amax, h[u] & 0x7fffu);
            }
            w[j] = h[0] | (h[1] << 16);
        }
        x[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return amax;
}

// Largest magnitude (bf16 bits) of a warp's new rows, made finite.
template <int NR>
__device__ __forceinline__ uint32_t largest(uint4 (&x)[NR], int32_t *err, int lane) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const uint32_t a = __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu);
        const uint32_t b = __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu);
        top = __vmaxu2(top, __vmaxu2(a, b));
    }
    uint32_t amax = __reduce_max_sync(FULL, max(top & 0xffffu, top >> 16));
    if (amax >= 0x7f80u) {
        if (lane == 0) set_err(err, VX_DATA_BAD_VALUE);
        uint4 y[NR];  // a copy, so that x stays in registers on the usual path
#pragma unroll
        for (int i = 0; i < NR; ++i) y[i] = x[i];
        amax = __reduce_max_sync(FULL, make_finite<NR>(y));
#pragma unroll
        for (int i = 0; i < NR; ++i) x[i] = y[i];
    }
    return amax;
}

// One unit of a page without older tokens, by its WPU warps (this warp: rows [16 * part, 16 * part +
// 16) of m); every warp of the block takes part in the barriers, `go`: the unit exists.
template <int D, int WPU, int FMT, typename RowF, typename PageF>
__device__ __forceinline__ void quant_new_unit(bool go, bool is_key, int part, RowF new_row, PageF page, int m,
                                               int32_t *err, int lane, uint32_t *s_max, float (*s_sum)[D]) {
    constexpr int CPR = D / 8, RPL = 32 / CPR, NR = 16 / RPL;
    const int chunk = lane % CPR, t0 = part * 16 + lane / CPR;
    uint4 x[NR];
    if (go && m == 16 * WPU) {
        const __nv_bfloat16 *p = new_row(t0) + chunk * 8;
        const int64_t step = new_row(RPL) - new_row(0);
#pragma unroll
        for (int i = 0; i < NR; ++i) x[i] = ld_nc_v4(p + i * step);
    } else {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (go && t0 + i * RPL < m) x[i] = ld_nc_v4(new_row(t0 + i * RPL) + chunk * 8);
        }
    }
    uint8_t *codes;
    float *scale;
    __nv_bfloat16 *cen;
    go = page(codes, scale, cen) && go;
    uint32_t amax = largest<NR>(x, err, lane);
    if constexpr (WPU > 1) {
        if (lane == 0) s_max[threadIdx.x >> 5] = amax;
        __syncthreads();
        const int first = (threadIdx.x >> 5) - part;
#pragma unroll
        for (int w = 0; w < WPU; ++w) amax = max(amax, s_max[first + w]);
    }
    const float s = scale_of<FMT>(amax), inv = 1.f / s;
    uint32_t isum[8];
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        isum[e] = 0u;
        sum[e] = 0.f;
    }
    if (go) {
        // e4m3: scaled two at a time in bf16, exactly (s is a power of two; what falls below bf16's range
        // is far below half the smallest code)
        const __nv_bfloat162 inv2 = __float2bfloat162_rn(inv);
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            if constexpr (FMT == VX_QUANT_E4M3) {
                auto times = [&](uint32_t &w) {
                    const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w), inv2);
                    w = *reinterpret_cast<const uint32_t *>(&y);
                };
                times(x[i].x);
                times(x[i].y);
                times(x[i].z);
                times(x[i].w);
            }
            float f[8];
            bf16x8_to_f32(x[i], f);
            uint32_t b[2][4] = {};
            const float by = FMT == VX_QUANT_E4M3 ? 1.f : inv;
            const uint2 c = make_uint2(four_codes<FMT>(f[0], f[1], f[2], f[3], by, b[0]),
                                       four_codes<FMT>(f[4], f[5], f[6], f[7], by, b[1]));
            if (t0 + i * RPL < m) *reinterpret_cast<uint2 *>(codes + (t0 + i * RPL) * D + chunk * 8) = c;
            if (is_key) {  // rows past m are zeros
                if constexpr (FMT == VX_QUANT_INT8) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) isum[e] += b[e >> 2][e & 3];
                } else {
                    const uint32_t w[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 h(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[e]), __NV_E4M3));
                        sum[2 * e] += __low2float(h);
                        sum[2 * e + 1] += __high2float(h);
                    }
                }
            }
        }
    }
    if (go && part == 0 && lane == 0) *scale = s;
    if (WPU == 1 && !is_key) return;
    if constexpr (FMT == VX_QUANT_INT8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = static_cast<float>(static_cast<int32_t>(isum[e] - NR * 0x4b400000u));
    }
#pragma unroll
    for (int off = CPR; off < 32; off <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(FULL, sum[e], off);
    if constexpr (WPU > 1) {
        if (lane < CPR) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s_sum[threadIdx.x >> 5][chunk * 8 + e] = sum[e];
        }
        __syncthreads();
        if (part == 0) {
#pragma unroll
            for (int w = 1; w < WPU; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += s_sum[(threadIdx.x >> 5) + w][chunk * 8 + e];
        }
        __syncthreads();  // s_max and s_sum are free again
    }
    if (go && part == 0 && is_key && lane < CPR) {
        const bool plain = plain_scale(s);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = centroid_bits(plain, s, sum[2 * e], m) | (centroid_bits(plain, s, sum[2 * e + 1], m) << 16);
        *reinterpret_cast<uint4 *>(cen + chunk * 8) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// One unit of a page with older tokens, by its WPU warps (this warp: rows [16 * part, 16 * part +
// 16)).  Rows [0, n_old) are the page's older tokens, row t of [n_old, m) is src + t * stride.
// `go`: the unit exists (warps of missing units only take part in the block barriers).  At most one
// page of a chunk: not inlined, so that the usual path keeps its registers.
template <int D, int WPU, int FMT>
__device__ __noinline__ void quant_unit(bool go, bool is_key, int part, const __nv_bfloat16 *__restrict__ src,
                                        int64_t stride, uint8_t *__restrict__ codes, float *__restrict__ scale,
                                        __nv_bfloat16 *__restrict__ cen, int n_old, int m, int32_t *err, int lane,
                                        uint32_t *s_max, float (*s_sum)[D]) {
    constexpr int CPR = D / 8;    // 16-byte chunks of a new row = 8-byte chunks of a code row
    constexpr int RPL = 32 / CPR; // rows per warp-wide load
    constexpr int NR = 16 / RPL;  // rows per lane
    const int chunk = lane % CPR, t0 = part * 16 + lane / CPR;
    uint4 x[NR];
    uint2 old[NR];
    float s_old = 0.f;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const int t = t0 + i * RPL;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        old[i] = make_uint2(0u, 0u);
        if (go && t >= n_old && t < m) x[i] = ld_nc_v4(src + t * stride + chunk * 8);
    }
    if (go && n_old > 0) {
        s_old = *scale;
        if (is_key) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
                if (t0 + i * RPL < n_old) old[i] = *reinterpret_cast<const uint2 *>(codes + (t0 + i * RPL) * D + chunk * 8);
        }
    }
    amax = largest<NR>(x, err, lane);
    if constexpr (WPU > 1) {
        if (lane == 0) s_max[threadIdx.x >> 5] = amax;
        __syncthreads();
        const int first = (threadIdx.x >> 5) - part;
#pragma unroll
        for (int w = 0; w < WPU; ++w) amax = max(amax, s_max[first + w]);
    }
    const float s = fmaxf(scale_of<FMT>(amax), s_old);
    const float inv = 1.f / s;
    const bool grew = n_old > 0 && s > s_old;
    float sum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.f;
    if (go) {
        if (grew && !is_key) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
                if (t0 + i * RPL < n_old) old[i] = *reinterpret_cast<const uint2 *>(codes + (t0 + i * RPL) * D + chunk * 8);
        }
        const float ratio = s_old / s;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int t = t0 + i * RPL;
            uint2 c = old[i];
            if (t >= n_old) {
                float f[8];
                bf16x8_to_f32(x[i], f);
                c.x = c.y = 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    c.x |= float_to_code<FMT>(f[e] * inv) << (8 * e);
                    c.y |= float_to_code<FMT>(f[4 + e] * inv) << (8 * e);
                }
            } else if (grew) {
                uint2 r = make_uint2(0u, 0u);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    r.x |= float_to_code<FMT>(code_to_float<FMT>((c.x >> (8 * e)) & 0xff) * ratio) << (8 * e);
                    r.y |= float_to_code<FMT>(code_to_float<FMT>((c.y >> (8 * e)) & 0xff) * ratio) << (8 * e);
                }
                c = r;
            }
            if (t < m) {
                if (t >= n_old || grew) *reinterpret_cast<uint2 *>(codes + t * D + chunk * 8) = c;
                if (is_key) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        sum[e] += code_to_float<FMT>((c.x >> (8 * e)) & 0xff);
                        sum[4 + e] += code_to_float<FMT>((c.y >> (8 * e)) & 0xff);
                    }
                }
            }
        }
    }
#pragma unroll
    for (int off = CPR; off < 32; off <<= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(FULL, sum[e], off);
    if constexpr (WPU > 1) {
        if (lane < CPR) {
#pragma unroll
            for (int e = 0; e < 8; ++e) s_sum[threadIdx.x >> 5][chunk * 8 + e] = sum[e];
        }
        __syncthreads();
        if (part == 0) {
#pragma unroll
            for (int w = 1; w < WPU; ++w)
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += s_sum[(threadIdx.x >> 5) + w][chunk * 8 + e];
        }
        __syncthreads();  // s_max and s_sum are free again
    }
    if (go && part == 0) {
        if (lane == 0) *scale = s;
        if (is_key && lane < CPR) {
            const bool plain = plain_scale(s);
            uint32_t w[4];
#pragma unroll 1
            for (int e = 0; e < 4; ++e)
                w[e] = centroid_bits(plain, s, sum[2 * e], m) | (centroid_bits(plain, s, sum[2 * e + 1], m) << 16);
            *reinterpret_cast<uint4 *>(cen + chunk * 8) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Sums stop at 2^32 - 1: the lengths of a few requests may add up to more, and a sum that wrapped
// would look small again.
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return a + min(b, ~a); }

// Inclusive sum over the block; total: the block's sum.  s_part: QZ_WARPS words.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *s_part, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t y = __shfl_up_sync(FULL, v, off);
        if (lane >= off) v = sat_add(v, y);
    }
    if (lane == 31) s_part[warp] = v;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < QZ_WARPS; ++w) {
        if (w < warp) v = sat_add(v, s_part[w]);
        total = sat_add(total, s_part[w]);
    }
    __syncthreads();
    return v;
}

// Prefill write.  The units of all requests form one flat list: the touched pages request by request
// (request b's from the one holding first_pos[b] on), of a page the keys head by head, then the
// values.  Block i takes units [i * per_block, (i + 1) * per_block); a table of the requests' first
// pages in shared memory tells a warp whose unit it has.  Request b's new rows start in the packed
// input after those of requests 0..b-1.
template <int D, int WPU, int FMT>
__global__ void __launch_bounds__(QZ_WARPS * 32, 4) k_quant_prefill(const CentroidArgs a, const QuantArgs qa, const int per_block) {
    constexpr int UNITS = QZ_WARPS / WPU;  // units in flight per block
    __shared__ uint32_t s_max[QZ_WARPS], s_part[QZ_WARPS];
    __shared__ float s_sum[WPU > 1 ? QZ_WARPS : 1][D];
    // [B] (pages before the request's, its first row less first_pos, first_pos, length): with them at
    // hand a unit's rows are asked for at once
    extern __shared__ int4 s_req[];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t rows = 0, pages = 0;  // of the requests so far
    for (int b0 = 0; b0 < a.B; b0 += QZ_WARPS * 32) {
        const int b = b0 + threadIdx.x;
        const int32_t L = b < a.B ? a.seq_lens[b] : 0, fp = b < a.B ? a.first_pos[b] : 0;
        bool sound = b < a.B && L >= 1 && L <= a.max_pages * a.P && fp >= 0 && fp <= L;
        const uint32_t n_new = sound ? L - fp : 0;
        uint32_t total;
        const uint32_t end = sat_add(rows, block_scan(n_new, s_part, total));
        rows = sat_add(rows, total);
        sound = sound && end <= (uint64_t)qa.num_new;
        if (b < a.B && !sound && blockIdx.x == 0) set_err(a.err, VX_DATA_BAD_SEQ_LEN);
        const uint32_t n_pages = sound && L > fp ? ceil_div(L, a.P) - fp / a.P : 0;
        const uint32_t last = pages + block_scan(n_pages, s_part, total);
        pages += total;
        if (b < a.B) s_req[b] = make_int4((int32_t)(last - n_pages), (int32_t)(end - n_new) - fp, fp, L);
    }
    __syncthreads();
    const int log2_p = __ffs(a.P) - 1;
    const uint32_t heads2 = a.Hkv * 2;
    const uint64_t units = (uint64_t)pages * heads2, it_lo = (uint64_t)blockIdx.x * per_block,
                   it_hi = min(units, it_lo + per_block);
    const auto *kn = static_cast<const __nv_bfloat16 *>(a.k_new);
    const auto *vn = static_cast<const __nv_bfloat16 *>(a.v_new);
    auto *cen = static_cast<__nv_bfloat16 *>(a.centroids);
    for (uint64_t it0 = it_lo; it0 < it_hi; it0 += UNITS) {
        const bool go = it0 + warp / WPU < it_hi;
        const uint64_t it = go ? it0 + warp / WPU : it0;
        const uint32_t page_at = (uint32_t)div64((int64_t)it, heads2), rem = (uint32_t)(it - (uint64_t)page_at * heads2);
        int b = 0, hi = a.B - 1;  // the last request whose pages start at or before this one
        while (b < hi) {
            const int mid = (b + hi + 1) >> 1;
            if ((uint32_t)s_req[mid].x <= page_at) b = mid;
            else hi = mid - 1;
        }
        const int4 req = s_req[b];
        const int32_t L = req.w, fp = req.z;
        const int j = (fp >> log2_p) + (int)(page_at - (uint32_t)req.x);
        const int32_t id = a.page_indices[a.page_ptr[b] + j];
        const bool is_key = rem < (uint32_t)a.Hkv;
        const int h = is_key ? rem : rem - a.Hkv;
        const int m = min(a.P, L - j * a.P), n_old = max(0, fp - j * a.P);
        const __nv_bfloat16 *src = (is_key ? kn : vn) + (((int64_t)req.y + (int64_t)j * a.P) * a.Hkv + h) * D;
        auto new_row = [&](int t) { return src + (int64_t)t * a.Hkv * D; };
        auto page = [&](uint8_t *&codes, float *&scale, __nv_bfloat16 *&centroid) {
            const bool ok = id >= 0 && id < a.num_pool_pages;
            if (!ok && go && lane == 0) set_err(a.err, VX_DATA_BAD_PAGE_ID);
            const size_t blk = (size_t)(ok ? id : 0) * a.Hkv + h;
            codes = (is_key ? qa.k_cache : qa.v_cache) + blk * a.P * D;
            scale = (is_key ? qa.k_scale : qa.v_scale) + blk;
            centroid = cen + blk * D;
            return ok;
        };
        // units of several warps meet at barriers: their block takes one path
        const bool old = WPU == 1 ? n_old > 0 : __syncthreads_or(n_old > 0);
        if (old) {
            uint8_t *codes;
            float *scale;
            __nv_bfloat16 *centroid;
            const bool ok = page(codes, scale, centroid) && go;
            quant_unit<D, WPU, FMT>(ok, is_key, warp % WPU, src, (int64_t)a.Hkv * D, codes, scale, centroid, n_old, m,
                                    a.err, lane, s_max, s_sum);
        } else {
            quant_new_unit<D, WPU, FMT>(go, is_key, warp % WPU, new_row, page, m, a.err, lane, s_max, s_sum);
        }
    }
}

// Append: grid (ceil(2 Hkv / QZ_WARPS), B), a warp per unit.  A lane holds 16 codes (D / 16 lanes to
// a row) of every RPL-th row, and the new row's elements that belong to them.
template <int D, int NR, int FMT>
__global__ void __launch_bounds__(QZ_WARPS * 32) k_quant_append(const CentroidArgs a, const QuantArgs qa) {
    pdl_wait();
    // a dependent scorer (vx_block_topk_decode_append_quant) may launch now; it waits for this
    // grid's end and writes before it reads anything
    pdl_trigger();
    constexpr int CPR = D / 16, RPL = 32 / CPR;
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const int unit = blockIdx.x * QZ_WARPS + (threadIdx.x >> 5);
    if (unit >= 2 * a.Hkv) return;
    const bool is_key = unit < a.Hkv;
    const int h = is_key ? unit : unit - a.Hkv;
    const int chunk = lane % CPR, t0 = lane / CPR;
    const auto *src = static_cast<const __nv_bfloat16 *>(is_key ? a.k_new : a.v_new) + ((size_t)b * a.Hkv + h) * D + chunk * 16;
    uint4 x[2] = {ld_nc_v4(src), ld_nc_v4(src + 8)};
    const int32_t L = a.seq_lens[b], row = a.page_ptr[b];
    if (L < 1 || L > a.max_pages * a.P) {
        if (unit == 0 && lane == 0) set_err(a.err, VX_DATA_BAD_SEQ_LEN);
        return;
    }
    const int slot = (L - 1) & (a.P - 1);
    const int32_t id = a.page_indices[row + (L - 1) / a.P];
    if (id < 0 || id >= a.num_pool_pages) {
        if (lane == 0) set_err(a.err, VX_DATA_BAD_PAGE_ID);
        return;
    }
    const size_t blk = (size_t)id * a.Hkv + h;
    uint8_t *codes = (is_key ? qa.k_cache : qa.v_cache) + blk * a.P * D + chunk * 16;
    float *scale = (is_key ? qa.k_scale : qa.v_scale) + blk;
    const float s_old = slot > 0 ? *scale : 0.f;
    uint4 old[NR];
    auto load_old = [&]() {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            old[i] = make_uint4(0u, 0u, 0u, 0u);
            if (t0 + i * RPL < slot) old[i] = *reinterpret_cast<const uint4 *>(codes + (t0 + i * RPL) * D);
        }
    };
    if (is_key) load_old();
    const uint32_t amax = largest<2>(x, a.err, lane);
    const float s = fmaxf(scale_of<FMT>(amax), s_old), inv = 1.f / s;
    float f[16];
    bf16x8_to_f32(x[0], reinterpret_cast<float(&)[8]>(f));
    bf16x8_to_f32(x[1], reinterpret_cast<float(&)[8]>(f[8]));
    uint32_t c[4], bits[4];
    // the product is rounded to fp32 before it is rounded to a code, as in quant_unit: under a scale that
    // is no power of two one rounding less gives other int8 codes (9 of 4 million random values)
#pragma unroll
    for (int e = 0; e < 16; ++e) f[e] = __fmul_rn(f[e], inv);
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] = four_codes<FMT>(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3], 1.f, bits);
    if (slot > 0 && s > s_old) {  // the older codes in the new scale
        const float ratio = s_old / s;
#pragma unroll 1
        for (int i = 0; i < NR; ++i) {
            if (t0 + i * RPL >= slot) break;
            uint32_t w[4];
            const uint4 o = *reinterpret_cast<const uint4 *>(codes + (t0 + i * RPL) * D);
            const uint32_t v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    w[e] |= float_to_code<FMT>(code_to_float<FMT>((v[e] >> (8 * u)) & 0xff) * ratio) << (8 * u);
            }
            *reinterpret_cast<uint4 *>(codes + (t0 + i * RPL) * D) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (is_key) load_old();  // this lane's own stores
    }
    const bool owner = t0 == slot % RPL;  // of the new row's chunk
    if (owner) *reinterpret_cast<uint4 *>(codes + slot * D) = make_uint4(c[0], c[1], c[2], c[3]);
    if (lane == 0) *scale = s;
    if (!is_key) return;
    // sums of the codes, 16 columns per lane
    float sum[16];
    if constexpr (FMT == VX_QUANT_INT8) {
        // code + 128 in 16-bit halves: at most 64 rows of 255
        uint32_t even[4] = {}, odd[4] = {};
        auto add = [&](const uint32_t (&w)[4]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t u = w[e] ^ 0x80808080u;
                even[e] += u & 0x00ff00ffu;
                odd[e] += (u >> 8) & 0x00ff00ffu;
            }
        };
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (t0 + i * RPL < slot) {
                const uint32_t w[4] = {old[i].x, old[i].y, old[i].z, old[i].w};
                add(w);
            }
        if (owner) add(c);
#pragma unroll
        for (int off = CPR; off < 32; off <<= 1)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                even[e] += __shfl_xor_sync(FULL, even[e], off);
                odd[e] += __shfl_xor_sync(FULL, odd[e], off);
            }
        const int bias = 128 * (slot + 1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            sum[4 * e] = static_cast<float>((int)(even[e] & 0xffffu) - bias);
            sum[4 * e + 1] = static_cast<float>((int)(odd[e] & 0xffffu) - bias);
            sum[4 * e + 2] = static_cast<float>((int)(even[e] >> 16) - bias);
            sum[4 * e + 3] = static_cast<float>((int)(odd[e] >> 16) - bias);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) sum[e] = 0.f;
        auto add = [&](const uint32_t (&w)[4]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t v = (w[e >> 1] >> (16 * (e & 1))) & 0xffffu;
                const __half2 h2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(v), __NV_E4M3));
                sum[2 * e] += __low2float(h2);
                sum[2 * e + 1] += __high2float(h2);
            }
        };
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const uint32_t w[4] = {old[i].x, old[i].y, old[i].z, old[i].w};  // zeros past the older rows
            add(w);
        }
        if (owner) add(c);
#pragma unroll
        for (int off = CPR; off < 32; off <<= 1)
#pragma unroll
            for (int e = 0; e < 16; ++e) sum[e] += __shfl_xor_sync(FULL, sum[e], off);
    }
    // every row lane holds all 16 sums: row lane r writes words r, r + RPL, ... of the chunk's 8
    // (taken out of the registers first: the arithmetic runs once for all lanes)
    auto *cen = reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(a.centroids) + blk * D + chunk * 16);
    const bool plain = plain_scale(s);
#pragma unroll
    for (int j = 0; j < 8 / RPL; ++j) {
        float x0 = 0.f, x1 = 0.f;
#pragma unroll
        for (int r = 0; r < RPL; ++r)
            if (r == t0) {
                x0 = sum[2 * (j * RPL + r)];
                x1 = sum[2 * (j * RPL + r) + 1];
            }
        cen[j * RPL + t0] = centroid_bits(plain, s, x0, slot + 1) | (centroid_bits(plain, s, x1, slot + 1) << 16);
    }
}

template <int D, int P, int FMT>
cudaError_t launch_qdpf(const CentroidArgs &a, const QuantArgs &qa, int mode, cudaStream_t s) {
    if (mode == CEN_APPEND) {
        const dim3 grid((2 * a.Hkv + QZ_WARPS - 1) / QZ_WARPS, a.B);
        return launch_k(k_quant_append<D, P * D / 512, FMT>, grid, dim3(QZ_WARPS * 32), 0, s, true, a, qa);
    } else {
        // a block takes one set of units after the other when there are many; a small write spreads
        // over the GPU (one request of 3,000 tokens on 4 heads, 64-token pages: 73 us with 8 pages
        // per block).  A request touches at most its new rows / P + 2 pages.
        constexpr int UNITS = QZ_WARPS / (P / 16);
        const int64_t pages = std::min(qa.num_new / P + 2 * (int64_t)a.B, (int64_t)a.B * a.max_pages);
        const int64_t sets = (pages * a.Hkv * 2 + UNITS - 1) / UNITS;
        const int64_t resident = (int64_t)std::max(1, current_sm_count()) * 4;
        const int64_t steps = std::min<int64_t>(QZ_MAX_STEPS, std::max<int64_t>(1, sets / (4 * resident)));
        const int64_t blocks = (sets + steps - 1) / steps;
        if (blocks > INT32_MAX) return cudaErrorInvalidValue;
        static std::atomic<unsigned long long> done;
        const cudaError_t e = ensure_smem_limit(k_quant_prefill<D, P / 16, FMT>, 4096 * (int)sizeof(int4), done);
        if (e != cudaSuccess) return e;
        return launch_k(k_quant_prefill<D, P / 16, FMT>, dim3((unsigned)blocks), dim3(QZ_WARPS * 32),
                        (size_t)a.B * sizeof(int4), s, true, a, qa, (int)(steps * UNITS));
    }
}

template <int D, int P>
cudaError_t launch_qdp(const CentroidArgs &a, const QuantArgs &qa, int mode, cudaStream_t s) {
    return qa.format == VX_QUANT_INT8 ? launch_qdpf<D, P, VX_QUANT_INT8>(a, qa, mode, s)
                                      : launch_qdpf<D, P, VX_QUANT_E4M3>(a, qa, mode, s);
}

template <int D>
cudaError_t launch_qd(const CentroidArgs &a, const QuantArgs &qa, int mode, cudaStream_t s) {
    switch (a.P) {
        case 16: return launch_qdp<D, 16>(a, qa, mode, s);
        case 32: return launch_qdp<D, 32>(a, qa, mode, s);
        case 64: return launch_qdp<D, 64>(a, qa, mode, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_quant_update(const CentroidArgs &a, const QuantArgs &qa, int mode, cudaStream_t s) {
    switch (a.Dqk) {
        case 64: return launch_qd<64>(a, qa, mode, s);
        case 128: return launch_qd<128>(a, qa, mode, s);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace vx
