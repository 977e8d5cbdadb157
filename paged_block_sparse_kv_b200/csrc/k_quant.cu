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
// One unit is the keys or the values of one (page, KV head).  Its page_size / 16 warps hold 16
// token rows each in registers (a lane: 16-byte chunks of rows, as they lie in memory), take
// the largest magnitude with a warp reduction (and through shared memory when the unit has
// several warps), convert, and store; nothing is read twice.  HBM bound: 2 bytes read and 1
// written per element.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "vx_internal.h"

namespace vx {

namespace {

constexpr int QZ_WARPS = 8;
constexpr int QZ_PAGES_PER_BLOCK = 8;  // prefill: pages per block

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

// One unit, by its WPU warps (this warp: rows [16 * part, 16 * part + 16)).  Rows [0, n_old) are
// the page's older tokens, [n_old, m) come from new_row(t).  `go`: the unit exists (warps of
// missing units only take part in the block barriers).
template <int D, int WPU, int FMT, typename RowF>
__device__ __forceinline__ void quant_unit(bool go, bool is_key, int part, RowF new_row, uint8_t *__restrict__ codes,
                                           float *__restrict__ scale, __nv_bfloat16 *__restrict__ cen, int n_old,
                                           int m, int32_t *err, int lane, uint32_t *s_max, float (*s_sum)[D]) {
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
        if (go && t >= n_old && t < m) x[i] = ld_nc_v4(new_row(t) + chunk * 8);
    }
    if (go && n_old > 0) {
        s_old = *scale;
        if (is_key) {
#pragma unroll
            for (int i = 0; i < NR; ++i)
                if (t0 + i * RPL < n_old) old[i] = *reinterpret_cast<const uint2 *>(codes + (t0 + i * RPL) * D + chunk * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const uint32_t a = __vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu);
        const uint32_t b = __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu);
        const uint32_t c = __vmaxu2(a, b);
        amax = max(amax, max(c & 0xffffu, c >> 16));
    }
    amax = __reduce_max_sync(FULL, amax);
    if (amax >= 0x7f80u) {  // an infinity becomes the largest finite value, a NaN zero
        if (lane == 0) set_err(err, VX_DATA_BAD_VALUE);
        amax = 0;
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t h[2] = {w[j] & 0xffffu, w[j] >> 16};
#pragma unroll
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
        amax = __reduce_max_sync(FULL, amax);
    }
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
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t lo = f64_to_bf16_rne((double)s * sum[2 * e] / m);
                const uint32_t hi = f64_to_bf16_rne((double)s * sum[2 * e + 1] / m);
                w[e] = lo | (hi << 16);
            }
            *reinterpret_cast<uint4 *>(cen + chunk * 8) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Prefill write: grid (ceil(max_pages / QZ_PAGES_PER_BLOCK), B), from the page holding first_pos[b]
// on.  Append: grid (ceil(2 Hkv WPU / QZ_WARPS), B), first_pos = L - 1, one new row per request.
template <int D, int WPU, int FMT, bool APPEND>
__global__ void __launch_bounds__(QZ_WARPS * 32) k_quant_update(const CentroidArgs a, const QuantArgs qa) {
    constexpr int UNITS = QZ_WARPS / WPU;  // units in flight per block
    __shared__ uint32_t s_max[QZ_WARPS];
    __shared__ float s_sum[WPU > 1 ? QZ_WARPS : 1][D];
    const int b = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // a dependent scorer (vx_block_topk_decode_append_quant) may launch now; it waits for this
    // grid's end and writes before it reads anything
    if constexpr (APPEND) pdl_trigger();
    int64_t row0 = b;  // packed row of request b's first new token
    const int32_t L = a.seq_lens[b];
    int32_t fp = L - 1;
    if constexpr (!APPEND) {
        __shared__ long long s_part[QZ_WARPS];
        long long part = 0;
        for (int i = threadIdx.x; i < b; i += blockDim.x) part += prefill_count(a, i);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) part += __shfl_xor_sync(FULL, part, off);
        if (lane == 0) s_part[warp] = part;
        __syncthreads();
        row0 = 0;
#pragma unroll
        for (int w = 0; w < QZ_WARPS; ++w) row0 += s_part[w];
        fp = a.first_pos[b];
    }
    if (L < 1 || L > a.max_pages * a.P || fp < 0 || fp > L || (!APPEND && row0 + (L - fp) > qa.num_new)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) set_err(a.err, VX_DATA_BAD_SEQ_LEN);
        return;
    }
    const int n = ceil_div(L, a.P);
    const int j_lo = fp / a.P + (APPEND ? 0 : blockIdx.x * QZ_PAGES_PER_BLOCK);
    const int j_hi = APPEND ? j_lo + 1 : min(n, j_lo + QZ_PAGES_PER_BLOCK);
    if (fp == L || j_lo >= n) return;
    const int items = (j_hi - j_lo) * a.Hkv * 2;
    const auto *kn = static_cast<const __nv_bfloat16 *>(a.k_new);
    const auto *vn = static_cast<const __nv_bfloat16 *>(a.v_new);
    auto *cen = static_cast<__nv_bfloat16 *>(a.centroids);
    const int it_lo = APPEND ? blockIdx.x * UNITS : 0;
    const int it_hi = APPEND ? min(items, it_lo + UNITS) : items;
    for (int it0 = it_lo; it0 < it_hi; it0 += UNITS) {
        const int it = it0 + warp / WPU;
        bool go = it < it_hi;
        const int j = j_lo + (go ? it / (2 * a.Hkv) : 0), rem = go ? it % (2 * a.Hkv) : 0;
        const bool is_key = rem < a.Hkv;
        const int h = is_key ? rem : rem - a.Hkv;
        int32_t phys = go ? a.page_indices[a.page_ptr[b] + j] : 0;
        if (phys < 0 || phys >= a.num_pool_pages) {
            if (lane == 0) set_err(a.err, VX_DATA_BAD_PAGE_ID);
            go = false;
            phys = 0;
        }
        const int m = min(a.P, L - j * a.P);
        const int n_old = max(0, fp - j * a.P);
        const size_t blk = (size_t)phys * a.Hkv + h;
        const __nv_bfloat16 *src = (is_key ? kn : vn) + ((row0 + (int64_t)j * a.P - fp) * a.Hkv + h) * D;
        quant_unit<D, WPU, FMT>(
            go, is_key, warp % WPU, [&](int t) { return src + (int64_t)t * a.Hkv * D; },
            (is_key ? qa.k_cache : qa.v_cache) + blk * a.P * D, (is_key ? qa.k_scale : qa.v_scale) + blk,
            cen + blk * D, n_old, m, a.err, lane, s_max, s_sum);
    }
}

template <int D, int WPU, int FMT>
cudaError_t launch_qdwf(const CentroidArgs &a, const QuantArgs &qa, int mode, cudaStream_t s) {
    if (mode == CEN_APPEND) {
        const dim3 grid((2 * a.Hkv * WPU + QZ_WARPS - 1) / QZ_WARPS, a.B);
        k_quant_update<D, WPU, FMT, true><<<grid, QZ_WARPS * 32, 0, s>>>(a, qa);
    } else {
        const dim3 grid((a.max_pages + QZ_PAGES_PER_BLOCK - 1) / QZ_PAGES_PER_BLOCK, a.B);
        k_quant_update<D, WPU, FMT, false><<<grid, QZ_WARPS * 32, 0, s>>>(a, qa);
    }
    return cudaGetLastError();
}

template <int D, int WPU>
cudaError_t launch_qdw(const CentroidArgs &a, const QuantArgs &qa, int mode, cudaStream_t s) {
    return qa.format == VX_QUANT_INT8 ? launch_qdwf<D, WPU, VX_QUANT_INT8>(a, qa, mode, s)
                                      : launch_qdwf<D, WPU, VX_QUANT_E4M3>(a, qa, mode, s);
}

template <int D>
cudaError_t launch_qd(const CentroidArgs &a, const QuantArgs &qa, int mode, cudaStream_t s) {
    switch (a.P) {
        case 16: return launch_qdw<D, 1>(a, qa, mode, s);
        case 32: return launch_qdw<D, 2>(a, qa, mode, s);
        case 64: return launch_qdw<D, 4>(a, qa, mode, s);
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
