// vx_common.cuh -- device helpers shared by the libvx kernels (sm_100a only).
//
// Inline-PTX wrappers for the Blackwell data path the kernels use: mbarrier
// transaction barriers, TMA tensor loads (cp.async.bulk.tensor, never with cluster
// multicast), ldmatrix / mma.sync / movmatrix for the small Q.K^T and P.V tiles,
// programmatic dependent launch, and bounded waits.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/vx.h"

#if defined(__CUDA_ARCH__) && (__CUDA_ARCH__ < 1000)
#error "libvx is built for sm_100a only"
#endif

namespace vx {

constexpr unsigned FULL = 0xffffffffu;
// A bounded wait gives up after this many nanoseconds of %globaltimer.
constexpr unsigned long long WAIT_LIMIT_NS = 2000000000ull;

__device__ __forceinline__ void set_err(int32_t *err, unsigned bits) {
    if (err) atomicOr(reinterpret_cast<unsigned *>(err), bits);
}

__device__ __forceinline__ unsigned long long globaltimer() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ------------------------------------------------------------------- PDL

// Wait until the previous kernel on the stream has finished and its writes are visible.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Let the next grid on the stream launch now (it still waits in pdl_wait for this grid's end
// and writes).  Only the top-k kernel triggers, late in each block: its dependent (the decode
// kernel) lands as top-k blocks leave and runs its prologue meanwhile.  Measured without
// gain: a trigger in the scorer (with many rows the top-k blocks beside a scorer block compete
// with it, -10% on the headline step; with the MLA batch's 16 rows, 39.9 against 34.6 us per
// step), at the GQA decode kernel's start (slower) or after its last loads, and in the MLA
// decode kernel once its producer has issued the last copy.  Without a trigger, the next grid
// launches at block exit.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------------- mbarrier

__device__ __forceinline__ void mbar_init(uint32_t bar, unsigned count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void fence_mbar_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, unsigned parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, unsigned parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// try_wait with a suspend-time hint: the thread may sleep (issuing nothing) for up to about
// `hint_ns` nanoseconds, and is woken when the phase completes.
__device__ __forceinline__ bool mbar_try_wait_hint(uint32_t bar, unsigned parity, uint32_t hint_ns) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(hint_ns)
        : "memory");
    return ok != 0;
}
// Wait for phase `parity` of the barrier to complete, for at most about WAIT_LIMIT_NS.
// Short waits spin on the non-blocking test_wait (a data tile usually lands within a
// microsecond); longer ones fall back to try_wait, which may suspend the thread, and
// read the (slow) global timer only every 1024 tries.
__device__ __forceinline__ bool mbar_wait_bounded(uint32_t bar, unsigned parity) {
    for (int i = 0; i < 4096; ++i)
        if (mbar_test_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (;;) {
        for (int i = 0; i < 1024; ++i)
            if (mbar_try_wait(bar, parity)) return true;
        if (globaltimer() - t0 > WAIT_LIMIT_NS) return false;
    }
}

// Like mbar_wait_bounded, but a waiter that misses the first test sleeps in try_wait with a
// suspend hint instead of spinning, leaving the issue slots to the warps doing math.
__device__ __forceinline__ bool mbar_wait_sleep(uint32_t bar, unsigned parity) {
    if (mbar_test_wait(bar, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try_wait_hint(bar, parity, 1000u)) return true;
        if (globaltimer() - t0 > WAIT_LIMIT_NS) return false;
    }
}

// ------------------------------------------------------------------- TMA

// 3-D tiled tensor load global -> shared, completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y, int z,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
// Bring the 128-byte line holding p into L2; returns nothing, so it cannot hand a thread data
// that another grid is still writing (loads after a dependency wait read the updated line).
__device__ __forceinline__ void prefetch_l2(const void *p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(p)) : "memory");
}
__device__ __forceinline__ void tma_prefetch_desc(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}

// Byte offset of 16-byte chunk `chunk` (0..7) of row `row` inside a tile written by TMA
// with 128-byte swizzling: rows are 128 bytes, chunks are XOR-permuted by row % 8.
__device__ __forceinline__ uint32_t swz128(int row, int chunk) {
    return static_cast<uint32_t>(row * 128 + ((chunk ^ (row & 7)) << 4));
}

// ------------------------------------------------------------------- warp MMA

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                        uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                          uint32_t &r3) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}
// D = A(16x16, row) * B(16x8, col) + D, bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                               uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose an 8x8 b16 matrix held in the mma fragment layout.
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

// ------------------------------------------------------------------- loads

// 16-byte read-only load; an intrinsic rather than volatile asm so the compiler may issue
// several before the first is used.
__device__ __forceinline__ uint4 ld_nc_v4(const void *p) { return __ldg(reinterpret_cast<const uint4 *>(p)); }
// 8 bf16 packed in a uint4 -> 8 floats (exact widening)
__device__ __forceinline__ void bf16x8_to_f32(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// Round a double to the nearest bf16, ties to even, directly from the double.
__device__ __forceinline__ uint16_t f64_to_bf16_rne(double x) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
    const uint16_t sign = static_cast<uint16_t>((u >> 48) & 0x8000u);
    const int ebits = static_cast<int>((u >> 52) & 0x7ff);
    if (ebits == 0x7ff) return (u & 0xfffffffffffffull) ? uint16_t(0x7fc0) : uint16_t(sign | 0x7f80);
    const double ax = fabs(x);
    if (ax == 0.0) return sign;
    const int e = ebits - 1023;  // ax in [2^e, 2^(e+1)) for normal doubles (ours always are)
    if (e < -126) {
        // bf16 subnormal range: spacing 2^-133
        const long long q = __double2ll_rn(ax * 0x1p133);  // exact scaling, RNE to integer
        return static_cast<uint16_t>(sign | static_cast<uint16_t>(q));  // q == 128 -> min normal
    }
    // 8 significant bits: scale into [128, 256) and round to an integer, ties to even
    long long q = __double2ll_rn(scalbn(ax, 7 - e));
    int ee = e;
    if (q == 256) {
        q = 128;
        ++ee;
    }
    if (ee > 127) return static_cast<uint16_t>(sign | 0x7f80);
    return static_cast<uint16_t>(sign | ((ee + 127) << 7) | (static_cast<int>(q) & 0x7f));
}

__device__ __forceinline__ int32_t ceil_div(int32_t a, int32_t b) { return (a + b - 1) / b; }

}  // namespace vx
