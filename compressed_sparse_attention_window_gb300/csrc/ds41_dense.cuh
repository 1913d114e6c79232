// ds41_dense.cuh - what the dense-attention entry points share: the paged
// key/value cache as kernels see it, the argument checks of its layout, and
// the conversions that more than one kernel uses.  Nothing here is shared with the CPU oracle.
#pragma once

#include <atomic>

#include "ds41_common.cuh"
#include "ds41_internal.cuh"

namespace ds41 {

// A paged cache: [n_pages][kvh][page][hd] values (bf16 or e4m3 codes) of K and
// V, and for e4m3 the f32 scales [n_pages][kvh][page].
struct PagedKv {
    const uint8_t* k;
    const uint8_t* v;
    const float* ks;  // null for bf16
    const float* vs;
    int64_t n_pages;
    int page, page_shift, kvh, hd;
};

// Host: a cache's format, heads and head width.
int check_cache_form(const char* name, int fmt, int64_t kvh, int64_t hd);
// Host: checks a cache's layout (DS41_E_ARG with a message) and fills `out`.
int check_paged(const char* name, const void* k, const void* v, const float* ks, const float* vs,
                int fmt, int64_t n_pages, int64_t page, int64_t kvh, int64_t hd, PagedKv* out);

// Host: the heads' counts, the head width, scale and window of a call.
int check_heads(const char* name, int64_t nh, int64_t kvh, int64_t hd, float scale,
                int64_t window);
// A window of 2^31 or more holds every sequence: none (sums and differences of a window
// and positions then stay far from the end of 64 bits).
inline int64_t finite_window(int64_t window) { return window >> 31 ? 0 : window; }
// strides between tokens and between heads, in elements
inline bool good_strides(int64_t tok, int64_t head, int64_t hd) {
    return tok % 8 == 0 && head % 8 == 0 && head >= hd && tok >= hd;
}
inline bool aligned_to(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// Host: a kernel's dynamic shared memory limit, raised once per device.
template <auto KERNEL>
int allow_smem(int bytes, const char* what) {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    if (int rc = cuda_check(cudaGetDevice(&dev), what)) return rc;
    if (dev < 64 && ((done.load(std::memory_order_relaxed) >> dev) & 1)) return DS41_OK;
    if (int rc = cuda_check(
            cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes), what))
        return rc;
    if (dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
    return DS41_OK;
}
// Host: the current device's SM count, looked up once per device.
inline int sm_count_once() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return device_sm_count();
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) known[dev].store(n = device_sm_count(), std::memory_order_relaxed);
    return n;
}

// two f32 operations in one instruction
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// First element of row `off` of page `pg`, head `h`, counted in elements.
// 64-bit: a cache of a few million rows passes 2^31 elements.
__device__ __forceinline__ int64_t paged_row(const PagedKv& c, int64_t pg, int h, int off) {
    return (pg * c.kvh + h) * c.page + off;
}

// c += a b of 16 x 8 x 16 as mma_bf16, with f16 operands
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes -> their exact values as f16 (every e4m3 value is a normal f16
// or zero): lo = codes 0, 1, hi = codes 2, 3.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\n"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

// The exponent that brings a row of queries with the largest magnitude amax (bf16
// bits) to [2^14, 2^15), so that bf16 values become f16 exactly down to 2^-28 of
// it (at least -120: below 2^-106 the row becomes smaller f16 values, still
// exact); 0 for a row of zeros or one that is not finite.
__device__ __forceinline__ int query_exponent(uint32_t amax_bits) {
    const int e = (int)(amax_bits >> 7);
    return e == 0 || e == 255 ? 0 : max(e - 127 - 14, -120);
}
// two bf16 times 2^-e as f16
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t x, float down) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;"
        : "=r"(r)
        : "f"(__uint_as_float(x & 0xffff0000u) * down), "f"(__uint_as_float(x << 16) * down));
    return r;
}

}  // namespace ds41
