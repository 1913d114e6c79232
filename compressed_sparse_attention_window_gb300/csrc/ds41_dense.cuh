// ds41_dense.cuh - what the dense-attention entry points share: the paged
// key/value cache as kernels see it, the argument checks of its layout, and
// the e4m3 codec of its rows.  Nothing here is shared with the CPU oracle.
#pragma once

#include "ds41_common.cuh"

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

// Host: checks a cache's layout (DS41_E_ARG with a message) and fills `out`.
int check_paged(const char* name, const void* k, const void* v, const float* ks, const float* vs,
                int fmt, int64_t n_pages, int64_t page, int64_t kvh, int64_t hd, PagedKv* out);

// Host: the heads' counts, the head width, scale and window of a call.
int check_heads(const char* name, int64_t nh, int64_t kvh, int64_t hd, float scale,
                int64_t window);
// strides between tokens and between heads, in elements
inline bool good_strides(int64_t tok, int64_t head, int64_t hd) {
    return tok % 8 == 0 && head % 8 == 0 && head >= hd && tok >= hd;
}
inline bool aligned_to(const void* p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

// First element of row `off` of page `pg`, head `h`, counted in elements.
// 64-bit: a cache of a few million rows passes 2^31 elements.
__device__ __forceinline__ int64_t paged_row(const PagedKv& c, int64_t pg, int h, int off) {
    return (pg * c.kvh + h) * c.page + off;
}

// Two e4m3 codes, in the upper bytes of the halves of x (the lower bytes are
// ignored), as bf16x2, exact.  The code's exponent and mantissa bits moved into
// a bf16's give the value times 2^-120 (exponent bias 7 against 127, subnormals
// included); one exact bf16 product restores it.  The NaN codes 0x7f and 0xff,
// which the cache never holds, would come out as +-480.
__device__ __forceinline__ uint32_t e4m3_spread(uint32_t x) {
    const uint32_t r = (x & 0x80008000u) | ((x >> 4) & 0x07f007f0u);
    uint32_t out;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(out) : "r"(r), "r"(0x7b807b80u));  // 2^120
    return out;
}

}  // namespace ds41
