// ds41_kv_cache.cu - the paged key/value cache: rows quantised (or copied) as
// they are written, and read back as bf16.
//
// Mathematics.  An e4m3 row x[0..hd) of one token and head keeps one scale
//   s = max(amax |x|, 448 * 2^-126) / 448        (f32, correctly rounded)
// and the codes e4m3(x / s), to nearest, ties to the even code.  448 is the
// largest e4m3 value, so the largest element gets the largest code; the floor
// keeps s a normal number, so a zero row has codes +-0.  A row that holds a NaN
// or an infinity keeps the scale NaN and zero codes: whatever reads it sees NaN.
// Reading back is bf16(code * s), the product rounded to f32 first.
//
// Both kernels move bytes and little else.
#include "ds41_dense.cuh"

namespace ds41 {

int check_cache_form(const char* name, int fmt, int64_t kvh, int64_t hd) {
    DS41_REQUIRE(fmt == DS41_KV_BF16 || fmt == DS41_KV_E4M3, DS41_E_ARG,
                 "%s: fmt=%d is neither DS41_KV_BF16 nor DS41_KV_E4M3", name, fmt);
    DS41_REQUIRE(kvh >= 1 && kvh <= 1024 && hd >= 16 && hd <= 128 && hd % 16 == 0, DS41_E_ARG,
                 "%s: kvh=%lld hd=%lld (hd a multiple of 16, at most 128)", name, (long long)kvh,
                 (long long)hd);
    return DS41_OK;
}

int check_paged(const char* name, const void* k, const void* v, const float* ks, const float* vs,
                int fmt, int64_t n_pages, int64_t page, int64_t kvh, int64_t hd, PagedKv* out) {
    if (int rc = check_cache_form(name, fmt, kvh, hd)) return rc;
    DS41_REQUIRE(page >= 16 && page <= 256 && (page & (page - 1)) == 0, DS41_E_ARG,
                 "%s: page=%lld must be a power of two of 16 .. 256", name, (long long)page);
    DS41_REQUIRE(n_pages >= 1 && n_pages < (int64_t(1) << 31) / kvh, DS41_E_ARG,
                 "%s: n_pages=%lld kvh=%lld", name, (long long)n_pages, (long long)kvh);
    DS41_REQUIRE(k && v && aligned16(k) && aligned16(v), DS41_E_ARG,
                 "%s: the caches must be non-null and 16-byte aligned", name);
    if (fmt == DS41_KV_E4M3)
        DS41_REQUIRE(ks && vs && aligned16(ks) && aligned16(vs), DS41_E_ARG,
                     "%s: an e4m3 cache needs its scales (non-null, 16-byte aligned)", name);
    out->k = static_cast<const uint8_t*>(k);
    out->v = static_cast<const uint8_t*>(v);
    out->ks = fmt == DS41_KV_E4M3 ? ks : nullptr;
    out->vs = fmt == DS41_KV_E4M3 ? vs : nullptr;
    out->n_pages = n_pages;
    out->page = (int)page;
    out->page_shift = 0;
    while ((1 << out->page_shift) < page) out->page_shift++;
    out->kvh = (int)kvh;
    out->hd = (int)hd;
    return DS41_OK;
}

int check_heads(const char* name, int64_t nh, int64_t kvh, int64_t hd, float scale,
                int64_t window) {
    DS41_REQUIRE(kvh >= 1 && nh >= kvh && nh % kvh == 0 && nh <= 4096, DS41_E_ARG,
                 "%s: nh=%lld must be a multiple of kvh=%lld (at most 4096)", name, (long long)nh,
                 (long long)kvh);
    DS41_REQUIRE(hd >= 16 && hd <= 128 && hd % 16 == 0, DS41_E_ARG,
                 "%s: hd=%lld must be a multiple of 16 of at most 128", name, (long long)hd);
    // (the kernels take scale log2(e))
    DS41_REQUIRE(scale > 0.0f && scale <= 0x1p127f, DS41_E_ARG,
                 "%s: scale=%g must be positive and at most 2^127", name, (double)scale);
    DS41_REQUIRE(window >= 0, DS41_E_ARG, "%s: window=%lld", name, (long long)window);
    return DS41_OK;
}

namespace {

constexpr int THREADS = 256;

// CTAs are numbered by head first, then by block of rows, in two dimensions of the
// grid as one holds 65535.
__device__ __forceinline__ int64_t row_block() {
    return (int64_t)blockIdx.z * gridDim.y + blockIdx.y;
}
dim3 row_grid(int64_t kvh, int64_t rows, int64_t per) {
    const int64_t blocks = (rows + per - 1) / per, nz = (blocks + 65534) / 65535;
    return dim3((unsigned)kvh, (unsigned)((blocks + nz - 1) / nz), (unsigned)nz);
}

// Two quotients x / s, correctly rounded, from the correctly rounded reciprocal r of s:
// with q = x r within one unit of the quotient, q + r (x - q s), the remainder exact in
// a fused multiply-add, rounds as the quotient does (P. Markstein, Computation of
// elementary functions on the IBM RISC System/6000 processor, 1990).  A quotient of
// -0 comes out as +0.
__device__ __forceinline__ uint64_t quotients(uint64_t x, uint64_t minus_s, uint64_t r) {
    const uint64_t q = mul2(x, r);
    return fma2(fma2(q, minus_s, x), r, q);
}
// x / 448, correctly rounded, by the same rule (x is at least 448 * 2^-126).
__device__ __forceinline__ float by_448(float x) {
    constexpr float R = 1.0f / 448.0f;
    const float q = __fmul_rn(x, R);
    return __fmaf_rn(__fmaf_rn(q, -448.0f, x), R, q);
}

struct WriteArgs {
    const uint16_t* x[2];  // k, v
    int64_t stride[2];     // elements from a token's rows to the next token's
    uint8_t* cache[2];
    float* scales[2];
    const int64_t* slots;
    int64_t n, n_slots;
    int kvh, hd, page, page_shift;
    unsigned int* status;
};

// L lanes take one (token, head): 8 elements of its K row and of its V row each, so
// both rows' loads are in flight together; a CTA has one head of consecutive
// tokens.  What bounds it is the instructions as much as the bytes, so the maxima of
// K and V share their exchanges, each half of the lanes works out one of the two
// scales, and the quotients go two at a time.  (16383 tokens of 8
// heads of 128, 101 MB: 22.6 us of GPU time, two thirds of the copy rate, the issue
// slots 62% busy; 30.6 us with a maximum, a scale and a division for each.  Two and
// four rows a thread, heads innermost, and CTAs of 128 and 512 threads are level or
// slower.)
template <int L, bool E4M3>
__global__ void __launch_bounds__(THREADS) kv_write_kernel(const WriteArgs a) {
    pdl_wait();
    pdl_trigger();
    const int c = (threadIdx.x % L) * 8, h = blockIdx.x;
    const int64_t t = row_block() * (THREADS / L) + threadIdx.x / L;
    const bool mine = t < a.n && c < a.hd;
    const int64_t slot = t < a.n ? a.slots[t] : -1;
    uint4 x[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
        x[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 2; i++)
        if (mine)
            x[i] = __ldcs(reinterpret_cast<const uint4*>(a.x[i] + t * a.stride[i] + h * a.hd + c));
    const bool keep = slot >= 0 && slot < a.n_slots;
    if (!keep && slot != -1 && c == 0 && h == 0) raise_status(a.status, DS41_E_INDEX);
    // (the number of a page and head fits 32 bits: check_paged)
    const int64_t row = ((int64_t)((int)(slot >> a.page_shift) * a.kvh + h) << a.page_shift) +
                        ((int)slot & (a.page - 1));
    if (!E4M3) {
        if (keep && mine)
            for (int i = 0; i < 2; i++)
                *reinterpret_cast<uint4*>(a.cache[i] + (row * a.hd + c) * 2) = x[i];
        return;
    }
    // the rows' largest magnitudes as bf16 bits (ordered like the values; the bits of
    // infinities and NaN are the largest of all): K's in the lower half, V's above
    uint32_t m2[2];
#pragma unroll
    for (int i = 0; i < 2; i++)
        m2[i] = __vmaxu2(__vmaxu2(x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu),
                         __vmaxu2(x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu));
    uint32_t m = __vmaxu2(__byte_perm(m2[0], m2[1], 0x5410), __byte_perm(m2[0], m2[1], 0x7632));
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1)
        m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, off));
    // the lower lanes have K's scale, the upper ones V's.  A scale below 2^-90 and its
    // row are taken 2^100 times: the remainders stay normal numbers.
    const int l = threadIdx.x % L, own = l / (L / 2);
    const uint32_t m_own = own ? m >> 16 : m & 0xffffu;
    const float s_own = by_448(fmaxf(bf2f((uint16_t)m_own), 448.0f * 0x1p-126f));
    const float up = s_own < 0x1p-90f ? 0x1p100f : 1.0f;
    const float r_own = __frcp_rn(s_own * up);
    if (keep && mine && l == own * (L / 2))
        (own ? a.scales[1] : a.scales[0])[row] =
            m_own < 0x7f80u ? s_own : __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const float s = __shfl_sync(0xffffffffu, s_own * up, i * (L / 2), L);
        const float r = __shfl_sync(0xffffffffu, r_own, i * (L / 2), L);
        const float f = __shfl_sync(0xffffffffu, up, i * (L / 2), L);
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint64_t y[4];
#pragma unroll
        for (int e = 0; e < 4; e++)
            y[e] = f2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
        if (f != 1.0f) {
#pragma unroll
            for (int e = 0; e < 4; e++) y[e] = mul2(y[e], f2(f, f));
        }
        uint16_t two[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            float lo, hi;
            unf2(quotients(y[e], f2(-s, -s), f2(r, r)), lo, hi);
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(two[e]) : "f"(hi), "f"(lo));
        }
        uint2 codes;  // (with the signs of the elements: a zero keeps its own)
        codes.x = (two[0] | (uint32_t)two[1] << 16) |
                  (__byte_perm(w[0], w[1], 0x7531) & 0x80808080u);
        codes.y = (two[2] | (uint32_t)two[3] << 16) |
                  (__byte_perm(w[2], w[3], 0x7531) & 0x80808080u);
        if ((i ? m >> 16 : m & 0xffffu) >= 0x7f80u) codes = make_uint2(0, 0);
        if (keep && mine)
            *reinterpret_cast<uint2*>(a.cache[i] + row * a.hd + c) = codes;
    }
}

struct ReadArgs {
    PagedKv kv;
    const int32_t* table;
    const int32_t* cu;
    const int32_t* starts;
    uint16_t* out[2];
    int64_t rows;
    int B, max_pages;
    unsigned int* status;
};

// L lanes take one (row, head), 16 elements of K and of V each; the rows of a CTA
// are consecutive, as they lie in a page.  (33000 rows of 8 heads of 128, 205 MB: 38
// us of GPU time, 79% of the copy rate.)
template <int L, bool E4M3>
__global__ void __launch_bounds__(THREADS) kv_read_kernel(const ReadArgs a) {
    pdl_wait();
    pdl_trigger();
    const int h = blockIdx.x, c = (threadIdx.x % L) * 16;
    const int64_t r = row_block() * (THREADS / L) + threadIdx.x / L;
    if (h == 0 && row_block() == 0)  // one CTA reports the sequences that break their limits
        for (int i = threadIdx.x; i < a.B; i += THREADS)
            if (a.cu[i] < 0 || a.cu[i + 1] < a.cu[i] || a.cu[i + 1] > a.rows)
                raise_status(a.status, DS41_E_INDEX);
    if (c >= a.kv.hd || r >= a.rows) return;
    int b = 0, end = a.B;  // the last b with cu[b] <= r
    while (end - b > 1) {
        const int mid = (b + end) >> 1;
        if (a.cu[mid] <= r) b = mid;
        else end = mid;
    }
    const int64_t first = a.cu[b], last = a.cu[b + 1];
    // before the first sequence, behind the last: nobody's
    if (r < first || r >= last || first < 0 || last > a.rows) return;
    const int64_t pos = r - first + (a.starts ? a.starts[b] : 0);
    const int64_t pi = pos >> a.kv.page_shift;
    int64_t pg = -1;
    if (pos >= 0 && pi < a.max_pages) pg = a.table[(int64_t)b * a.max_pages + pi];
    const bool ok = pg >= 0 && pg < a.kv.n_pages;
    if (!ok) raise_status(a.status, DS41_E_INDEX);
    const int64_t row = paged_row(a.kv, ok ? pg : 0, h, (int)pos & (a.kv.page - 1));
    uint4 in[2][2];
    float s[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint8_t* src = i ? a.kv.v : a.kv.k;
        in[i][0] = in[i][1] = make_uint4(0, 0, 0, 0);
        s[i] = 0.0f;
        if (!ok) continue;
        if (E4M3) {
            in[i][0] = __ldcs(reinterpret_cast<const uint4*>(src + row * a.kv.hd + c));
            s[i] = (i ? a.kv.vs : a.kv.ks)[row];
        } else {
            const uint4* x = reinterpret_cast<const uint4*>(src + (row * a.kv.hd + c) * 2);
            in[i][0] = __ldcs(x);
            in[i][1] = __ldcs(x + 1);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        uint4* dst = reinterpret_cast<uint4*>(a.out[i] + (r * a.kv.kvh + h) * a.kv.hd + c);
        if (!E4M3) {
            dst[0] = in[i][0];
            dst[1] = in[i][1];
            continue;
        }
        const uint32_t w[4] = {in[i][0].x, in[i][0].y, in[i][0].z, in[i][0].w};
        uint32_t o[8];
#pragma unroll
        for (int e = 0; e < 4; e++) {
            uint32_t h2[2];
            e4m3x4_to_f16(w[e], h2[0], h2[1]);
#pragma unroll
            for (int y = 0; y < 2; y++) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2[y]));
                const __nv_bfloat162 v = __floats2bfloat162_rn(f.x * s[i], f.y * s[i]);
                o[2 * e + y] = *reinterpret_cast<const uint32_t*>(&v);
            }
        }
        dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
        dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
    }
}

// smallest power of two of lanes that covers n vectors (n <= 16)
int lanes_for(int64_t n) { return n <= 1 ? 1 : n <= 2 ? 2 : n <= 4 ? 4 : n <= 8 ? 8 : 16; }

template <bool E4M3>
void (*pick_write(int L))(const WriteArgs) {
    return L == 2 ? kv_write_kernel<2, E4M3>
                  : L == 4 ? kv_write_kernel<4, E4M3>
                           : L == 8 ? kv_write_kernel<8, E4M3> : kv_write_kernel<16, E4M3>;
}
template <bool E4M3>
void (*pick_read(int L))(const ReadArgs) {
    return L == 1 ? kv_read_kernel<1, E4M3>
                  : L == 2 ? kv_read_kernel<2, E4M3>
                           : L == 4 ? kv_read_kernel<4, E4M3> : kv_read_kernel<8, E4M3>;
}

}  // namespace
}  // namespace ds41

using namespace ds41;

extern "C" int ds41_kv_cache_write(const ds41_bf16* k, int64_t k_stride, const ds41_bf16* v,
                                   int64_t v_stride, const int64_t* slots, void* k_cache,
                                   void* v_cache, float* k_scales, float* v_scales, int fmt,
                                   int64_t n_pages, int64_t page, int64_t kvh, int64_t hd,
                                   int64_t n, ds41_stream_t stream) {
    const char* name = "ds41_kv_cache_write";
    PagedKv kv;
    if (int rc = check_paged(name, k_cache, v_cache, k_scales, v_scales, fmt, n_pages, page, kvh,
                             hd, &kv))
        return rc;
    DS41_REQUIRE(n >= 0 && n < (int64_t(1) << 31), DS41_E_RANGE, "%s: n=%lld", name, (long long)n);
    if (n == 0) return DS41_OK;
    DS41_REQUIRE(k && v && aligned16(k) && aligned16(v) && slots && aligned_to(slots, 8),
                 DS41_E_ARG,
                 "%s: k and v must be non-null and 16-byte aligned, slots non-null and aligned",
                 name);
    DS41_REQUIRE(k_stride >= kvh * hd && v_stride >= kvh * hd && k_stride % 8 == 0 &&
                     v_stride % 8 == 0,
                 DS41_E_ARG, "%s: token strides %lld, %lld (at least kvh*hd, multiples of 8)", name,
                 (long long)k_stride, (long long)v_stride);
    WriteArgs a{{k, v},
                {k_stride, v_stride},
                {static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache)},
                {k_scales, v_scales},
                slots,
                n,
                n_pages * page,
                (int)kvh,
                (int)hd,
                (int)page,
                kv.page_shift,
                nullptr};
    if (int rc = status_word(&a.status)) return rc;
    const int L = lanes_for(hd / 8);
    return launch_pdl(fmt == DS41_KV_E4M3 ? pick_write<true>(L) : pick_write<false>(L),
                      row_grid(kvh, n, THREADS / L), dim3(THREADS), 0, (cudaStream_t)stream, name,
                      a);
}

extern "C" int ds41_kv_cache_read(const void* k_cache, const void* v_cache, const float* k_scales,
                                  const float* v_scales, int fmt, int64_t n_pages, int64_t page,
                                  int64_t kvh, int64_t hd, const int32_t* page_table,
                                  int64_t max_pages, const int32_t* cu_k, const int32_t* starts,
                                  int64_t B, ds41_bf16* k, ds41_bf16* v, int64_t rows,
                                  ds41_stream_t stream) {
    const char* name = "ds41_kv_cache_read";
    ReadArgs a{};
    if (int rc = check_paged(name, k_cache, v_cache, k_scales, v_scales, fmt, n_pages, page, kvh,
                             hd, &a.kv))
        return rc;
    DS41_REQUIRE(B >= 0 && B < (int64_t(1) << 31) && rows >= 0 && rows < (int64_t(1) << 31) &&
                     max_pages >= 0 && max_pages < (int64_t(1) << 31),
                 DS41_E_RANGE, "%s: B=%lld rows=%lld max_pages=%lld", name, (long long)B,
                 (long long)rows, (long long)max_pages);
    if (B == 0 || rows == 0) return DS41_OK;
    DS41_REQUIRE(k && v && aligned16(k) && aligned16(v) && cu_k && page_table &&
                     aligned_to(cu_k, 4) && aligned_to(page_table, 4) && aligned_to(starts, 4),
                 DS41_E_ARG,
                 "%s: k and v must be non-null and 16-byte aligned, cu_k and page_table non-null "
                 "and aligned", name);
    a.table = page_table;
    a.cu = cu_k;
    a.starts = starts;
    a.out[0] = k;
    a.out[1] = v;
    a.rows = rows;
    a.B = (int)B;
    a.max_pages = (int)max_pages;
    if (int rc = status_word(&a.status)) return rc;
    const int L = lanes_for(hd / 16);
    return launch_pdl(fmt == DS41_KV_E4M3 ? pick_read<true>(L) : pick_read<false>(L),
                      row_grid(kvh, rows, THREADS / L), dim3(THREADS), 0, (cudaStream_t)stream,
                      name, a);
}
