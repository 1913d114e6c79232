// ds41_pages.cu - the pages of the paged cache: handed out, forked, freed, copied
// and compacted, with the counts of who has them on the device.
//
// Mathematics.  refs[p] counts the sequences that have page p.  Forking adds, for every
// full page of a parent with c children, c (c - 1 if the children replace it); the free
// pages are those at 0, numbered in order by a prefix sum of zeros, and the r-th copy of a
// last page goes to the r-th of them.  Compacting n pages in use pairs the i-th zero
// below n with the i-th count above zero from n on: as many of one as of the other.
//
// What bounds it.  The copies: HBM, two bytes moved for each byte of a page.  What comes
// before them reads a few thousand words, and is a chain of short launches.  (4099 pages of
// 256 KB, 60% in use: 7 us for the scan, 77 for 516 MB of copies, 6.7 TB/s; the last pages of 256
// samples: 10 us for the counts and free pages, 11 for 77 MB.)  Taking pages is one thread's
// chain of loads and stores for each sequence: a page for some of 1000 sequences 10 us, 2048 pages
// for one 94 us.  A fork's counts read all children for each child and each parent.
#include "ds41_dense.cuh"

namespace ds41 {
namespace pages {

constexpr int SCAN = 1024;      // threads of the one CTA that scans
constexpr int STEP = 8;         // pages a thread looks at in a round
constexpr int COPY = 256;       // threads of a copying CTA

__device__ __forceinline__ int sequence_len(const int32_t* lens, int64_t b, int64_t cap,
                                            unsigned int* status, bool report) {
    const int len = lens[b];
    if (len >= 0 && len <= cap) return len;
    if (report) raise_status(status, DS41_E_INDEX);
    return 0;
}

// Exclusive prefix of v over the CTA's threads, and the sum.  sh: 33 int64.
__device__ __forceinline__ int64_t block_prefix(int64_t v, int64_t* sh, int64_t& sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t w = sh[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += y;
        }
        sh[lane] = w;
    }
    __syncthreads();
    sum = sh[31];
    const int64_t before = (warp ? sh[warp - 1] : 0) + x - v;
    __syncthreads();
    return before;
}

// One round of a walk over the pages in order: thread t looks at the pages p0 + k * SCAN +
// t; `yes` has a bit for each k whose page counts.  rank[k]: how many count before it in
// the round; returns how many count in all.  sh: STEP * 32 + 1 int.
__device__ __forceinline__ int round_ranks(uint32_t yes, int (&rank)[STEP], int* sh) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t m[STEP];
#pragma unroll
    for (int k = 0; k < STEP; k++) {
        m[k] = __ballot_sync(0xffffffffu, (yes >> k) & 1);
        if (lane == 0) sh[k * 32 + warp] = __popc(m[k]);
    }
    __syncthreads();
    if (warp == 0) {  // exclusive prefixes of the 256 counts, 8 a lane
        int c[STEP], sum = 0;
#pragma unroll
        for (int i = 0; i < STEP; i++) {
            c[i] = sum;
            sum += sh[lane * STEP + i];
        }
        int x = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, off);
            if (lane >= off) x += y;
        }
#pragma unroll
        for (int i = 0; i < STEP; i++) sh[lane * STEP + i] = x - sum + c[i];
        if (lane == 31) sh[STEP * 32] = x;
    }
    __syncthreads();
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int k = 0; k < STEP; k++) rank[k] = sh[k * 32 + warp] + __popc(m[k] & below);
    const int sum = sh[STEP * 32];
    __syncthreads();
    return sum;
}

// The first `want` free pages, in order, into list, their refs to 1; how many there were.
__device__ __forceinline__ int64_t take_free(int32_t* refs, int64_t n_pages, int64_t want,
                                             int32_t* list, int* sh) {
    int64_t found = 0;
    for (int64_t p0 = 0; p0 < n_pages && found < want; p0 += SCAN * STEP) {
        int32_t r[STEP];
        uint32_t yes = 0;
#pragma unroll
        for (int k = 0; k < STEP; k++) {
            const int64_t p = p0 + k * SCAN + threadIdx.x;
            r[k] = p < n_pages ? refs[p] : 1;
        }
#pragma unroll
        for (int k = 0; k < STEP; k++) yes |= (r[k] == 0 ? 1u : 0u) << k;
        int rank[STEP];
        const int sum = round_ranks(yes, rank, sh);
#pragma unroll
        for (int k = 0; k < STEP; k++)
            if (((yes >> k) & 1) && found + rank[k] < want) {
                const int64_t p = p0 + k * SCAN + threadIdx.x;
                list[found + rank[k]] = (int32_t)p;
                refs[p] = 1;
            }
        found += sum;
    }
    __syncthreads();  // the list is there for the whole CTA
    return found < want ? found : want;
}

struct TakeArgs {
    int32_t* refs;
    int32_t* table;
    const int32_t* lens;
    const int32_t* new_lens;
    int32_t* list;
    int64_t n_pages, max_pages, B;
    int page_shift;
    unsigned int* status;
};

__global__ void __launch_bounds__(SCAN) take_kernel(const TakeArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ int64_t sh64[33];
    __shared__ int sh[STEP * 32 + 1];
    const int up = (1 << a.page_shift) - 1;
    auto need = [&](int64_t b, int& first, bool report) {
        const int64_t cap = a.max_pages << a.page_shift;
        const int len = a.lens[b], to = a.new_lens[b];
        if (len < 0 || len > cap || to > cap) {
            if (report) raise_status(a.status, DS41_E_INDEX);
            return 0;
        }
        first = (int)(((int64_t)len + up) >> a.page_shift);
        return to <= len ? 0 : (int)(((int64_t)to + up) >> a.page_shift) - first;
    };
    int64_t want = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += SCAN) {
        int first;
        const int64_t b = b0 + threadIdx.x;
        int64_t sum;
        block_prefix(b < a.B ? need(b, first, true) : 0, sh64, sum);
        want += sum;
    }
    const int64_t found = take_free(a.refs, a.n_pages, want, a.list, sh);
    int64_t at = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += SCAN) {
        int first = 0;
        const int64_t b = b0 + threadIdx.x;
        int64_t sum;
        const int n = b < a.B ? need(b, first, false) : 0;
        const int64_t r0 = at + block_prefix(n, sh64, sum);
        for (int i = 0; i < n; i++) {
            const bool ok = r0 + i < found;
            a.table[b * a.max_pages + first + i] = ok ? a.list[r0 + i] : -1;
            if (!ok) raise_status(a.status, DS41_E_PAGES);
        }
        at += sum;
    }
}

struct FreeArgs {
    int32_t* refs;
    const int32_t* table;
    const int32_t* lens;
    int64_t n_pages, max_pages;
    int page_shift;
    unsigned int* status;
};

// a CTA for a sequence
__global__ void __launch_bounds__(128) free_kernel(const FreeArgs a) {
    pdl_wait();
    pdl_trigger();
    const int64_t b = blockIdx.x, cap = a.max_pages << a.page_shift;
    const int len = sequence_len(a.lens, b, cap, a.status, threadIdx.x == 0);
    const int used = (int)(((int64_t)len + (1 << a.page_shift) - 1) >> a.page_shift);
    for (int x = threadIdx.x; x < used; x += 128) {
        const int pg = a.table[b * a.max_pages + x];
        if (pg < 0 || pg >= a.n_pages) {
            raise_status(a.status, DS41_E_INDEX);
        } else if (atomicSub(&a.refs[pg], 1) <= 0) {
            atomicAdd(&a.refs[pg], 1);
            raise_status(a.status, DS41_E_INDEX);
        }
    }
}

struct ForkArgs {
    int32_t* refs;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* parents;
    int32_t* out;
    int32_t* out_lens;
    int64_t n_pages, max_pages;
    int B, n, page_shift, replace;
    int32_t* src;   // [n] scratch: a needy child's page to copy (-1: the child needs none), then
    int32_t* dst;   // [n] the copies in order
    int32_t* rows;  // [n]
    int32_t* list;  // [n]: free pages
    unsigned int* status;
};

// Row r of the work: r < n: a child's row of the table; n .. n + B - 1: a parent's references.  By
// WIDTH threads, a warp or a CTA, of which this is number tid.
template <int WIDTH>
__device__ __forceinline__ void fork_row(const ForkArgs& a, int r, int tid) {
    const int64_t cap = a.max_pages << a.page_shift;
    const int mask = (1 << a.page_shift) - 1;
    if (r < a.n) {
        const int i = r, p = a.parents[i];
        int len = 0;
        if (p >= 0 && p < a.B) len = sequence_len(a.lens, p, cap, a.status, false);
        else if (p != -1 && tid == 0) raise_status(a.status, DS41_E_INDEX);
        const int whole = len >> a.page_shift, part = len & mask;
        bool elder = false;  // an earlier child takes the last page over
        if (a.replace && part)
            for (int j = tid; j < i && !elder; j += WIDTH) elder = a.parents[j] == p;
        const bool some = WIDTH == 32 ? __any_sync(0xffffffffu, elder) : __syncthreads_or(elder);
        const bool heir = !some && a.replace;
        for (int64_t x = tid; x < a.max_pages; x += WIDTH) {
            int pg = -1;
            if (x < whole || (x == whole && part)) {
                pg = a.table[(int64_t)p * a.max_pages + x];
                if (pg < 0 || pg >= a.n_pages) {
                    raise_status(a.status, DS41_E_INDEX);
                    pg = -1;
                }
            }
            if (x == whole && part && !heir) {
                a.src[i] = pg;  // to be copied
                a.rows[i] = part;
                pg = -1;
            }
            a.out[(int64_t)i * a.max_pages + x] = pg;
        }
        if (tid == 0) {
            a.out_lens[i] = len;
            if (!part || heir) a.src[i] = -1;
        }
        return;
    }
    const int b = r - a.n;
    const int len = sequence_len(a.lens, b, cap, a.status, tid == 0);
    int born = 0;
    for (int j = tid; j < a.n; j += WIDTH) born += a.parents[j] == b;
    born = __reduce_add_sync(0xffffffffu, born);
    if (WIDTH > 32) {
        __shared__ int sums[WIDTH / 32];
        if ((tid & 31) == 0) sums[tid >> 5] = born;
        __syncthreads();
        born = 0;
#pragma unroll
        for (int w = 0; w < WIDTH / 32; w++) born += sums[w];
    }
    const int whole = len >> a.page_shift, part = len & mask;
    for (int x = tid; x < whole + (part ? 1 : 0); x += WIDTH) {
        const int change = x < whole ? born - a.replace : (a.replace && !born ? -1 : 0);
        const int pg = a.table[(int64_t)b * a.max_pages + x];
        if (pg < 0 || pg >= a.n_pages) {
            raise_status(a.status, DS41_E_INDEX);
        } else if (change && atomicAdd(&a.refs[pg], change) + change < 0) {
            atomicMax(&a.refs[pg], 0);
            raise_status(a.status, DS41_E_INDEX);
        }
    }
}

// The pages for the copies, in the children's order, by a CTA of SCAN threads.
__device__ __forceinline__ void fork_pages(const ForkArgs& a) {
    __shared__ int64_t sh64[33];
    __shared__ int sh[STEP * 32 + 1];
    int64_t want = 0;
    for (int i0 = 0; i0 < a.n; i0 += SCAN) {
        const int i = i0 + threadIdx.x;
        want += __syncthreads_count(i < a.n && a.src[i] >= 0);
    }
    const int64_t found = take_free(a.refs, a.n_pages, want, a.list, sh);
    int64_t at = 0;
    for (int i0 = 0; i0 < a.n; i0 += SCAN) {
        const int i = i0 + threadIdx.x;
        const int src = i < a.n ? a.src[i] : -1;
        int64_t sum;
        const int64_t r = at + block_prefix(src >= 0 ? 1 : 0, sh64, sum);
        if (i < a.n) {
            const int pg = src >= 0 && r < found ? a.list[r] : -1;
            a.dst[i] = pg;
            if (src >= 0) {
                a.out[(int64_t)i * a.max_pages + (a.out_lens[i] >> a.page_shift)] = pg;
                if (pg < 0) raise_status(a.status, DS41_E_PAGES);
            }
        }
        at += sum;
    }
}

// a CTA for a row
__global__ void __launch_bounds__(128) fork_kernel(const ForkArgs a) {
    pdl_wait();
    pdl_trigger();
    fork_row<128>(a, blockIdx.x, threadIdx.x);
}
__global__ void __launch_bounds__(SCAN) fork_pages_kernel(const ForkArgs a) {
    pdl_wait();
    pdl_trigger();
    fork_pages(a);
}
// Both in one launch, a cluster with a warp for a row, where the tables are small: 64 beams of 33
// entries 17.1 -> 15.4 us, 64 of 128 14.9 -> 14.4; 256 samples of 257 entries 20.7, this way 25.6.
constexpr int FORK_CTAS = 8, FORK_ROWS = 256, FORK_ENTRIES = 8192;
__global__ void __launch_bounds__(SCAN) fork_few_kernel(const ForkArgs a) {
    pdl_wait();
    pdl_trigger();
    for (int r = blockIdx.x * (SCAN / 32) + (threadIdx.x >> 5); r < a.n + a.B;
         r += FORK_CTAS * (SCAN / 32))
        fork_row<32>(a, r, threadIdx.x & 31);
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                     : "memory");
    if (blockIdx.x == 0) fork_pages(a);
}

struct CompactArgs {
    int32_t* refs;
    int64_t n_pages;
    int32_t* live;
    int32_t* to;     // [n_pages] scratch: where a page goes
    int32_t* src;    // [n_pages] and the pages that move,
    int32_t* dst;    // [n_pages]
    int32_t* count;  // how many
};

__global__ void __launch_bounds__(SCAN) compact_kernel(const CompactArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ int64_t sh64[33];
    __shared__ int sh[STEP * 32 + 1];
    int64_t mine = 0, live;
    for (int64_t p0 = 0; p0 < a.n_pages; p0 += SCAN * STEP)
#pragma unroll
        for (int k = 0; k < STEP; k++) {
            const int64_t p = p0 + k * SCAN + threadIdx.x;
            mine += p < a.n_pages && a.refs[p] != 0;
        }
    block_prefix(mine, sh64, live);
    int64_t holes = 0, movers = 0;
    for (int64_t p0 = 0; p0 < a.n_pages; p0 += SCAN * STEP) {
        uint32_t hole = 0, moves = 0;
#pragma unroll
        for (int k = 0; k < STEP; k++) {
            const int64_t p = p0 + k * SCAN + threadIdx.x;
            if (p >= a.n_pages) continue;
            const bool used = a.refs[p] != 0;
            hole |= (!used && p < live ? 1u : 0u) << k;
            moves |= (used && p >= live ? 1u : 0u) << k;
            a.to[p] = (int32_t)p;
        }
        int rank[STEP];
        int sum = round_ranks(hole, rank, sh);
#pragma unroll
        for (int k = 0; k < STEP; k++)
            if ((hole >> k) & 1) a.dst[holes + rank[k]] = (int32_t)(p0 + k * SCAN + threadIdx.x);
        holes += sum;
        sum = round_ranks(moves, rank, sh);
#pragma unroll
        for (int k = 0; k < STEP; k++)
            if ((moves >> k) & 1) a.src[movers + rank[k]] = (int32_t)(p0 + k * SCAN + threadIdx.x);
        movers += sum;
    }
    __syncthreads();
    for (int64_t i = threadIdx.x; i < movers; i += SCAN) {
        const int s = a.src[i], d = a.dst[i];
        a.to[s] = d;
        a.refs[d] = a.refs[s];
        a.refs[s] = 0;
    }
    if (threadIdx.x == 0) {
        a.live[0] = (int32_t)live;
        a.count[0] = (int32_t)movers;
    }
}

struct CopyArgs {
    uint8_t* x[2];     // k, v
    float* scales[2];  // null for bf16
    int8_t* codes;     // null: no block keys
    float* key_scales;
    const int32_t* src;
    const int32_t* dst;
    const int32_t* rows;   // null: whole pages
    const int32_t* count;  // null: n
    int64_t n, n_pages;
    int kvh, page, row_bytes, hd;
    // the table whose entries follow (compacting)
    int32_t* table;
    const int32_t* lens;
    const int32_t* to;
    int64_t max_pages;
    int B, page_shift;
    unsigned int* status;
};

// A CTA moves one head of one page: a contiguous run of K and one of V.
__global__ void __launch_bounds__(COPY) copy_kernel(const CopyArgs a) {
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    if (a.to)
        for (int64_t b = blockIdx.x; b < a.B; b += gridDim.x) {
            const int len = sequence_len(a.lens, b, a.max_pages << a.page_shift, a.status, tid == 0);
            const int used = (int)(((int64_t)len + a.page - 1) >> a.page_shift);
            // (all entries, not the counted ones alone: behind those may be pages that were taken
            // for rows to come, which have moved like the rest)
            for (int64_t i = tid; i < a.max_pages; i += COPY) {
                int32_t* e = a.table + b * a.max_pages + i;
                const int pg = *e;
                if (pg >= 0 && pg < a.n_pages) *e = a.to[pg];
                else if (i < used) raise_status(a.status, DS41_E_INDEX);
            }
        }
    const int64_t units = (a.count ? (int64_t)*a.count : a.n) * a.kvh;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t i = u / a.kvh;
        const int h = (int)(u - i * a.kvh);
        const int s = a.src[i], d = a.dst[i];
        if (s < -1 || s >= a.n_pages || d < -1 || d >= a.n_pages) {
            if (tid == 0) raise_status(a.status, DS41_E_INDEX);
            continue;
        }
        if (s < 0 || d < 0) continue;
        const int rows = a.rows ? a.rows[i] : a.page;
        if (rows < 0 || rows > a.page) {
            if (tid == 0) raise_status(a.status, DS41_E_INDEX);
            continue;
        }
        const int64_t sr = ((int64_t)s * a.kvh + h) * a.page, dr = ((int64_t)d * a.kvh + h) * a.page;
        const int nv = rows * a.row_bytes / 16;  // 16-byte pieces of each run
        const uint4* from[2];
        uint4* into[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            from[t] = reinterpret_cast<const uint4*>(a.x[t] + sr * a.row_bytes);
            into[t] = reinterpret_cast<uint4*>(a.x[t] + dr * a.row_bytes);
        }
        for (int v0 = tid; v0 < nv; v0 += 4 * COPY) {
            uint4 r[2][4];
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int k = 0; k < 4; k++)
                    if (v0 + k * COPY < nv) r[t][k] = __ldcs(from[t] + v0 + k * COPY);
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int k = 0; k < 4; k++)
                    if (v0 + k * COPY < nv) __stcs(into[t] + v0 + k * COPY, r[t][k]);
        }
        if (a.scales[0] && tid < rows) {  // a page has at most 256 rows
            a.scales[0][dr + tid] = a.scales[0][sr + tid];
            a.scales[1][dr + tid] = a.scales[1][sr + tid];
        }
        if (a.codes && tid < a.hd / 4) {
            const int64_t sk = (int64_t)s * a.kvh + h, dk = (int64_t)d * a.kvh + h;
            reinterpret_cast<uint32_t*>(a.codes + dk * a.hd)[tid] =
                reinterpret_cast<const uint32_t*>(a.codes + sk * a.hd)[tid];
            if (tid == 0) a.key_scales[dk] = a.key_scales[sk];
        }
    }
}
static_assert(COPY >= 256, "a thread for each scale of a page");

struct Pool {
    int64_t n_pages, page, max_pages, B;
    int shift;
};
int check_pool(const char* name, int64_t n_pages, int64_t page, int64_t max_pages, int64_t B,
               Pool* out) {
    const int64_t lim = int64_t(1) << 31;
    DS41_REQUIRE(page >= 16 && page <= 256 && (page & (page - 1)) == 0, DS41_E_ARG,
                 "%s: page=%lld must be a power of two of 16 .. 256", name, (long long)page);
    DS41_REQUIRE(n_pages >= 1 && n_pages < lim, DS41_E_ARG, "%s: n_pages=%lld", name,
                 (long long)n_pages);
    DS41_REQUIRE(max_pages >= 0 && max_pages < lim && B >= 0 && B < lim / 2, DS41_E_RANGE,
                 "%s: max_pages=%lld B=%lld", name, (long long)max_pages, (long long)B);
    *out = {n_pages, page, max_pages, B, 0};
    while ((1 << out->shift) < page) out->shift++;
    return DS41_OK;
}
bool words(const void* p) { return p && aligned_to(p, 4); }

// What is copied, checked.
int check_copy(const char* name, void* k, void* v, float* ks, float* vs, int fmt, int64_t n_pages,
               int64_t page, int64_t kvh, int64_t hd, int8_t* codes, float* key_scales,
               CopyArgs* out) {
    PagedKv kv;
    if (int rc = check_paged(name, k, v, ks, vs, fmt, n_pages, page, kvh, hd, &kv)) return rc;
    DS41_REQUIRE((codes == nullptr) == (key_scales == nullptr) && aligned16(codes) &&
                     aligned_to(key_scales, 4),
                 DS41_E_ARG, "%s: codes (16-byte aligned) and key_scales are both given or both NULL",
                 name);
    *out = CopyArgs{};
    out->x[0] = static_cast<uint8_t*>(k);
    out->x[1] = static_cast<uint8_t*>(v);
    if (fmt == DS41_KV_E4M3) {
        out->scales[0] = ks;
        out->scales[1] = vs;
    }
    out->codes = codes;
    out->key_scales = key_scales;
    out->n_pages = n_pages;
    out->kvh = (int)kvh;
    out->page = (int)page;
    out->page_shift = kv.page_shift;
    out->row_bytes = (int)hd * (fmt == DS41_KV_E4M3 ? 1 : 2);
    out->hd = (int)hd;
    return DS41_OK;
}
// As many CTAs as there can be work, at most eight an SM.
int launch_copy(const CopyArgs& c, int64_t most, cudaStream_t st, const char* name) {
    const int64_t want = most * c.kvh, full = (int64_t)sm_count_once() * 8;
    return launch_pdl(copy_kernel, dim3((unsigned)(want < 1 ? 1 : want < full ? want : full)),
                      dim3(COPY), 0, st, name, c);
}
size_t up16(size_t x) { return (x + 15) & ~size_t(15); }

}  // namespace pages
}  // namespace ds41

using namespace ds41;
using namespace ds41::pages;

extern "C" int ds41_kv_pages_take(int32_t* refs, int64_t n_pages, int64_t page,
                                  int32_t* page_table, int64_t max_pages, const int32_t* lens,
                                  const int32_t* new_lens, int64_t B, void* ws, size_t ws_bytes,
                                  ds41_stream_t stream) {
    const char* name = "ds41_kv_pages_take";
    Pool p;
    if (int rc = check_pool(name, n_pages, page, max_pages, B, &p)) return rc;
    if (B == 0) return DS41_OK;
    DS41_REQUIRE(words(refs) && words(page_table) && words(lens) && words(new_lens), DS41_E_ARG,
                 "%s: refs, page_table, lens and new_lens must be non-null and aligned", name);
    DS41_REQUIRE(words(ws) && ws_bytes >= (size_t)n_pages * 4, DS41_E_WORKSPACE,
                 "%s: needs %zu bytes of workspace, got %zu", name, (size_t)n_pages * 4,
                 ws ? ws_bytes : 0);
    TakeArgs a{refs, page_table, lens, new_lens, static_cast<int32_t*>(ws), n_pages, max_pages, B,
               p.shift, nullptr};
    if (int rc = status_word(&a.status)) return rc;
    return launch_pdl(take_kernel, dim3(1), dim3(SCAN), 0, (cudaStream_t)stream, name, a);
}

extern "C" int ds41_kv_pages_free(int32_t* refs, int64_t n_pages, int64_t page,
                                  const int32_t* page_table, int64_t max_pages,
                                  const int32_t* lens, int64_t B, ds41_stream_t stream) {
    const char* name = "ds41_kv_pages_free";
    Pool p;
    if (int rc = check_pool(name, n_pages, page, max_pages, B, &p)) return rc;
    if (B == 0) return DS41_OK;
    DS41_REQUIRE(words(refs) && words(page_table) && words(lens), DS41_E_ARG,
                 "%s: refs, page_table and lens must be non-null and aligned", name);
    FreeArgs a{refs, page_table, lens, n_pages, max_pages, p.shift, nullptr};
    if (int rc = status_word(&a.status)) return rc;
    return launch_pdl(free_kernel, dim3((unsigned)B), dim3(128), 0, (cudaStream_t)stream, name, a);
}

extern "C" size_t ds41_kv_pages_fork_workspace_bytes(int64_t n_pages, int64_t B, int64_t n) {
    if (n_pages < 1 || B < 0 || n < 0) return 0;
    return 4 * up16((size_t)n * 4);
}

extern "C" int ds41_kv_pages_fork(void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                                  int fmt, int64_t n_pages, int64_t page, int64_t kvh, int64_t hd,
                                  int8_t* codes, float* key_scales, int32_t* refs,
                                  const int32_t* page_table, int64_t max_pages,
                                  const int32_t* lens, int64_t B, const int32_t* parents,
                                  int64_t n, int replace, int32_t* table_out, int32_t* lens_out,
                                  void* ws, size_t ws_bytes, ds41_stream_t stream) {
    const char* name = "ds41_kv_pages_fork";
    CopyArgs c;
    if (int rc = check_copy(name, k_cache, v_cache, k_scales, v_scales, fmt, n_pages, page, kvh, hd,
                            codes, key_scales, &c))
        return rc;
    Pool p;
    if (int rc = check_pool(name, n_pages, page, max_pages, B, &p)) return rc;
    // (each child and each parent counts among all children: (n + B) n reads)
    DS41_REQUIRE(n >= 0 && n < 65536 && B < 65536, DS41_E_RANGE, "%s: n=%lld B=%lld (below 65536)",
                 name, (long long)n, (long long)B);
    if (n + (replace ? B : 0) == 0) return DS41_OK;
    DS41_REQUIRE(words(refs) && (B == 0 || (words(page_table) && words(lens))) &&
                     (n == 0 || (words(parents) && words(table_out) && words(lens_out))),
                 DS41_E_ARG,
                 "%s: refs, page_table, lens, parents, table_out and lens_out must be non-null and "
                 "aligned", name);
    DS41_REQUIRE(n == 0 || B == 0 ||
                     ((page_table + B * max_pages <= table_out ||
                       table_out + n * max_pages <= page_table) &&
                      (lens + B <= lens_out || lens_out + n <= lens)),
                 DS41_E_ARG, "%s: table_out lies in page_table, or lens_out in lens", name);
    const size_t one = up16((size_t)n * 4);
    DS41_REQUIRE(n == 0 || (ws && aligned16(ws) && ws_bytes >= 4 * one), DS41_E_WORKSPACE,
                 "%s: needs %zu bytes of workspace, got %zu", name, 4 * one, ws ? ws_bytes : 0);
    ForkArgs a{refs, page_table, lens, parents, table_out, lens_out, n_pages, max_pages, (int)B,
               (int)n, p.shift, replace ? 1 : 0, nullptr, nullptr, nullptr, nullptr, nullptr};
    int32_t** parts[4] = {&a.src, &a.dst, &a.rows, &a.list};
    for (int i = 0; i < 4; i++)
        *parts[i] = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + i * one);
    if (int rc = status_word(&a.status)) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    if (n > 0 && n + B <= FORK_ROWS && (n + B) * max_pages <= FORK_ENTRIES) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(FORK_CTAS);
        cfg.blockDim = dim3(SCAN);
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = FORK_CTAS;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        if (int rc = cuda_check(cudaLaunchKernelEx(&cfg, fork_few_kernel, a), name)) return rc;
        if (int rc = launch_check(name)) return rc;
    } else {
        if (int rc = launch_pdl(fork_kernel, dim3((unsigned)(n + B)), dim3(128), 0, st, name, a))
            return rc;
        if (n == 0) return DS41_OK;
        if (int rc = launch_pdl(fork_pages_kernel, dim3(1), dim3(SCAN), 0, st, name, a)) return rc;
    }
    c.src = a.src;
    c.dst = a.dst;
    c.rows = a.rows;
    c.n = n;
    c.status = a.status;
    return launch_copy(c, n, st, name);
}

extern "C" int ds41_kv_pages_copy(void* k_cache, void* v_cache, float* k_scales, float* v_scales,
                                  int fmt, int64_t n_pages, int64_t page, int64_t kvh, int64_t hd,
                                  int8_t* codes, float* key_scales, const int32_t* src,
                                  const int32_t* dst, const int32_t* rows, int64_t n,
                                  ds41_stream_t stream) {
    const char* name = "ds41_kv_pages_copy";
    CopyArgs c;
    if (int rc = check_copy(name, k_cache, v_cache, k_scales, v_scales, fmt, n_pages, page, kvh, hd,
                            codes, key_scales, &c))
        return rc;
    DS41_REQUIRE(n >= 0 && n < int64_t(1) << 31, DS41_E_RANGE, "%s: n=%lld", name, (long long)n);
    if (n == 0) return DS41_OK;
    DS41_REQUIRE(words(src) && words(dst) && aligned_to(rows, 4), DS41_E_ARG,
                 "%s: src and dst must be non-null and aligned", name);
    c.src = src;
    c.dst = dst;
    c.rows = rows;
    c.n = n;
    if (int rc = status_word(&c.status)) return rc;
    return launch_copy(c, n, (cudaStream_t)stream, name);
}

extern "C" size_t ds41_kv_pages_compact_workspace_bytes(int64_t n_pages) {
    return n_pages < 1 ? 0 : 3 * up16((size_t)n_pages * 4) + 16;
}

extern "C" int ds41_kv_pages_compact(void* k_cache, void* v_cache, float* k_scales,
                                     float* v_scales, int fmt, int64_t n_pages, int64_t page,
                                     int64_t kvh, int64_t hd, int8_t* codes, float* key_scales,
                                     int32_t* refs, int32_t* page_table, int64_t max_pages,
                                     const int32_t* lens, int64_t B, int32_t* live, void* ws,
                                     size_t ws_bytes, ds41_stream_t stream) {
    const char* name = "ds41_kv_pages_compact";
    CopyArgs c;
    if (int rc = check_copy(name, k_cache, v_cache, k_scales, v_scales, fmt, n_pages, page, kvh, hd,
                            codes, key_scales, &c))
        return rc;
    Pool p;
    if (int rc = check_pool(name, n_pages, page, max_pages, B, &p)) return rc;
    DS41_REQUIRE(words(refs) && words(live) && (B == 0 || (words(page_table) && words(lens))),
                 DS41_E_ARG, "%s: refs, page_table, lens and live must be non-null and aligned",
                 name);
    const size_t need = ds41_kv_pages_compact_workspace_bytes(n_pages);
    DS41_REQUIRE(ws && aligned16(ws) && ws_bytes >= need, DS41_E_WORKSPACE,
                 "%s: needs %zu bytes of workspace, got %zu", name, need, ws ? ws_bytes : 0);
    const size_t one = up16((size_t)n_pages * 4);
    uint8_t* w = static_cast<uint8_t*>(ws);
    CompactArgs a{refs, n_pages, live, reinterpret_cast<int32_t*>(w),
                  reinterpret_cast<int32_t*>(w + one), reinterpret_cast<int32_t*>(w + 2 * one),
                  reinterpret_cast<int32_t*>(w + 3 * one)};
    if (int rc = status_word(&c.status)) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    if (int rc = launch_pdl(compact_kernel, dim3(1), dim3(SCAN), 0, st, name, a)) return rc;
    c.src = a.src;
    c.dst = a.dst;
    c.count = a.count;
    c.table = page_table;
    c.lens = lens;
    c.to = a.to;
    c.max_pages = max_pages;
    c.B = (int)B;
    // (no more than half of the pages move)
    return launch_copy(c, n_pages / 2 > B ? n_pages / 2 : (B > 0 ? B : 1), st, name);
}
