// ds41_blocks.cu - one key for each block (page) of the paged cache, and the blocks that
// a cheap score against those keys picks for each query.
//
// Mathematics.  A block's key is the mean of its rows, summed in f32 in their order, as int8
// codes with one scale: s = max(amax, 127 2^-126) f32(1/127), c = rint(m / s).  A
// query row is rounded alike.  The product of the codes is a whole number below 127^2 128 <
// 2^21, which f16 operands (exact up to 2048) and f32 sums give exactly in any order; the
// score is two f32 products away, so the picks are the same wherever they are worked out.
// The scale of a block is not negative, so it may follow the maximum over the heads.
//
// What bounds it.  The keys' sums read the new rows' pages once, by latencies: a warp has one
// page and head, 16 rows of it in flight behind the table's entry (8 heads of 128, bf16, pages
// of 64: 8192 rows 8.6 us, 2.0 TB/s; 32768 rows 16.8 us, 4.0 TB/s).  Selection for a step of few
// tokens: a chain of latencies (the page table, the keys, the scores' exchange, the ranking).  For
// prompts: instructions, a third of them around the products (m16n8k16, blocks by columns of
// query heads), 40% in the ranking.  (One token of 24 sequences, up to 512 blocks, 32 heads of 128
// over 8: 12 us; 8192 tokens, up to 512 blocks: 221 us.  64 picks of 2048 blocks against 512: 24
// tokens 35 us against 16, 2048 tokens 258 against 74: from 43 picks on no sample gives a bound,
// and all ranks are counted several times.)
#include "ds41_softmax_tc.cuh"

namespace ds41 {
namespace blocks {

constexpr float STEP = 1.0f / 127.0f;
constexpr float FLOOR = 127.0f * 0x1p-126f;

// The int8 form of a row, from the bits of its largest magnitude (they are ordered as the
// magnitudes are, infinities and NaN above all: the scale is NaN then, the codes 0).
struct Int8 {
    float scale;
    float f, d, r;  // quotients by the scale: see code()
    __device__ __forceinline__ explicit Int8(uint32_t top) {
        const bool bad = top >= 0x7f800000u;
        const float s = __fmul_rn(fmaxf(__uint_as_float(top), FLOOR), STEP);
        // A scale below 2^-90 and its row are taken 2^100 times, one above 2^100 and its row
        // 2^-60 times: the remainders stay normal numbers.
        f = bad ? 0.0f : s < 0x1p-90f ? 0x1p100f : s > 0x1p100f ? 0x1p-60f : 1.0f;
        d = bad ? 1.0f : s * f;
        r = __frcp_rn(d);
        scale = bad ? __uint_as_float(0x7fc00000u) : s;
    }
    // rint(x / scale): the quotient correctly rounded, from the correctly rounded reciprocal
    // and the exact remainder of a fused multiply-add (P. Markstein, 1990).
    __device__ __forceinline__ float code(float x) const {
        const float y = f == 0.0f ? 0.0f : x * f, q = __fmul_rn(y, r);
        return rintf(__fmaf_rn(__fmaf_rn(q, -d, y), r, q));
    }
};

struct KeyArgs {
    PagedKv kv;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* starts;
    int64_t max_pages, max_new;
    int8_t* codes;
    float* scales;
    unsigned int* status;
};

constexpr int KEY_WARPS = 4;

// A warp for a page and head, four elements a lane, 16 rows (32 of codes) in flight.
template <bool E4M3>
__global__ void __launch_bounds__(KEY_WARPS * 32) keys_kernel(const KeyArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int h = blockIdx.x * KEY_WARPS + (threadIdx.x >> 5);
    const int64_t b = blockIdx.z;
    const int len = a.lens[b], start = a.starts ? a.starts[b] : 0;
    if (len < 0 || start < 0 || start > len || len - start > a.max_new ||
        len > a.max_pages * a.kv.page) {
        if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
            raise_status(a.status, DS41_E_INDEX);
        return;
    }
    if (h >= a.kv.kvh) return;
    for (int64_t i = (start >> a.kv.page_shift) + (int64_t)blockIdx.y;
         (i << a.kv.page_shift) < len && start < len; i += gridDim.y) {
        const int64_t pg = a.table[b * a.max_pages + i];
        if (pg < 0 || pg >= a.kv.n_pages) {
            if (lane == 0) raise_status(a.status, DS41_E_INDEX);
            continue;
        }
        const int n = (int)min((int64_t)a.kv.page, len - (i << a.kv.page_shift));
        const bool mine = lane * 4 < a.kv.hd;
        const int64_t row = paged_row(a.kv, pg, h, 0);
        const uint8_t* p = a.kv.k + (row * a.kv.hd + (mine ? lane * 4 : 0)) * (E4M3 ? 1 : 2);
        const int step = a.kv.hd * (E4M3 ? 1 : 2);
        float sum[4] = {0, 0, 0, 0};
        constexpr int U = E4M3 ? 32 : 16;
        for (int r0 = 0; r0 < n; r0 += U) {
            uint2 w[U];
            // (rows behind the last are that one once more: no load waits for a branch)
#pragma unroll
            for (int u = 0; u < U; u++) {
                const uint8_t* at = p + min(r0 + u, n - 1) * step;
                if (E4M3) w[u].x = __ldcs(reinterpret_cast<const uint32_t*>(at));
                else w[u] = __ldcs(reinterpret_cast<const uint2*>(at));
            }
            const float scale = E4M3 ? a.kv.ks[row + min(r0 + lane, n - 1)] : 0.0f;
#pragma unroll
            for (int u = 0; u < U; u++) {
                float x[4];
                if (E4M3) {
                    const float s = __shfl_sync(0xffffffffu, scale, u);
                    uint32_t lo, hi;
                    e4m3x4_to_f16(w[u].x, lo, hi);
                    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&lo));
                    const float2 g = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                    x[0] = __fmul_rn(f.x, s);
                    x[1] = __fmul_rn(f.y, s);
                    x[2] = __fmul_rn(g.x, s);
                    x[3] = __fmul_rn(g.y, s);
                } else {
                    x[0] = __uint_as_float(w[u].x << 16);
                    x[1] = __uint_as_float(w[u].x & 0xffff0000u);
                    x[2] = __uint_as_float(w[u].y << 16);
                    x[3] = __uint_as_float(w[u].y & 0xffff0000u);
                }
                if (r0 + u < n)
#pragma unroll
                    for (int e = 0; e < 4; e++) sum[e] = __fadd_rn(sum[e], x[e]);
            }
        }
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 4; e++) {
            sum[e] = mine ? __fdiv_rn(sum[e], (float)n) : 0.0f;
            top = max(top, __float_as_uint(sum[e]) & 0x7fffffffu);
        }
        const Int8 key(__reduce_max_sync(0xffffffffu, top));
        if (mine) {
            uint32_t c = 0;
#pragma unroll
            for (int e = 0; e < 4; e++) c |= ((uint32_t)(int)key.code(sum[e]) & 0xffu) << (8 * e);
            *reinterpret_cast<uint32_t*>(a.codes + (pg * a.kv.kvh + h) * a.kv.hd + lane * 4) = c;
        }
        if (lane == 0) a.scales[pg * a.kv.kvh + h] = key.scale;
    }
}

struct SelectArgs {
    const uint16_t* q;
    int64_t q_tok, q_head;
    const int8_t* codes;
    const float* scales;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu_q;
    int32_t* idx;
    int64_t Tq, n_pages, max_pages;
    int page, page_shift, kvh, hd, G, max_q, max_len, topk, first, local;
    int TT;       // tokens of a CTA
    int NB;       // room for a token's scores: tokens next to each other in different banks
    int heads;    // query heads at a time, even
    int runs;     // CTAs that share the blocks of a few tokens: a cluster
    unsigned int* status;
};

template <bool FEW>
constexpr int SELECT_WARPS = FEW ? 8 : 16;  // of a CTA

// four int8 codes -> their values as f16, exactly: a code plus 128 in the low bits of 1024
__device__ __forceinline__ void int8x4_to_f16(uint32_t x, uint32_t& lo, uint32_t& hi) {
    x ^= 0x80808080u;
    const __half2 off = __half2half2(__ushort_as_half((uint16_t)0x6480));  // 1152
    uint32_t a = __byte_perm(x, 0x64646464u, 0x4140), b = __byte_perm(x, 0x64646464u, 0x4342);
    __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), off);
    lo = *reinterpret_cast<uint32_t*>(&r);
    r = __hsub2(*reinterpret_cast<__half2*>(&b), off);
    hi = *reinterpret_cast<uint32_t*>(&r);
}
// larger for larger scores; a score that is not a number counts as -inf
__device__ __forceinline__ uint32_t rank_of(float s) {
    if (!(s == s)) s = -INFINITY;
    const uint32_t u = __float_as_uint(s + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// the score of a rank that is neither 0 nor the largest
__device__ __forceinline__ float score_of(uint32_t rank) {
    return __uint_as_float((rank >> 31) ? rank ^ 0x80000000u : ~rank);
}

// Where the k-th largest of m ranks would be if their scores were normally distributed
// (mean and spread from every second register; the quantile by Hastings' approximation,
// Abramowitz and Stegun 26.2.22), and what a doubling of the count moves it by there.
template <int R>
__device__ __forceinline__ float normal(const uint32_t (&v)[R], int m, int k, int lane,
                                        float& slope) {
    float sum = 0.0f, squares = 0.0f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < R; i += 2) {
        const float x = 32 * i + lane < m ? score_of(v[i]) : 0.0f;
        sum += x;
        squares += x * x;
        n += max(0, min(32, m - 32 * i));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        squares += __shfl_xor_sync(0xffffffffu, squares, o);
    }
    const float mean = sum / n, spread = sqrtf(fmaxf(squares / n - mean * mean, 0.0f));
    const float t = sqrtf(-2.0f * tc::SM_LN2 * tc::lg2(fminf((float)k / (float)m, 0.5f)));
    const float z = t - (2.30753f + 0.27061f * t) / (1.0f + t * (0.99229f + 0.04481f * t));
    slope = spread / z * tc::SM_LN2 * 1.3f;
    return mean + spread * z;
}

// Where the k-th largest of m > k ranks lies (a warp, 32 R of them in registers, 0 behind the
// last): more than k ranks are lo or above, `above` <= k are hi or above.  Looked for between
// the smallest and the largest: where it would be among normally distributed scores, then by
// halving what is left, as scores (about five counts of all ranks in all, where bit by bit
// it is 30; a guess that is wrong, or no number, costs a count), and as integers if that
// has not ended it.  It ends with above == k, with nothing between lo and hi, or, with
// slack, once at most k + slack are lo or above.
struct Cut {
    uint32_t lo, hi;
    int above;
};
template <int R>
__device__ __forceinline__ Cut cut(const uint32_t (&v)[R], int m, int k, int slack, int lane) {
    Cut c{0xffffffffu, 0, 0};
#pragma unroll
    for (int i = 0; i < R; i++) {
        c.lo = min(c.lo, 32 * i + lane < m ? v[i] : 0xffffffffu);
        c.hi = max(c.hi, v[i]);
    }
    c.lo = __reduce_min_sync(0xffffffffu, c.lo);
    c.hi = __reduce_max_sync(0xffffffffu, c.hi) + 1;
    int n = m, n_lo = m;
    float slope = 0.0f, at = 0.0f;
    for (int i = 0; c.above < k && (slack == 0 || n_lo > k + slack) && c.hi - c.lo > 1; i++) {
        uint32_t mid = c.lo + (c.hi - c.lo) / 2;
        if (i < 16) {
            if (i == 0) at = normal<R>(v, m, k, lane, slope);
            else if (i == 1) at += slope * tc::lg2((float)n / (float)k);
            else at = 0.5f * score_of(c.lo) + 0.5f * score_of(c.hi);
            const uint32_t x = rank_of(at);
            if (x > c.lo && x < c.hi) mid = x;
        }
        n = 0;
#pragma unroll
        for (int i = 0; i < R; i++) n += v[i] >= mid;
        n = __reduce_add_sync(0xffffffffu, n);
        if (n > k) {
            c.lo = mid;
            n_lo = n;
        } else {
            c.hi = mid;
            c.above = n;
        }
    }
    return c;
}
// What a cut leaves, written in order: all from hi on, and the first of those equal to lo.
struct Writer {
    int32_t* out;
    int ties, to, lane;
    uint32_t lo, hi;
    __device__ __forceinline__ Writer(int32_t* out, const Cut& c, int k, int lane)
        : out(out), ties(k - c.above), to(0), lane(lane), lo(c.lo), hi(c.hi) {}
    // (a lane's rank x of block j; real: there is one)
    __device__ __forceinline__ void put(uint32_t x, int j, bool real) {
        const uint32_t below = (1u << lane) - 1u;
        bool take = x >= hi;
        if (ties > 0) {
            const uint32_t eq = __ballot_sync(0xffffffffu, x == lo && real);
            take |= x == lo && real && __popc(eq & below) < ties;
            ties -= min(ties, __popc(eq));
        }
        const uint32_t all = __ballot_sync(0xffffffffu, take);
        if (take) out[to + __popc(all & below)] = j;
        to += __popc(all);
    }
};

// The k of m > k ranks at s, at most 32 R of them, by a warp: ties to the first, ascending to
// out as j0 + place.
template <int R>
__device__ __forceinline__ void pick(const uint32_t* s, int m, int k, int32_t* out, int j0,
                                     int lane) {
    uint32_t v[R];
#pragma unroll
    for (int i = 0; i < R; i++) v[i] = 32 * i + lane < m ? s[32 * i + lane] : 0;
    Writer w(out, cut(v, m, k, 0, lane), k, lane);
#pragma unroll
    for (int i = 0; i < R; i++) w.put(v[i], j0 + 32 * i + lane, 32 * i + lane < m);
}

// The same of any number.  First those that may be among the k: from a sample of 128,
// evenly spread, follows a bound that at least k reach (the k-th largest of some is never
// above that of all) and about m / 100 k others; their places go to `list`, 16 bits each,
// and they alone are cut.  (Up to 512 ranks the registers of pick hold, and two cuts cost
// more than one: 448 ranks, 29 of them, 219 us for a chunk's selection, this way 240.)
constexpr int LIST = 256;
__device__ __forceinline__ void pick_of_many(const uint32_t* s, int m, int k, int32_t* out,
                                             int j0, uint16_t* list, int lane) {
    uint32_t v[LIST / 32];
    auto count = [&](uint32_t least) {
        int n = 0;
#pragma unroll 8
        for (int j = lane; j < m; j += 32) n += s[j] >= least;
        return __reduce_add_sync(0xffffffffu, n);
    };
    // a bound that at least k ranks reach
    uint32_t lo = 1, hi = 0;
    if (3 * k <= 128) {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; i++) x[i] = s[((32 * i + lane) * m) >> 7];
        const Cut c = cut(x, 128, k, k / 4 + 2, lane);
        lo = c.above == k ? c.hi : c.lo;
    }
    for (int j = lane; j < m; j += 32) hi = max(hi, s[j]);
    hi = __reduce_max_sync(0xffffffffu, hi) + 1;
    // raised until the list holds those that do; `above` < k are hi or above
    int n = count(lo), above = 0;
    for (int i = 0; n > LIST && hi - lo > 1; i++) {
        uint32_t mid = lo + (hi - lo) / 2;
        const uint32_t x = rank_of(0.5f * score_of(lo) + 0.5f * score_of(hi));
        if (i < 16 && x > lo && x < hi) mid = x;
        const int at_mid = count(mid);
        if (at_mid >= k) {
            lo = mid;
            n = at_mid;
        } else {
            hi = mid;
            above = at_mid;
        }
    }
    const uint32_t below = (1u << lane) - 1u;
    if (n > LIST) {  // (equal scores in masses)
        Writer w(out, Cut{lo, hi, above}, k, lane);
        for (int j = 0; j < m; j += 32)
            w.put(j + lane < m ? s[j + lane] : 0, j0 + j + lane, j + lane < m);
        return;
    }
    int to = 0;
#pragma unroll 4
    for (int j = 0; j < m; j += 32) {
        const bool keep = j + lane < m && s[j + lane] >= lo;
        const uint32_t all = __ballot_sync(0xffffffffu, keep);
        if (keep) list[to + __popc(all & below)] = (uint16_t)(j + lane);
        to += __popc(all);
    }
    __syncwarp();
    int place[LIST / 32];
#pragma unroll
    for (int i = 0; i < LIST / 32; i++) {
        place[i] = 32 * i + lane < n ? list[32 * i + lane] : 0;
        v[i] = 32 * i + lane < n ? s[place[i]] : 0;
    }
    const Cut c = n == k ? Cut{0, 1, k} : cut(v, n, k, 0, lane);
    Writer w(out, c, k, lane);
#pragma unroll
    for (int i = 0; i < LIST / 32; i++) w.put(v[i], j0 + place[i], 32 * i + lane < n);
    __syncwarp();  // (the list is the warp's next token's, too)
}

// Scores of TT tokens of a sequence for one key/value head, then the tokens' picks.
// Products: 16 blocks (rows, codes straight from global memory into the fragments) by 8
// columns; column 2 t + e of tile (quad, i) is token 4 quad + t, head 2 i + e, so that a lane
// has all heads of its token and their maximum takes no exchange.  hd in the order of tree
// attention's e4m3 fragments: lane c owns the codes 16 c .. and 64 + 16 c .. of a row.
// FEW: a few tokens, one CTA an SM or so: the next blocks' codes are under way while the products
// of these run (else 32 warps an SM hide that); where there are fewer CTAs than that, a
// cluster shares the blocks, and each token's scores go to the CTA that picks for it.
template <int HD, bool FEW>
__global__ void __launch_bounds__(SELECT_WARPS<FEW> * 32, 2) select_kernel(const SelectArgs a) {
    constexpr int SEL_WARPS = SELECT_WARPS<FEW>;
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) uint8_t smem[];
    constexpr int KS = HD / 16;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int b = blockIdx.y, h = blockIdx.z;
    const int q0 = a.cu_q[b];
    const int64_t n64 = (int64_t)a.cu_q[b + 1] - q0;
    const int len = a.lens[b];
    if (q0 < 0 || n64 < 0 || n64 > a.max_q || q0 + n64 > a.Tq || len < n64 || len > a.max_len ||
        len > a.max_pages * a.page) {
        if (blockIdx.x == 0 && h == 0 && tid == 0) raise_status(a.status, DS41_E_INDEX);
        return;
    }
    const int runs = FEW ? a.runs : 1, run = FEW ? (int)blockIdx.x % runs : 0;
    const int n = (int)n64, t0 = (FEW ? (int)blockIdx.x / runs : (int)blockIdx.x) * a.TT;
    if (t0 >= n) return;
    const int toks = min(a.TT, n - t0), quads = (toks + 3) / 4;
    const int p0 = len - n + t0;                           // the first token's place
    const int vis = ((p0 + toks - 1) >> a.page_shift) + 1;  // blocks that some token sees
    // (nobody writes into a CTA that has not started)
    if (FEW && runs > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;\n" ::: "memory");
    // shared memory: the queries' fragments, their scales, the scores
    const int pairs = a.heads / 2;
    uint4* frag = reinterpret_cast<uint4*>(smem);  // [quad][pair][two k steps][32]
    float* qs = reinterpret_cast<float*>(frag + (a.TT + 3) / 4 * pairs * KS * 16);  // [token][heads]
    uint32_t* sc = reinterpret_cast<uint32_t*>(qs + (a.TT + 3) / 4 * 4 * a.heads);  // [token][NB]
    uint16_t* lists = reinterpret_cast<uint16_t*>(sc + a.TT * a.NB);               // [warp][LIST]
    const int32_t* table = a.table + (int64_t)b * a.max_pages;

    for (int h0 = 0; h0 < a.G; h0 += a.heads) {
        const int hs = min(a.heads, a.G - h0), hp = (hs + 1) / 2;
        // rows g and g + 8 of 16 blocks: pages a round ahead of codes
        int page[2];
        uint4 raw[2][KS / 4];
        float scale[2];
        auto look = [&](int j0) {
#pragma unroll
            for (int r = 0; r < 2; r++) page[r] = j0 + g + 8 * r < vis ? table[j0 + g + 8 * r] : 0;
        };
        auto fetch = [&] {
#pragma unroll
            for (int r = 0; r < 2; r++) {
                const bool ok = page[r] >= 0 && page[r] < a.n_pages;
                if (!ok && c == 0) raise_status(a.status, DS41_E_INDEX);
                const int64_t at = (int64_t)(ok ? page[r] : 0) * a.kvh + h;
                scale[r] = ok ? a.scales[at] : __uint_as_float(0x7fc00000u);
#pragma unroll
                for (int x = 0; x < KS / 4; x++) {
                    raw[r][x] = make_uint4(0, 0, 0, 0);
                    if ((c + 4 * x) * 16 < a.hd && ok)
                        raw[r][x] =
                            *reinterpret_cast<const uint4*>(a.codes + at * a.hd + (c + 4 * x) * 16);
                }
            }
        };
        const int round = runs * SEL_WARPS * 16, start = (run * SEL_WARPS + warp) * 16;
        look(start);
        if (FEW) {
            fetch();
            look(start + round);
        }
        // the queries: half a warp a row, eight elements a lane, two rows of each half at a time
        const int rows = quads * 4 * hp * 2, half = lane >> 4, l = lane & 15;
        const int by = (65536 + 2 * hp - 1) / (2 * hp);  // x / (2 hp), x at most 32 * 32
        for (int x0 = 2 * warp + half; x0 < rows; x0 += 4 * SEL_WARPS) {
            uint4 w[2];
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int x = x0 + u * 2 * SEL_WARPS, t = (x * by) >> 16, y = x - t * 2 * hp;
                w[u] = make_uint4(0, 0, 0, 0);
                if (t < toks && y < hs && l * 8 < a.hd)
                    w[u] = *reinterpret_cast<const uint4*>(a.q + (q0 + t0 + t) * a.q_tok +
                                                           ((int64_t)h * a.G + h0 + y) * a.q_head +
                                                           l * 8);
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int x = x0 + u * 2 * SEL_WARPS, t = (x * by) >> 16, y = x - t * 2 * hp;
                uint32_t top = __vmaxu2(__vmaxu2(w[u].x & 0x7fff7fffu, w[u].y & 0x7fff7fffu),
                                        __vmaxu2(w[u].z & 0x7fff7fffu, w[u].w & 0x7fff7fffu));
#pragma unroll
                for (int o = 8; o > 0; o >>= 1)
                    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
                const Int8 r(max(top & 0xffffu, top >> 16) << 16);
                const uint32_t in[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
                uint32_t out[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const __half2 c2 =
                        __floats2half2_rn(r.code(__uint_as_float(in[e] << 16)),
                                          r.code(__uint_as_float(in[e] & 0xffff0000u)));
                    out[e] = *reinterpret_cast<const uint32_t*>(&c2);
                }
                if (x >= rows) continue;
                // elements 8 l ..: two steps' words of lane (column, l / 2 % 4), side by side
                if (l * 8 < HD) {
                    const int st = (l >> 3) * 4 + 2 * (l & 1), col = 2 * (t & 3) + (y & 1);
                    frag[(((t >> 2) * pairs + (y >> 1)) * KS + st) * 16 + col * 4 +
                         ((l >> 1) & 3)] = make_uint4(out[0], out[1], out[2], out[3]);
                }
                // (a head that is not there does not count)
                if (l == 0)
                    qs[t * a.heads + y] =
                        t < toks && y < hs ? r.scale : __uint_as_float(0x7fc00000u);
            }
        }
        __syncthreads();
        if (FEW && runs > 1) asm volatile("barrier.cluster.wait.aligned;\n" ::: "memory");
        for (int j0 = start; j0 < vis; j0 += round) {
            uint32_t af[KS][4];
            if (!FEW) {
                fetch();
                look(j0 + round);
            }
            const float ks[2] = {scale[0], scale[1]};
#pragma unroll
            for (int r = 0; r < 2; r++)
#pragma unroll
                for (int x = 0; x < KS / 4; x++) {
                    const uint4 w = raw[r][x];
                    int8x4_to_f16(w.x, af[4 * x][r], af[4 * x][r + 2]);
                    int8x4_to_f16(w.y, af[4 * x + 1][r], af[4 * x + 1][r + 2]);
                    int8x4_to_f16(w.z, af[4 * x + 2][r], af[4 * x + 2][r + 2]);
                    int8x4_to_f16(w.w, af[4 * x + 3][r], af[4 * x + 3][r + 2]);
                }
            if (FEW) {
                fetch();
                look(j0 + 2 * round);
            }
            for (int qd = 0; qd < quads; qd++) {
                const int t = qd * 4 + c;
                float best[2] = {__uint_as_float(0x7fc00000u), __uint_as_float(0x7fc00000u)};
                for (int i = 0; i < hp; i++) {
                    const uint4* f = frag + (qd * pairs + i) * KS * 16 + lane;
                    float d[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int st = 0; st < KS; st += 2) {
                        const uint4 w = f[st * 16];
                        mma_f16(d, af[st][0], af[st][1], af[st][2], af[st][3], w.x, w.y);
                        mma_f16(d, af[st + 1][0], af[st + 1][1], af[st + 1][2], af[st + 1][3], w.z,
                                w.w);
                    }
                    const float2 s = *reinterpret_cast<const float2*>(qs + t * a.heads + 2 * i);
                    best[0] = fmaxf(best[0], fmaxf(__fmul_rn(d[0], s.x), __fmul_rn(d[1], s.y)));
                    best[1] = fmaxf(best[1], fmaxf(__fmul_rn(d[2], s.x), __fmul_rn(d[3], s.y)));
                }
                if (t >= toks) continue;
                uint32_t* to = sc + t * a.NB + j0 + g;
#pragma unroll
                for (int r = 0; r < 2; r++, to += 8) {
                    if (j0 + g + 8 * r >= vis) break;
                    float s = best[r];
                    if (a.heads < a.G) {  // the group's heads come in turns
                        if (h0 > 0) s = fmaxf(s, __uint_as_float(*to));
                        if (h0 + a.heads < a.G) {
                            *to = __float_as_uint(s);
                            continue;
                        }
                    }
                    const uint32_t rank = rank_of(__fmul_rn(s, ks[r]));
                    if (FEW && runs > 1)
                        asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(
                                         cluster_addr(to, t % runs)),
                                     "r"(rank)
                                     : "memory");
                    else
                        *to = rank;
                }
            }
        }
        __syncthreads();
    }
    if (FEW && runs > 1)
        asm volatile("barrier.cluster.arrive.release.aligned;\n"
                     "barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
    // ---- the picks: a warp for a token ----
    for (int t = warp; t < toks; t += SEL_WARPS) {
        if (FEW && t % runs != run) continue;
        const uint32_t* s = sc + t * a.NB;
        const int cur = (p0 + t) >> a.page_shift;
        int32_t* out = a.idx + ((int64_t)(q0 + t0 + t) * a.kvh + h) * a.topk;
        // all that it sees, or the first and the last ones and what is picked in between
        if (cur < a.topk) {
            for (int j = lane; j < a.topk; j += 32) out[j] = j <= cur ? j : -1;
            continue;
        }
        const int k = a.topk - a.first - a.local, m = cur + 1 - a.first - a.local;
        for (int j = lane; j < a.first; j += 32) out[j] = j;
        for (int j = lane; j < a.local; j += 32) out[a.first + k + j] = a.first + m + j;
        s += a.first;
        out += a.first;
        if (k == 0) continue;
        if (m <= 256) pick<8>(s, m, k, out, a.first, lane);
        else if (m <= 512) pick<16>(s, m, k, out, a.first, lane);
        else pick_of_many(s, m, k, out, a.first, lists + warp * LIST, lane);
    }
}

}  // namespace blocks
}  // namespace ds41

using namespace ds41;

extern "C" int ds41_kv_block_keys(const void* k_cache, const float* k_scales, int fmt,
                                  int64_t n_pages, int64_t page, int64_t kvh, int64_t hd,
                                  const int32_t* page_table, int64_t max_pages,
                                  const int32_t* lens, const int32_t* starts, int64_t B,
                                  int64_t max_new, int8_t* codes, float* key_scales,
                                  ds41_stream_t stream) {
    const char* name = "ds41_kv_block_keys";
    blocks::KeyArgs a{};
    // (V is not read)
    if (int rc = check_paged(name, k_cache, k_cache, k_scales, k_scales, fmt, n_pages, page, kvh,
                             hd, &a.kv))
        return rc;
    DS41_REQUIRE(B >= 0 && B < 65536 && max_new >= 0 && max_new < int64_t(1) << 31 &&
                     max_pages >= 0 && max_pages < int64_t(1) << 31,
                 DS41_E_RANGE, "%s: B=%lld max_new=%lld max_pages=%lld", name, (long long)B,
                 (long long)max_new, (long long)max_pages);
    if (B == 0 || max_new == 0) return DS41_OK;
    DS41_REQUIRE(codes && aligned16(codes) && key_scales && aligned_to(key_scales, 4) &&
                     page_table && aligned_to(page_table, 4) && lens && aligned_to(lens, 4) &&
                     aligned_to(starts, 4),
                 DS41_E_ARG,
                 "%s: codes (16-byte aligned), key_scales, page_table and lens must be non-null", name);
    a.table = page_table;
    a.lens = lens;
    a.starts = starts;
    a.max_pages = max_pages;
    a.max_new = max_new;
    a.codes = codes;
    a.scales = key_scales;
    if (int rc = status_word(&a.status)) return rc;
    // pages of a sequence's new rows: one more when they begin inside a page
    int64_t pages = (max_new + page - 1) / page + (starts ? 1 : 0);
    if (pages > max_pages) pages = max_pages;
    if (pages > 65535) pages = 65535;  // (a CTA goes on behind the grid)
    if (pages < 1) pages = 1;
    return launch_pdl(fmt == DS41_KV_E4M3 ? blocks::keys_kernel<true> : blocks::keys_kernel<false>,
                      dim3((unsigned)((kvh + blocks::KEY_WARPS - 1) / blocks::KEY_WARPS),
                           (unsigned)pages, (unsigned)B),
                      dim3(blocks::KEY_WARPS * 32), 0, (cudaStream_t)stream, name, a);
}

extern "C" int ds41_block_select(const ds41_bf16* q, int64_t q_tok, int64_t q_head,
                                 const int8_t* codes, const float* key_scales, int64_t n_pages,
                                 int64_t page, int64_t kvh, int64_t hd, const int32_t* page_table,
                                 int64_t max_pages, const int32_t* lens, const int32_t* cu_q,
                                 int64_t B, int64_t Tq, int64_t max_q, int64_t max_len, int64_t nh,
                                 int64_t topk, int64_t first, int64_t local, int32_t* idx,
                                 ds41_stream_t stream) {
    const char* name = "ds41_block_select";
    if (int rc = check_heads(name, nh, kvh, hd, 1.0f, 0)) return rc;
    if (int rc = check_cache_form(name, DS41_KV_BF16, kvh, hd)) return rc;
    DS41_REQUIRE(page >= 16 && page <= 256 && (page & (page - 1)) == 0, DS41_E_ARG,
                 "%s: page=%lld must be a power of two of 16 .. 256", name, (long long)page);
    DS41_REQUIRE(n_pages >= 1 && n_pages < (int64_t(1) << 31) / kvh, DS41_E_ARG,
                 "%s: n_pages=%lld kvh=%lld", name, (long long)n_pages, (long long)kvh);
    const int64_t lim = int64_t(1) << 31;
    DS41_REQUIRE(B >= 0 && B < 65536 && Tq >= 0 && Tq < lim && max_q >= 0 && max_q < lim &&
                     max_len >= 0 && max_len <= 32768 * page && max_pages >= 0 && max_pages < lim,
                 DS41_E_RANGE,
                 "%s: B=%lld Tq=%lld max_q=%lld max_len=%lld (at most 32768 pages) max_pages=%lld",
                 name, (long long)B, (long long)Tq, (long long)max_q, (long long)max_len,
                 (long long)max_pages);
    DS41_REQUIRE(topk >= 1 && topk <= 1024 && first >= 0 && first <= topk && local >= 1 &&
                     local <= topk - first,
                 DS41_E_ARG, "%s: topk=%lld (1 .. 1024) first=%lld local=%lld (at least 1)", name,
                 (long long)topk, (long long)first, (long long)local);
    if (B == 0 || Tq == 0 || max_q == 0) return DS41_OK;
    DS41_REQUIRE(q && aligned16(q) && codes && aligned16(codes) && key_scales &&
                     aligned_to(key_scales, 4) && page_table && aligned_to(page_table, 4) && lens &&
                     aligned_to(lens, 4) && cu_q && aligned_to(cu_q, 4) && idx && aligned_to(idx, 4),
                 DS41_E_ARG,
                 "%s: q and codes must be non-null and 16-byte aligned, key_scales, page_table, "
                 "lens, cu_q and idx non-null and aligned", name);
    DS41_REQUIRE(good_strides(q_tok, q_head, hd), DS41_E_ARG,
                 "%s: strides must be multiples of 8 and at least hd", name);
    blocks::SelectArgs a{};
    a.q = q;
    a.q_tok = q_tok;
    a.q_head = q_head;
    a.codes = codes;
    a.scales = key_scales;
    a.table = page_table;
    a.lens = lens;
    a.cu_q = cu_q;
    a.idx = idx;
    a.Tq = Tq;
    a.n_pages = n_pages;
    a.max_pages = max_pages;
    a.page = (int)page;
    while ((1 << a.page_shift) < page) a.page_shift++;
    a.kvh = (int)kvh;
    a.hd = (int)hd;
    a.G = (int)(nh / kvh);
    a.max_q = (int)(max_q < Tq ? max_q : Tq);
    a.max_len = (int)max_len;
    a.topk = (int)topk;
    a.first = (int)first;
    a.local = (int)local;
    if (int rc = status_word(&a.status)) return rc;
    // Tokens of a CTA: 32, or what their scores leave room for (two CTAs an SM), or all; query
    // heads at a time: a group, or 32 of it.
    a.NB = (int)((max_len + page - 1) / page + 31) / 32 * 32 + 8;
    a.heads = a.G >= 32 ? 32 : (a.G + 1) / 2 * 2;
    const int HD = hd <= 64 ? 64 : 128;
    const bool few = a.max_q <= 4;
    auto bytes = [&](int tt) {
        const int quads = (tt + 3) / 4;
        return (size_t)quads * (a.heads / 2) * (HD / 16) * 256 + (size_t)quads * 16 * a.heads +
               (size_t)tt * a.NB * 4 + (few ? 8 : 16) * blocks::LIST * 2;
    };
    a.TT = a.max_q < 32 ? a.max_q : 32;
    while (a.TT > 1 && bytes(a.TT) > 110 * 1024)
        a.TT = a.TT > 4 ? (a.TT - 1) / 4 * 4 : a.TT - 1;
    const size_t smem = bytes(a.TT);
    constexpr int MOST = 224 * 1024;
    auto kern = HD == 64 ? (few ? blocks::select_kernel<64, true> : blocks::select_kernel<64, false>)
                         : (few ? blocks::select_kernel<128, true>
                                : blocks::select_kernel<128, false>);
    if (int rc = HD == 64 ? (few ? allow_smem<blocks::select_kernel<64, true>>(MOST, name)
                                 : allow_smem<blocks::select_kernel<64, false>>(MOST, name))
                          : (few ? allow_smem<blocks::select_kernel<128, true>>(MOST, name)
                                 : allow_smem<blocks::select_kernel<128, false>>(MOST, name)))
        return rc;
    const unsigned tiles = (unsigned)((a.max_q + a.TT - 1) / a.TT);
    // CTAs of a cluster: what two an SM leave room for, of a round of blocks each; heads that
    // come in turns read their scores back, which only a CTA's own are for
    const int64_t fit = 2 * (int64_t)sm_count_once() / ((int64_t)tiles * B * kvh);
    const int64_t rounds = (max_len / page + 127) / 128;
    int64_t runs = !few || a.heads < a.G ? 1 : fit < rounds ? fit : rounds;
    a.runs = (int)(runs < 1 ? 1 : runs < 8 ? runs : 8);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles * (unsigned)a.runs, (unsigned)B, (unsigned)kvh);
    cfg.blockDim = dim3((few ? blocks::SELECT_WARPS<true> : blocks::SELECT_WARPS<false>) * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = (cudaStream_t)stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.runs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.runs > 1 ? 2 : 1;
    if (int rc = cuda_check(cudaLaunchKernelEx(&cfg, kern, a), name)) return rc;
    return launch_check(name);
}
