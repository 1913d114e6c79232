// ds41_beam.cu - beam search's selection over beams and vocabulary.
//
// Mathematics.  Beam w offers token t at s_w + x_t - L, L = m + ln l with l = sum_t
// e^{x_t - m}.  Within a beam the order of the offers is that of the x_t, so one pass
// over a row gives both L (a running reference m and sum l for each thread, joined at
// the end) and the row's best k logits; the beams' lists are then merged by offers
// worked out in 64 bits.  l's terms and their sums are f32 (a lane adds at most 32 steps of 9, and
// a tree): L is off by less than 2^-15.6 whatever the row; measured 3.4e-7 at most, rows of
// 5000 .. 129281 logits spread by 0.01 .. 8, of which 8e-8 alike for all rows (ex2.approx).
//
// The best k.  The pass keeps the largest of each 16 logits (a cell); a bound that k logits of
// the run reach follows from the lanes' largest: k lanes at least have one that is not below
// the lowest, over the 8 warps, of a warp's (k / 8)-th largest.  Few cells reach it; their
// logits are read once more and become keys, x as an ordered integer and then the lower
// token, ranked by counting what is better.
//
// What bounds it.  The logits are read once: HBM, if the exponentials (16 a cycle and SM)
// and the instructions around them keep up.  A row is cut into runs so that every SM has
// some; a warp goes through its part of a run alone, with the next steps' logits in flight.
// (64 searches of 8 beams over 129281 bf16 logits, a fifth of them ended: 39 us with the
// merge, 33 in runs_kernel, 3.2 TB/s.)
#include <cfloat>
#include <type_traits>

#include "ds41_softmax_tc.cuh"

namespace ds41 {
namespace beam {

constexpr int WARPS = 8;
constexpr int NT = WARPS * 32;
constexpr int PER = 16;          // logits of a lane in a step
constexpr int STEP = 32 * PER;   // tokens of a warp's step
constexpr int PART = WARPS * STEP;
constexpr int CELLS = 512;       // cells that are looked into at once
constexpr int MAX_PARTS = 32;    // of a run: 32 KiB of cells
constexpr int STAGES = 3;        // of a warp's ring: a step each, and the piece that may begin
template <typename T>            // before it
constexpr int STAGE = STEP * (int)sizeof(T) + 16;
constexpr int MAX_K = 128;
constexpr int OFFERS = 1024;     // that are ranked at once
constexpr int HOLD = 4;          // of them that a merging thread has in registers
constexpr float LOG2E = 1.4426950408889634f;

struct Args {
    const void* x;
    int64_t b_stride, w_stride;
    const float* scores;
    const uint8_t* ended;
    int B, W, V, k, end_token;
    int splits, run;            // runs of a row, tokens of a run
    float* out;
    int32_t* parents;
    int32_t* tokens;
    uint64_t* keys;             // [B * W][splits][k]: the runs' best, 0 behind them
    float2* sums;               // [B * W][splits]: m, l
};

// larger key: larger x, then lower token; -0 is 0
__device__ __forceinline__ uint64_t key_of(float x, int t) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    const uint32_t o = u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
    return ((uint64_t)o << 32) | (uint32_t)~t;
}
__device__ __forceinline__ float x_of(uint64_t key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o >> 31) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int token_of(uint64_t key) { return (int)~(uint32_t)key; }
// larger for larger numbers; a NaN is a number like the least
__device__ __forceinline__ uint32_t rank_of(float x) {
    const uint32_t u = __float_as_uint(x == x ? x : -INFINITY);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float score_of(uint32_t rank) {
    return __uint_as_float((rank >> 31) ? rank ^ 0x80000000u : ~rank);
}
// whether a beam reads its logits
__device__ __forceinline__ bool reads(const Args& a, int64_t row) {
    const float s = a.scores[row];
    return s > -INFINITY && s < INFINITY && !(a.ended && a.ended[row]);
}

// The order of offers: the value (as an ordered integer), then the lower beam, then within
// a beam the logit and the lower token.
struct Offer {
    uint64_t v, key;
    int w;
};
__device__ __forceinline__ bool better(const Offer& x, const Offer& y) {
    if (x.v != y.v) return x.v > y.v;
    if (x.w != y.w) return x.w < y.w;
    return x.key > y.key;
}
// larger for larger numbers (finite ones), -0 as 0; 0 is none
__device__ __forceinline__ uint64_t order_of(double v) {
    uint64_t u = (uint64_t)__double_as_longlong(v);
    if (u == 0x8000000000000000ull) u = 0;
    return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double number_of(uint64_t o) {
    return __longlong_as_double((long long)((o >> 63) ? o ^ 0x8000000000000000ull : ~o));
}

// log (x + lo), x a normal f32 number, lo below its last bit: x = 2^e f with f of 3/4 .. 3/2, whose
// logarithm in f32 is off by 2^-25.  (The logarithm of a sum of thousands in f32 is off by
// 2^-21: offers of two beams that differ by less changed places.  One in 64 bits is some
// sixty operations at two a cycle and SM.)
__device__ __forceinline__ double log_of(float x, float lo) {
    const int e = (int)(__float_as_uint(x) - 0x3f400000u) >> 23;
    const float f = __uint_as_float(__float_as_uint(x) - ((uint32_t)e << 23));
    return fma((double)e, 0.69314718055994530942, (double)(logf(f) + lo / x));
}

// A warp has the tokens of every eighth step of 512 of a run, a lane those at `lane` of each 32
// of them (a cell), whatever the row's alignment: equal rows have equal sums to the last
// bit, and their offers tie.
template <bool BF16>
__device__ __forceinline__ void one_run(const Args& a, int64_t row, int split, float* most) {
    using T = typename std::conditional<BF16, uint16_t, uint32_t>::type;
    // most: [cells] a cell's largest logit, and the ring behind them
    __shared__ uint64_t keys[OFFERS], best[WARPS];
    __shared__ int open[CELLS], n_open, n_keys;
    __shared__ uint32_t nth[WARPS];
    __shared__ float2 parts[WARPS];
    if (!reads(a, row)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k;
    const int64_t b = row / a.W;
    const T* from = static_cast<const T*>(a.x) + b * a.b_stride + (row - b * a.W) * a.w_stride;
    const int j0 = split * a.run, j1 = min(a.V, j0 + a.run);
    auto logit = [&](int t) {
        const uint32_t w = __ldcs(from + t);
        return __uint_as_float(BF16 ? w << 16 : w);
    };
    // The run comes through a ring of stages of each warp, in pieces of 16 bytes on 16-byte
    // boundaries, whatever the row's (off: the row's first logit in its first piece; that
    // piece, which begins before the row, is read logit by logit).
    constexpr int SIZE = sizeof(T), VE = 16 / SIZE, PIECES = STEP / VE;
    uint8_t* ring = reinterpret_cast<uint8_t*>(most + a.run / PER) + warp * (STAGES * STAGE<T>);
    const uint32_t ring_u = smem_u32(ring);
    const int off = (int)(reinterpret_cast<uintptr_t>(from) & 15) / SIZE;
    const T* base = from - off;
    auto fetch = [&](int step) {
        const int s0 = j0 + (step * WARPS + warp) * STEP;  // (a multiple of VE)
        const uint32_t to = ring_u + step % STAGES * STAGE<T>;
        if (s0 > 0 && s0 + STEP + VE <= j1) {  // whole pieces
            const T* at = base + s0 + lane * VE;
#pragma unroll
            for (int u = 0; u < PIECES / 32; u++)
                cp_async16(to + (u * 32 + lane) * 16, at + u * 32 * VE, true);
            if (lane == 0) cp_async16(to + PIECES * 16, at + PIECES * VE, true);
            cp_async_commit();
            return;
        }
#pragma unroll
        for (int u = 0; u < PIECES / 32 + 1; u++) {
            const int i = u * 32 + lane;
            const int t = s0 + i * VE - off;  // the piece's first logit
            if (i > PIECES || t >= j1) continue;
            if (t >= 0) {
                const int bytes = min(16, (a.V - t) * SIZE);  // (none behind the row's last)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to + i * 16),
                             "l"(base + s0 + i * VE), "r"(bytes));
            } else {
                T* at = reinterpret_cast<T*>(ring + step % STAGES * STAGE<T>);
                for (int e = off; e < VE && e - off < a.V; e++) at[e] = from[e - off];
            }
        }
        cp_async_commit();
    };
    // ---- one pass: the sum, and the largest of each cell ----
#pragma unroll
    for (int x = 0; x < STAGES - 1; x++) fetch(x);
    float m = -INFINITY, sum = 0.0f;
    int j = j0 + warp * STEP + lane;
    for (int cell = tid, step = 0; j - lane < j1; j += PART, cell += NT, step++) {
        cp_async_wait<STAGES - 2>();
        __syncwarp();  // the stage is there for all lanes, and the one before it has been read
        fetch(step + STAGES - 1);
        const T* in = reinterpret_cast<const T*>(ring + step % STAGES * STAGE<T>) + off + lane;
        float x[PER];
#pragma unroll
        for (int e = 0; e < PER; e++) {
            uint32_t w = in[e * 32];
            if (BF16) w <<= 16;
            x[e] = __uint_as_float(w);
        }
        if (j - lane + STEP > j1) {
#pragma unroll
            for (int e = 0; e < PER; e++)
                if (j + e * 32 >= j1) x[e] = -INFINITY;
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < PER; e += 2)
            top = e + 1 < PER ? tc::max3(top, x[e], x[e + 1]) : fmaxf(top, x[e]);
        most[cell] = top;
        const float up = fmaxf(m, top), at = up == -INFINITY ? 0.0f : up;
        // (the difference first: x log2(e) rounded would be off by as much as x is large)
        uint64_t s2 = f2(m == up ? sum : sum * tc::ex2((m - at) * LOG2E), 0.0f);
        m = up;
        const uint64_t minus = f2(-at, -at), log2e = f2(LOG2E, LOG2E);
#pragma unroll
        for (int e = 0; e < PER; e += 2) {
            float y, z;
            unf2(mul2(add2(f2(x[e], x[e + 1]), minus), log2e), y, z);
            s2 = add2(s2, f2(tc::ex2(y), tc::ex2(z)));
        }
        float y, z;
        unf2(s2, y, z);
        sum = y + z;
    }
    cp_async_wait<0>();
    // ---- a bound that k logits reach: k lanes at least, `share` of each warp that has tokens,
    // have a largest one that is not below the lowest of those warps' share-th largest ----
    const int busy = min(WARPS, (j1 - j0 + STEP - 1) / STEP), share = (k + busy - 1) / busy;
    if (share <= 32) {
        uint32_t mine = rank_of(m), lowest = 0;
        for (int i = 0; i < share; i++) {
            lowest = __reduce_max_sync(0xffffffffu, mine);
            const unsigned who = __ballot_sync(0xffffffffu, mine == lowest);
            if (lane == __ffs(who) - 1) mine = 0;
        }
        if (lane == 0) nth[warp] = lowest;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        const float s2 = __shfl_xor_sync(0xffffffffu, sum, o);
        const float to = fmaxf(m, m2), ref = to == -INFINITY ? 0.0f : to;
        sum = sum * tc::ex2((m - ref) * LOG2E) + s2 * tc::ex2((m2 - ref) * LOG2E);
        m = to;
    }
    if (lane == 0) parts[warp] = make_float2(m, sum);
    if (tid == 0) n_open = n_keys = 0;
    __syncthreads();
    const int64_t at = row * a.splits + split;
    if (warp == WARPS - 1) {  // the run's sum
        const float2 p = lane < WARPS ? parts[lane] : make_float2(-INFINITY, 0.0f);
        m = p.x;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = __shfl_sync(0xffffffffu, m, 0);
        sum = lane < WARPS ? p.y * tc::ex2((p.x - (m == -INFINITY ? 0.0f : m)) * LOG2E) : 0.0f;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) a.sums[at] = make_float2(m, sum);
    }
    float bound = -FLT_MAX;
    if (share <= 32)
        bound = fmaxf(bound, score_of(__reduce_min_sync(
                                 0xffffffffu, lane < busy ? nth[lane % WARPS] : 0xffffffffu)));
    // ---- the cells that reach it, and their logits that do ----
    const int cells = (j1 - j0 + STEP - 1) / STEP * 32;
    for (int c = tid; c < cells; c += NT)
        if (most[c] >= bound) {
            const int to = atomicAdd(&n_open, 1);
            if (to < CELLS) open[to] = c;
        }
    __syncthreads();
    auto token = [&](int c, int e) { return j0 + (c >> 5) * STEP + e * 32 + (c & 31); };
    if (n_open <= CELLS)
        for (int i = tid; i < n_open * PER; i += NT) {
            const int t = token(open[i / PER], i % PER);
            const float x = t < j1 ? logit(t) : -INFINITY;
            if (x >= bound) {
                const int to = atomicAdd(&n_keys, 1);
                if (to < OFFERS) keys[to] = key_of(x, t);
            }
        }
    __syncthreads();
    // ---- the best k: by counting what is better ----
    const int n = n_keys;
    uint64_t* out = a.keys + at * k;
    if (n_open <= CELLS && n <= OFFERS) {
        for (int i = tid; i < n; i += NT) {
            const uint64_t mine = keys[i];
            int rank = 0;
            for (int y = 0; y < n; y++) rank += keys[y] > mine;
            if (rank < k) out[rank] = mine;
        }
        for (int i = n + tid; i < k; i += NT) out[i] = 0;
        return;
    }
    // (equal logits) one by one: a cell is read again if it may hold a better one than the
    // thread's best so far
    uint64_t below = ~0ull;
    for (int i = 0; i < k; i++) {
        uint64_t mine = 0;
        for (int c = tid; c < cells; c += NT) {
            if (!(most[c] >= -FLT_MAX) || key_of(most[c], token(c, 0)) < mine) continue;
            for (int e = 0; e < PER; e++) {
                const int t = token(c, e);
                const float x = t < j1 ? logit(t) : -INFINITY;
                const uint64_t key = key_of(x, t);
                if (x >= -FLT_MAX && key < below && key > mine) mine = key;
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t v = __shfl_xor_sync(0xffffffffu, mine, o);
            if (v > mine) mine = v;
        }
        if (lane == 0) best[warp] = mine;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WARPS; w++)
            if (best[w] > mine) mine = best[w];
        below = mine;
        if (tid == 0) out[i] = mine;
        __syncthreads();
        if (mine == 0) {
            for (int y = i + 1 + tid; y < k; y += NT) out[y] = 0;
            break;
        }
    }
}

// The lists of all runs of a search's beams merged, best first, by a CTA.  What is not
// below the last entry of some full list (k offers at least are not) is ranked by counting
// what is better; more of it than fits is merged from the lists' heads.
__device__ __forceinline__ void merge(const Args& a, int b, double* base) {
    // base [W]: s_w - L; NaN: the beam offers nothing, or has ended
    uint64_t* ends = reinterpret_cast<uint64_t*>(base + a.W);  // [W]: an ended beam's offer
    __shared__ Offer all[OFFERS];
    __shared__ uint64_t least[NT / 32];
    __shared__ int n_all, taken[NT / 32];
    __shared__ Offer best[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k;
    const int n_lists = a.W * a.splits, n_keys = n_lists * k;
    const uint64_t* keys = a.keys + (int64_t)b * n_keys;
    // (on their way while the sums are joined; keys of beams that have none may be anything)
    uint64_t held[HOLD];
#pragma unroll
    for (int u = 0; u < HOLD; u++) held[u] = u * NT + tid < n_keys ? __ldcg(keys + u * NT + tid) : 0;
    if (tid == 0) n_all = 0;
    for (int w = tid; w < a.W; w += NT) {
        const int64_t row = (int64_t)b * a.W + w;
        const float score = a.scores[row];
        const bool over = a.ended && a.ended[row];
        float m = -INFINITY, sum = 0.0f, lo = 0.0f;  // (the sum, and what its roundings leave out)
        for (int s = 0; s < a.splits; s++) m = fmaxf(m, __ldcg(a.sums + row * a.splits + s).x);
        const float ref = m == -INFINITY ? 0.0f : m;
        for (int s = 0; s < a.splits; s++) {
            const float2 p = __ldcg(a.sums + row * a.splits + s);
            const float y = p.y * expf(p.x - ref), next = __fadd_rn(sum, y);
            const float part = __fsub_rn(next, sum);
            lo += __fadd_rn(__fsub_rn(sum, __fsub_rn(next, part)), __fsub_rn(y, part));
            sum = next;
        }
        // (a sum that a NaN or an infinity is in is NaN; one of nothing but -inf is 0)
        double to = NAN;
        if (!over && score > -INFINITY && score < INFINITY && sum > 0.0f && sum < INFINITY)
            to = (double)score - ((double)m + log_of(sum, lo));
        base[w] = to;
        // an ended beam's one offer is in the place of its first list's first
        ends[w] = over && score > -INFINITY && score < INFINITY ? order_of(score) : 0;
    }
    __syncthreads();
    // offer i of list h, which is run h % splits of beam h / splits
    auto offer_of = [&](int h, int i, uint64_t key) {
        const int w = h / a.splits;
        Offer o{0, 0, w};
        if (i >= k) return o;
        if (base[w] == base[w]) {
            o.key = key;
            if (key) o.v = order_of(base[w] + (double)x_of(key));
        } else if (i == 0 && h == w * a.splits) {
            o.key = key_of(0.0f, a.end_token);
            o.v = ends[w];
        }
        return o;
    };
    auto offer = [&](int h, int i) { return offer_of(h, i, i < k ? __ldcg(keys + h * k + i) : 0); };
    auto write = [&](int i, const Offer& o) {
        const int64_t to = (int64_t)b * k + i;
        // (one that f32 does not hold any more is none: those are the last)
        const float v = o.v ? (float)number_of(o.v) : -INFINITY;
        a.out[to] = v;
        a.parents[to] = v > -INFINITY ? b * a.W + o.w : -1;
        a.tokens[to] = v > -INFINITY ? token_of(o.key) : -1;
    };
    // (arithmetic in 64 bits is slow here, two operations a cycle and SM: once an offer)
    Offer mine_of[HOLD];
    uint64_t from = 0;
#pragma unroll
    for (int u = 0; u < HOLD; u++) {
        const int x = u * NT + tid, h = x / k;
        mine_of[u] = x < n_keys ? offer_of(h, x - h * k, held[u]) : Offer{0, 0, 0};
        if (x < n_keys && x - h * k == k - 1) from = max(from, mine_of[u].v);
    }
    for (int h = HOLD * NT / k + tid; h < n_lists; h += NT)  // (lists that end behind those)
        from = max(from, offer(h, k - 1).v);
    // (an atomic of 64 bits on shared memory is a loop that 32 lists take one after another)
    const uint32_t high = __reduce_max_sync(0xffffffffu, (uint32_t)(from >> 32));
    const uint32_t low =
        __reduce_max_sync(0xffffffffu, (uint32_t)(from >> 32) == high ? (uint32_t)from : 0u);
    if (lane == 0) least[warp] = (uint64_t)high << 32 | low;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; w++) from = max(from, least[w]);
    auto keep = [&](const Offer& o) {
        if (o.v == 0 || o.v < from) return;
        const int to = atomicAdd(&n_all, 1);
        if (to < OFFERS) all[to] = o;
    };
#pragma unroll
    for (int u = 0; u < HOLD; u++) keep(mine_of[u]);
    for (int x = HOLD * NT + tid; x < n_keys; x += NT) {
        const int h = x / k;
        keep(offer(h, x - h * k));
    }
    __syncthreads();
    const int n = n_all;
    if (n <= OFFERS) {
        for (int i = tid; i < n; i += NT) {
            const Offer mine = all[i];
            int rank = 0;
            for (int y = 0; y < n; y++) rank += better(all[y], mine);
            if (rank < k) write(rank, mine);
        }
        for (int i = n + tid; i < k; i += NT) write(i, Offer{0, 0, 0});
        return;
    }
    int* at = reinterpret_cast<int*>(ends + a.W);  // [lists]: the heads' places
    for (int h = tid; h < n_lists; h += NT) at[h] = 0;
    Offer mine;
    int list;
    auto scan = [&] {  // the best head of this thread's lists
        mine = Offer{0, 0, 0x7fffffff};
        list = -1;
        for (int h = tid; h < n_lists; h += NT) {
            const Offer o = offer(h, at[h]);
            if (o.v && (list < 0 || better(o, mine))) {
                mine = o;
                list = h;
            }
        }
    };
    scan();
    for (int i = 0; i < k; i++) {
        Offer o = mine;
        int f = list;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            Offer y;
            y.v = __shfl_xor_sync(0xffffffffu, o.v, d);
            y.key = __shfl_xor_sync(0xffffffffu, o.key, d);
            y.w = __shfl_xor_sync(0xffffffffu, o.w, d);
            const int g = __shfl_xor_sync(0xffffffffu, f, d);
            if (g >= 0 && (f < 0 || better(y, o))) {
                o = y;
                f = g;
            }
        }
        if (lane == 0) {
            best[warp] = o;
            taken[warp] = f;
        }
        __syncthreads();
        for (int w = 0; w < NT / 32; w++)
            if (taken[w] >= 0 && (f < 0 || better(best[w], o))) {
                o = best[w];
                f = taken[w];
            }
        if (tid == 0) write(i, f >= 0 ? o : Offer{0, 0, 0});
        if (f >= 0 && f % NT == tid) {
            at[f]++;
            scan();
        }
        __syncthreads();
    }
}

template <bool BF16>
__global__ void __launch_bounds__(NT, 4) runs_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) float smem[];
    one_run<BF16>(a, blockIdx.y, blockIdx.x, smem);
}
__global__ void __launch_bounds__(NT, 2) merge_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) float smem[];
    merge(a, blockIdx.x, reinterpret_cast<double*>(smem));
}
// Few short rows: a search's runs are a cluster, whose first CTA merges them.
template <bool BF16>
__global__ void __launch_bounds__(NT, 2) search_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ __align__(16) float smem[];
    const int b = blockIdx.y, run = blockIdx.x;
    one_run<BF16>(a, (int64_t)b * a.W + run / a.splits, run % a.splits, smem);
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                     : "memory");
    if (run == 0) merge(a, b, reinterpret_cast<double*>(smem));
}

// Runs of a row: what makes the SM with the most of them end soonest (a run costs its parts and
// about one more).
constexpr int CLUSTER = 8;  // CTAs of a search that is merged in its own launch
constexpr int SHORT = 4;    // parts of a run there, at most
struct Plan {
    int splits, parts;  // runs, and parts of a run
    bool whole;         // one launch (one search of 4 beams over 32000 tokens 9.3 us, two launches 10.2)
    size_t keys_bytes, sums_bytes;
};
Plan make_plan(int64_t B, int64_t W, int64_t V, int64_t k, int sms) {
    const int64_t parts = (V + PART - 1) / PART, rows = B * W;
    int64_t splits = 0, best = 0;
    for (int64_t n = (parts + MAX_PARTS - 1) / MAX_PARTS, end = n + 64; n <= parts && n < end; n++) {
        if (splits > 0 && W * n > 32768) break;  // (the merge keeps a place for each list)
        const int64_t per = (parts + n - 1) / n;
        const int64_t cost = (rows * n + sms - 1) / sms * (per + 1);
        if (best == 0 || cost < best) {
            best = cost;
            splits = n;
        }
    }
    Plan p;
    p.whole = false;
    const int64_t runs = W <= CLUSTER ? CLUSTER / W : 0;  // of a row, in a cluster
    if (runs > 0 && rows * runs <= 2 * sms && (parts + runs - 1) / runs <= SHORT) {
        p.whole = true;
        splits = runs < parts ? runs : parts;
    }
    const int64_t per = (parts + splits - 1) / splits;
    p.splits = (int)((parts + per - 1) / per);
    p.parts = (int)per;
    p.keys_bytes = (size_t)rows * p.splits * k * 8;
    p.sums_bytes = (size_t)rows * p.splits * 8;
    return p;
}
int check_sizes(const char* name, int64_t B, int64_t W, int64_t V, int64_t k) {
    DS41_REQUIRE(B >= 0 && B < 65536 && W >= 1 && W <= 1024 && B * W < 65536 && V >= 1 &&
                     V <= int64_t(1) << 22,
                 DS41_E_RANGE, "%s: B=%lld W=%lld V=%lld", name, (long long)B, (long long)W,
                 (long long)V);
    DS41_REQUIRE(k >= 1 && k <= MAX_K, DS41_E_ARG, "%s: k=%lld (1 .. %d)", name, (long long)k,
                 MAX_K);
    return DS41_OK;
}

}  // namespace beam
}  // namespace ds41

using namespace ds41;

extern "C" size_t ds41_beam_select_workspace_bytes(int64_t B, int64_t W, int64_t V, int64_t k) {
    if (beam::check_sizes("ds41_beam_select_workspace_bytes", B, W, V, k) || B == 0) return 0;
    const beam::Plan p = beam::make_plan(B, W, V, k, sm_count_once());
    return p.keys_bytes + p.sums_bytes;
}

extern "C" int ds41_beam_select(const void* logits, int fmt, int64_t b_stride, int64_t w_stride,
                                const float* scores, const uint8_t* ended, int64_t end_token,
                                int64_t B, int64_t W, int64_t V, int64_t k, float* out_scores,
                                int32_t* parents, int32_t* tokens, void* ws, size_t ws_bytes,
                                ds41_stream_t stream) {
    const char* name = "ds41_beam_select";
    DS41_REQUIRE(fmt == DS41_LOGITS_F32 || fmt == DS41_LOGITS_BF16, DS41_E_ARG,
                 "%s: fmt=%d is neither DS41_LOGITS_F32 nor DS41_LOGITS_BF16", name, fmt);
    if (int rc = beam::check_sizes(name, B, W, V, k)) return rc;
    if (B == 0) return DS41_OK;
    const bool bf16 = fmt == DS41_LOGITS_BF16;
    DS41_REQUIRE(logits && aligned_to(logits, bf16 ? 2 : 4) && scores && aligned_to(scores, 4) &&
                     out_scores && aligned_to(out_scores, 4) && parents && aligned_to(parents, 4) &&
                     tokens && aligned_to(tokens, 4),
                 DS41_E_ARG, "%s: logits, scores and the outputs must be non-null and aligned",
                 name);
    DS41_REQUIRE((W == 1 || w_stride >= V) && (B == 1 || b_stride >= 0), DS41_E_ARG,
                 "%s: strides %lld, %lld", name, (long long)b_stride, (long long)w_stride);
    DS41_REQUIRE(!ended || (end_token >= 0 && end_token < V), DS41_E_ARG, "%s: end_token=%lld",
                 name, (long long)end_token);
    const beam::Plan p = beam::make_plan(B, W, V, k, sm_count_once());
    DS41_REQUIRE(ws && aligned16(ws) && ws_bytes >= p.keys_bytes + p.sums_bytes, DS41_E_WORKSPACE,
                 "%s: needs %zu bytes of workspace, got %zu", name, p.keys_bytes + p.sums_bytes,
                 ws ? ws_bytes : 0);
    beam::Args a{};
    a.x = logits;
    a.b_stride = b_stride;
    a.w_stride = w_stride;
    a.scores = scores;
    a.ended = ended;
    a.B = (int)B;
    a.W = (int)W;
    a.V = (int)V;
    a.k = (int)k;
    a.end_token = (int)end_token;
    a.splits = p.splits;
    a.run = p.parts * beam::PART;
    a.out = out_scores;
    a.parents = parents;
    a.tokens = tokens;
    a.keys = static_cast<uint64_t*>(ws);
    a.sums = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + p.keys_bytes);
    cudaStream_t st = (cudaStream_t)stream;
    const int ring = beam::WARPS * beam::STAGES *
                     (bf16 ? beam::STAGE<uint16_t> : beam::STAGE<uint32_t>);
    const int smem = p.parts * beam::NT * 4 + ring;
    constexpr int MOST = beam::MAX_PARTS * beam::NT * 4 +
                         beam::WARPS * beam::STAGES * beam::STAGE<uint32_t>;
    if (p.whole) {
        if (int rc = bf16 ? allow_smem<beam::search_kernel<true>>(MOST, name)
                          : allow_smem<beam::search_kernel<false>>(MOST, name))
            return rc;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(W * p.splits), (unsigned)B);
        cfg.blockDim = dim3(beam::NT);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = st;
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = (unsigned)(W * p.splits);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 2;
        if (int rc = cuda_check(cudaLaunchKernelEx(&cfg, bf16 ? beam::search_kernel<true>
                                                              : beam::search_kernel<false>, a),
                                name))
            return rc;
        return launch_check(name);
    }
    if (int rc = bf16 ? allow_smem<beam::runs_kernel<true>>(MOST, name)
                      : allow_smem<beam::runs_kernel<false>>(MOST, name))
        return rc;
    if (int rc = launch_pdl(bf16 ? beam::runs_kernel<true> : beam::runs_kernel<false>,
                            dim3((unsigned)p.splits, (unsigned)(B * W)), dim3(beam::NT),
                            smem, st, name, a))
        return rc;
    const size_t places = (size_t)W * 16 + (size_t)W * p.splits * 4;
    if (places > 16 * 1024)
        if (int rc = allow_smem<beam::merge_kernel>(200 * 1024, name)) return rc;
    return launch_pdl(beam::merge_kernel, dim3((unsigned)B), dim3(beam::NT), places, st, name, a);
}
