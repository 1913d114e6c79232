// ds41_beam.cu - beam search's selection over beams and vocabulary.
//
// Mathematics.  Beam w offers token t at s_w + x_t - L, L = m + ln l with l = sum_t
// e^{x_t - m}.  Within a beam the order of the offers is that of the x_t, so one pass
// over a row gives both L (a running reference m and sum l for each thread, joined at
// the end) and the row's best k logits; the beams' lists are then merged by offers
// worked out in 64 bits.
//
// The best k.  A bound that k logits of a run reach follows from the lanes' maxima: k lanes
// at least have one that is not below the lowest, over the 8 warps, of a warp's (k / 8)-th
// largest.  What is not below the bound (fewer and fewer) goes to the warp's list as a
// key, x as an ordered integer and then the lower token.  The lists are joined without
// sorting: what is among the best k has fewer than k above it.
//
// What bounds it.  The logits are read once: HBM, if the exponentials (16 a cycle and SM)
// and the instructions around them keep up.  A row is cut into runs so that every SM has
// some; a warp goes through its part of a run alone, with the next step's logits in flight.
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
constexpr int CAP = STEP;        // keys of a warp's list
constexpr int MAX_K = 128;
constexpr int OFFERS = 1024;     // that are ranked at once
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
// larger for larger numbers, 0 for -inf and what is none; -0 is 0
__device__ __forceinline__ uint64_t order_of(double v) {
    if (!(v > -INFINITY)) return 0;
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 0x8000000000000000ull);
}
__device__ __forceinline__ double number_of(uint64_t o) {
    return __longlong_as_double((long long)((o >> 63) ? o ^ 0x8000000000000000ull : ~o));
}

// A warp has the tokens of every eighth step of 512 of a run, token `lane` of each 32 of them,
// whatever the row's alignment: equal rows have equal sums to the last bit, and their
// offers tie.
template <bool BF16>
__global__ void __launch_bounds__(NT, 4) runs_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    __shared__ uint64_t lists[WARPS][CAP];
    __shared__ uint64_t all[WARPS * MAX_K];
    __shared__ int n_of[WARPS], n_all;
    __shared__ float bound_of[WARPS];
    __shared__ volatile uint32_t nth[WARPS];  // the warps' r-th largest lane maxima, as ranks
    __shared__ float2 parts[WARPS];
    const int64_t row = blockIdx.y;
    if (!reads(a, row)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k;
    const int64_t b = row / a.W, first = b * a.b_stride + (row - b * a.W) * a.w_stride;
    const int j0 = blockIdx.x * a.run, j1 = min(a.V, j0 + a.run);
    using T = typename std::conditional<BF16, uint16_t, uint32_t>::type;
    const T* from = static_cast<const T*>(a.x) + first;
    uint64_t* list = lists[warp];
    uint32_t next[PER];
    auto load = [&](int j) {  // a lane's logits of the step whose first one it has at j
        if (j - lane + STEP <= j1) {
            const T* at = from + j;
#pragma unroll
            for (int e = 0; e < PER; e++) next[e] = __ldcs(at + e * 32);
        } else {
#pragma unroll
            for (int e = 0; e < PER; e++)
                next[e] = j + e * 32 < j1 ? (uint32_t)__ldcs(from + j + e * 32)
                                          : BF16 ? 0xff80u : 0xff800000u;  // -inf
        }
    };
    int j = j0 + warp * STEP + lane;
    load(j);
    float m = -INFINITY, sum = 0.0f, bound = -FLT_MAX;
    int have = 0;  // keys of the list; at least k logits of the run's are not below the bound
    // k lanes at least, `share` of each warp that has tokens, have a maximum that is not below
    // the lowest of those warps' share-th largest
    const int busy = min(WARPS, (j1 - j0 + STEP - 1) / STEP), share = (k + busy - 1) / busy;
    for (int step = 1; step == 1 || j - lane < j1; j += WARPS * STEP, step++) {
        float x[PER];
#pragma unroll
        for (int e = 0; e < PER; e++) x[e] = __uint_as_float(BF16 ? next[e] << 16 : next[e]);
        load(j + WARPS * STEP);
        float top = x[0];
#pragma unroll
        for (int e = 1; e < PER; e += 2)
            top = e + 1 < PER ? tc::max3(top, x[e], x[e + 1]) : fmaxf(top, x[e]);
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
        // ---- the best: what bounds them rises with the lanes' maxima (looked at after 1, 2,
        // 4, 8 .. steps) ----
        if ((step & (step - 1)) == 0) {
            if (step == 1 && k <= 32) {  // the k-th largest of the warp's own
                int rank = 0;
#pragma unroll
                for (int o = 1; o < 32; o++) {
                    const float other = __shfl_xor_sync(0xffffffffu, m, o);
                    rank += other > m || (other == m && (lane ^ o) < lane);
                }
                const unsigned kth = __ballot_sync(0xffffffffu, rank == k - 1);
                if (kth) bound = fmaxf(bound, __shfl_sync(0xffffffffu, m, __ffs(kth) - 1));
            }
            if (share <= 16) {
                uint32_t mine = rank_of(m), top_most = 0;
                for (int i = 0; i < share; i++) {
                    top_most = __reduce_max_sync(0xffffffffu, mine);
                    const unsigned who = __ballot_sync(0xffffffffu, mine == top_most);
                    if (lane == __ffs(who) - 1) mine = 0;
                }
                if (lane == 0) nth[warp] = top_most;
            }
            if (step == 1) __syncthreads();  // (every warp has a first step, if one of none)
        }
        if (share <= 16) {
            const uint32_t least =
                __reduce_min_sync(0xffffffffu, lane < busy ? nth[lane % WARPS] : 0xffffffffu);
            bound = fmaxf(bound, score_of(least));
        }
        if (!__any_sync(0xffffffffu, top >= bound)) continue;
        uint32_t pass = 0;
#pragma unroll
        for (int e = 0; e < PER; e++) pass |= (x[e] >= bound ? 1u : 0u) << e;
        const int mine = __popc(pass);
        int before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += v;
        }
        const int added = __shfl_sync(0xffffffffu, before, 31);
        before += have - mine;
        if (have + added <= CAP) {
            for (; pass; pass &= pass - 1) {  // (read once more: no index into registers)
                const int t = j + (__ffs(pass) - 1) * 32;
                const uint32_t w = from[t];
                list[before++] = key_of(__uint_as_float(BF16 ? w << 16 : w), t);
            }
            have += added;
        } else {
            // more than the list holds: the best k of it and of the step, one by one, into
            // their places from the front (what is taken from there is kept in registers)
            uint64_t below = ~0ull, kept[MAX_K / 32] = {};
            int n = 0;
            for (; n < k; n++) {
                uint64_t best = 0;
                for (int i = lane; i < have; i += 32)
                    if (list[i] < below && list[i] > best) best = list[i];
#pragma unroll
                for (int e = 0; e < PER; e++) {
                    const uint64_t key = key_of(x[e], j + e * 32);
                    if (x[e] >= -FLT_MAX && key < below && key > best) best = key;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint64_t v = __shfl_xor_sync(0xffffffffu, best, o);
                    if (v > best) best = v;
                }
                if (best == 0) break;
                below = best;
#pragma unroll
                for (int i = 0; i < MAX_K / 32; i++)
                    if (n == 32 * i + lane) kept[i] = best;
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < MAX_K / 32; i++)
                if (32 * i + lane < n) list[32 * i + lane] = kept[i];
            have = n;
            if (n == k) bound = fmaxf(bound, x_of(below));
        }
        __syncwarp();
    }
    // ---- the run's sum ----
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        const float s2 = __shfl_xor_sync(0xffffffffu, sum, o);
        const float to = fmaxf(m, m2), ref = to == -INFINITY ? 0.0f : to;
        sum = sum * tc::ex2((m - ref) * LOG2E) + s2 * tc::ex2((m2 - ref) * LOG2E);
        m = to;
    }
    if (lane == 0) {
        parts[warp] = make_float2(m, sum);
        n_of[warp] = have;
        bound_of[warp] = bound;
    }
    if (tid == 0) n_all = 0;
    __syncthreads();
    const int64_t at = row * a.splits + blockIdx.x;
    if (tid == 0) {
        for (int w = 1; w < WARPS; w++) m = fmaxf(m, parts[w].x);
        const float ref = m == -INFINITY ? 0.0f : m;
        sum = 0.0f;
        for (int w = 0; w < WARPS; w++) sum += parts[w].y * tc::ex2((parts[w].x - ref) * LOG2E);
        a.sums[at] = make_float2(m, sum);
    }
    // ---- its best k: what is not below the highest bound, by counting what is better ----
    for (int w = 0; w < WARPS; w++) bound = fmaxf(bound, bound_of[w]);
    for (int w = 0; w < WARPS; w++)
        for (int i = tid; i < n_of[w]; i += NT) {
            const uint64_t key = lists[w][i];
            if (x_of(key) < bound) continue;
            const int to = atomicAdd(&n_all, 1);
            if (to < WARPS * MAX_K) all[to] = key;
        }
    __syncthreads();
    const int n = n_all;
    uint64_t* out = a.keys + at * k;
    if (n <= WARPS * MAX_K) {
        for (int i = tid; i < n; i += NT) {
            const uint64_t mine = all[i];
            int rank = 0;
            for (int y = 0; y < n; y++) rank += all[y] > mine;
            if (rank < k) out[rank] = mine;
        }
        for (int i = n + tid; i < k; i += NT) out[i] = 0;
    } else if (warp == 0) {  // (equal logits) one by one
        uint64_t below = ~0ull;
        for (int i = 0; i < k; i++) {
            uint64_t best = 0;
            for (int w = 0; w < WARPS; w++)
                for (int y = lane; y < n_of[w]; y += 32)
                    if (lists[w][y] < below && lists[w][y] > best) best = lists[w][y];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                const uint64_t v = __shfl_xor_sync(0xffffffffu, best, o);
                if (v > best) best = v;
            }
            below = best;
            if (lane == 0) out[i] = best;
        }
    }
}

// A CTA for a search: the lists of all runs of its beams merged, best first.  What is not
// below the last entry of some full list (k offers at least are not) is ranked by counting
// what is better; more of it than fits is merged from the lists' heads.
__global__ void __launch_bounds__(NT) merge_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ double base[];  // [W]: s_w - L; NaN: the beam offers nothing
    __shared__ Offer all[OFFERS];
    __shared__ unsigned long long least;
    __shared__ int n_all, taken[NT / 32];
    __shared__ Offer best[NT / 32];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k;
    const int n_lists = a.W * a.splits;
    if (tid == 0) {
        least = 0;
        n_all = 0;
    }
    for (int w = tid; w < a.W; w += NT) {
        const int64_t row = (int64_t)b * a.W + w;
        double to = NAN;
        if (a.ended && a.ended[row]) {
            to = 0.0;
        } else if (reads(a, row)) {
            float m = -INFINITY, sum = 0.0f;
            for (int s = 0; s < a.splits; s++) m = fmaxf(m, a.sums[row * a.splits + s].x);
            const float ref = m == -INFINITY ? 0.0f : m;
            for (int s = 0; s < a.splits; s++) {
                const float2 p = a.sums[row * a.splits + s];
                sum += p.y * expf(p.x - ref);
            }
            // (a sum that a NaN or an infinity is in is NaN; one of nothing but -inf is 0)
            if (sum > 0.0f && sum < INFINITY)
                to = (double)a.scores[row] - ((double)m + (double)logf(sum));
        }
        base[w] = to;
    }
    __syncthreads();
    // List h is run h % splits of beam h / splits; an ended beam's first list is its one offer.
    auto offer = [&](int h, int i) {
        const int w = h / a.splits;
        const int64_t row = (int64_t)b * a.W + w;
        Offer o{0, 0, w};
        if (a.ended && a.ended[row]) {
            const float s = a.scores[row];
            if (h % a.splits == 0 && i == 0 && s < INFINITY) {
                o.v = order_of(s);
                o.key = key_of(0.0f, a.end_token);
            }
        } else if (i < k && base[w] == base[w]) {
            o.key = a.keys[((int64_t)b * n_lists + h) * k + i];
            if (o.key) o.v = order_of(base[w] + (double)x_of(o.key));
        }
        return o;
    };
    auto write = [&](int i, const Offer& o) {
        const int64_t to = (int64_t)b * k + i;
        a.out[to] = o.v ? (float)number_of(o.v) : -INFINITY;
        a.parents[to] = o.v ? b * a.W + o.w : -1;
        a.tokens[to] = o.v ? token_of(o.key) : -1;
    };
    for (int h = tid; h < n_lists; h += NT) atomicMax(&least, (unsigned long long)offer(h, k - 1).v);
    __syncthreads();
    const uint64_t from = least;
    for (int x = tid; x < n_lists * k; x += NT) {
        const int h = x / k;
        const Offer o = offer(h, x - h * k);
        if (o.v == 0 || o.v < from) continue;
        const int to = atomicAdd(&n_all, 1);
        if (to < OFFERS) all[to] = o;
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
    int* at = reinterpret_cast<int*>(base + a.W);  // [lists]: the heads' places
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

// Runs of a row: what makes the SM with the most of them end soonest (a run costs its parts and
// about one more).
struct Plan {
    int splits, parts;  // runs, and parts of a run
    size_t keys_bytes, sums_bytes;
};
Plan make_plan(int64_t B, int64_t W, int64_t V, int64_t k, int sms) {
    const int64_t parts = (V + PART - 1) / PART, rows = B * W;
    int64_t splits = 1, best = 0;
    for (int64_t n = 1; n <= parts && n <= 64; n++) {
        const int64_t per = (parts + n - 1) / n;
        const int64_t cost = (rows * n + sms - 1) / sms * (per + 1);
        if (n == 1 || cost < best) {
            best = cost;
            splits = n;
        }
    }
    Plan p;
    const int64_t per = (parts + splits - 1) / splits;
    p.splits = (int)((parts + per - 1) / per);
    p.parts = (int)per;
    p.keys_bytes = (size_t)rows * p.splits * k * 8;
    p.sums_bytes = (size_t)rows * p.splits * 8;
    return p;
}
int check_sizes(const char* name, int64_t B, int64_t W, int64_t V, int64_t k) {
    DS41_REQUIRE(B >= 0 && B < 65536 && W >= 1 && W <= 1024 && B * W < 65536 && V >= 1 &&
                     V < int64_t(1) << 30,
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
    if (int rc = launch_pdl(bf16 ? beam::runs_kernel<true> : beam::runs_kernel<false>,
                            dim3((unsigned)p.splits, (unsigned)(B * W)), dim3(beam::NT), 0, st,
                            name, a))
        return rc;
    const size_t smem = (size_t)W * 8 + (size_t)W * p.splits * 4;
    if (smem > 40 * 1024)
        if (int rc = allow_smem<beam::merge_kernel>(200 * 1024, name)) return rc;
    return launch_pdl(beam::merge_kernel, dim3((unsigned)B), dim3(beam::NT), smem, st, name, a);
}
