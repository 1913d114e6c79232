// ds41_beam.cu - beam search's selection over beams and vocabulary.
//
// Mathematics.  Beam w offers token t at s_w + x_t - L, L = m + ln l with l = sum_t
// e^{x_t - m}.  Within a beam the order of the offers is that of the x_t, so one pass
// over a row gives both L (a running reference m and sum l for each thread, joined at
// the end) and the row's best k logits; the beams' lists are then merged by offers
// worked out in 64 bits.
//
// The best k.  A list of keys (x as an ordered integer, then the lower token) gets what
// passes the k-th best so far, which few do after the first part of a row: for that part
// the k-th largest of the threads' maxima is a bound that at least k logits reach.
//
// What bounds it.  The logits are read once: HBM.  A row is cut into runs so that every
// SM has some, and a thread has the next part of its run in flight while it works on
// one.
#include "ds41_softmax_tc.cuh"

namespace ds41 {
namespace beam {

constexpr int NT = 256;
constexpr int PER = 16;          // logits of a thread in a part of a run
constexpr int PART = NT * PER;
constexpr int CAP = 1024;        // keys of a list
constexpr int TRIM = 384;        // a list this long is cut to its best
constexpr int MAX_K = 128;
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
// whether a beam reads its logits
__device__ __forceinline__ bool reads(const Args& a, int64_t row) {
    const float s = a.scores[row];
    return s > -INFINITY && s < INFINITY && !(a.ended && a.ended[row]);
}

struct List {
    uint64_t key[CAP];
    uint64_t sorted[MAX_K];
    uint64_t best[NT / 32];
    float most[NT];
    float bound;
    int n;
};
// The list's best k, in order, and the bound that a further logit has to pass.  All threads.
__device__ __forceinline__ void trim(List& l, int k) {
    const int n = min(l.n, CAP);
    for (int i = threadIdx.x; i < n; i += NT) {
        const uint64_t mine = l.key[i];
        int rank = 0;
        for (int j = 0; j < n; j++) rank += l.key[j] > mine;
        if (rank < k) l.sorted[rank] = mine;
    }
    __syncthreads();
    const int kept = min(n, k);
    for (int i = threadIdx.x; i < kept; i += NT) l.key[i] = l.sorted[i];
    if (threadIdx.x == 0) {
        l.n = kept;
        if (kept == k) l.bound = x_of(l.sorted[k - 1]);
    }
    __syncthreads();
}

// Thread t has the tokens t, t + NT, ... of a part, whatever the row's alignment, so equal
// rows have equal sums to the last bit, and their offers tie.
template <bool BF16>
__global__ void __launch_bounds__(NT, 4) runs_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    __shared__ List l;
    __shared__ float2 parts[NT / 32];
    const int64_t row = blockIdx.y;
    if (!reads(a, row)) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = row / a.W, first = b * a.b_stride + (row - b * a.W) * a.w_stride;
    const int j0 = blockIdx.x * a.run, j1 = min(a.V, j0 + a.run);
    auto load = [&](int t) -> uint32_t {
        if (t >= j1) return BF16 ? 0xff80u : 0xff800000u;  // -inf
        return BF16 ? (uint32_t)__ldcs(static_cast<const uint16_t*>(a.x) + first + t)
                    : __ldcs(static_cast<const uint32_t*>(a.x) + first + t);
    };
    if (tid == 0) {
        l.n = 0;
        l.bound = -INFINITY;
    }
    uint32_t next[PER];
#pragma unroll
    for (int e = 0; e < PER; e++) next[e] = load(j0 + e * NT + tid);
    __syncthreads();
    float m = -INFINITY, sum = 0.0f;
    int have = 0;  // keys of the list
    for (int j = j0; j < j1; j += PART) {
        float x[PER];
#pragma unroll
        for (int e = 0; e < PER; e++) x[e] = __uint_as_float(BF16 ? next[e] << 16 : next[e]);
        if (j + PART < j1) {
#pragma unroll
            for (int e = 0; e < PER; e++) next[e] = load(j + PART + e * NT + tid);
        }
        float top = x[0];
#pragma unroll
        for (int e = 1; e < PER; e++) top = fmaxf(top, x[e]);
        if (top > m) {
            sum *= tc::ex2((m - top) * LOG2E);
            m = top;
        }
        // (the difference first: x log2(e) rounded would be off by as much as x is large)
        const float at = m == -INFINITY ? 0.0f : m;
#pragma unroll
        for (int e = 0; e < PER; e++) sum += tc::ex2((x[e] - at) * LOG2E);
        // ---- the best ----
        auto token = [&](int e) { return j + e * NT + tid; };
        float bound = l.bound;
        const bool start = bound == -INFINITY;
        if (start) {  // the k-th largest of the threads' maxima
            l.most[tid] = top;
            __syncthreads();
            int rank = 0;
            for (int i = 0; i < NT; i++)
                rank += l.most[i] > top || (l.most[i] == top && i < tid);
            if (rank == a.k - 1) l.bound = top;  // (a NaN has no rank; its row offers nothing)
            __syncthreads();
            bound = l.bound;
        }
        if (top > bound || (start && top == bound)) {
#pragma unroll
            for (int e = 0; e < PER; e++)
                if (x[e] > bound || (start && x[e] == bound && x[e] > -INFINITY)) {
                    const int at_n = atomicAdd(&l.n, 1);
                    if (at_n < CAP) l.key[at_n] = key_of(x[e], token(e));
                }
        }
        __syncthreads();
        const int n = l.n;
        __syncthreads();
        if (n > CAP) {
            // more than the list holds (equal logits): the part's best k one by one
            if (tid == 0) l.n = have;
            uint64_t below = ~0ull;
            for (int i = 0; i < a.k; i++) {
                uint64_t mine = 0;
#pragma unroll
                for (int e = 0; e < PER; e++) {
                    const uint64_t key = key_of(x[e], token(e));
                    if (x[e] > -INFINITY && key < below && key > mine) mine = key;
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    const uint64_t y = __shfl_xor_sync(0xffffffffu, mine, o);
                    if (y > mine) mine = y;
                }
                if (lane == 0) l.best[warp] = mine;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < NT / 32; w++)
                    if (l.best[w] > mine) mine = l.best[w];
                if (mine == 0) break;
                below = mine;
                if (tid == 0) l.key[l.n++] = mine;  // (at most TRIM + k of them)
                __syncthreads();
            }
            __syncthreads();
        }
        if (start || n > TRIM || j + PART >= j1) trim(l, a.k);
        have = l.n;
        __syncthreads();
    }
    // ---- the run's results ----
    const int64_t at = row * a.splits + blockIdx.x;
    for (int i = tid; i < a.k; i += NT) a.keys[at * a.k + i] = i < have ? l.key[i] : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
        const float s2 = __shfl_xor_sync(0xffffffffu, sum, o);
        const float to = fmaxf(m, m2), ref = to == -INFINITY ? 0.0f : to;
        sum = sum * tc::ex2((m - ref) * LOG2E) + s2 * tc::ex2((m2 - ref) * LOG2E);
        m = to;
    }
    if (lane == 0) parts[warp] = make_float2(m, sum);
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < NT / 32; w++) m = fmaxf(m, parts[w].x);
        const float ref = m == -INFINITY ? 0.0f : m;
        sum = 0.0f;
        for (int w = 0; w < NT / 32; w++) sum += parts[w].y * tc::ex2((parts[w].x - ref) * LOG2E);
        a.sums[at] = make_float2(m, sum);
    }
}

// The order of offers: the value, then the lower beam, then within a beam the logit and
// the lower token.
struct Offer {
    double v;
    int w;
    uint64_t key;
};
__device__ __forceinline__ bool better(const Offer& x, const Offer& y) {
    if (x.v != y.v) return x.v > y.v;
    if (x.w != y.w) return x.w < y.w;
    return x.key > y.key;
}

// A CTA for a search: the lists of all runs of its beams merged, best first.
__global__ void __launch_bounds__(NT) merge_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ double base[];  // [W]: s_w - L; -inf: the beam offers nothing
    __shared__ Offer best[NT / 32];
    __shared__ int winner[NT / 32];
    const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int w = tid; w < a.W; w += NT) {
        const int64_t row = (int64_t)b * a.W + w;
        double to = -INFINITY;
        if (reads(a, row)) {
            float m = -INFINITY;
            double sum = 0.0;
            for (int s = 0; s < a.splits; s++) m = fmaxf(m, a.sums[row * a.splits + s].x);
            for (int s = 0; s < a.splits; s++) {
                const float2 p = a.sums[row * a.splits + s];
                sum += (double)p.y * (p.x == -INFINITY && p.y == 0.0f ? 0.0 : exp((double)p.x - m));
            }
            // (a sum that a NaN or an infinity is in is NaN; one of nothing but -inf is 0)
            if (sum > 0.0 && sum < INFINITY) to = (double)a.scores[row] - ((double)m + log(sum));
        }
        base[w] = to;
    }
    __syncthreads();
    // the heads of the lists: list h is run h % splits of beam h / splits; an ended beam's
    // first list is its one offer.  A thread has the lists tid, tid + NT, ... and keeps the
    // best of their heads.
    const int lists = a.W * a.splits;
    auto head = [&](int h, int at) {
        Offer o{-INFINITY, h / a.splits, 0};
        const int64_t row = (int64_t)b * a.W + o.w;
        if (a.ended && a.ended[row]) {
            const float s = a.scores[row];
            if (h % a.splits == 0 && at == 0 && s < INFINITY) {
                o.v = s;
                o.key = key_of(0.0f, a.end_token);
            }
        } else if (at < a.k && base[o.w] > -INFINITY) {
            o.key = a.keys[((int64_t)b * lists + h) * a.k + at];
            if (o.key) o.v = base[o.w] + (double)x_of(o.key);
        }
        if (!(o.v > -INFINITY)) o.v = -INFINITY;
        return o;
    };
    int* at = reinterpret_cast<int*>(base + a.W);  // [lists]: the heads' places
    for (int h = tid; h < lists; h += NT) at[h] = 0;
    __syncthreads();
    Offer mine{-INFINITY, 0x7fffffff, 0};
    int from = -1;
    auto scan = [&] {
        mine = {-INFINITY, 0x7fffffff, 0};
        from = -1;
        for (int h = tid; h < lists; h += NT) {
            const Offer o = head(h, at[h]);
            if (o.v > -INFINITY && (from < 0 || better(o, mine))) {
                mine = o;
                from = h;
            }
        }
    };
    scan();
    for (int i = 0; i < a.k; i++) {
        Offer o = mine;
        int f = from;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            Offer y;
            y.v = __shfl_xor_sync(0xffffffffu, o.v, d);
            y.w = __shfl_xor_sync(0xffffffffu, o.w, d);
            y.key = __shfl_xor_sync(0xffffffffu, o.key, d);
            const int g = __shfl_xor_sync(0xffffffffu, f, d);
            if (g >= 0 && (f < 0 || better(y, o))) {
                o = y;
                f = g;
            }
        }
        if (lane == 0) {
            best[warp] = o;
            winner[warp] = f;
        }
        __syncthreads();
        for (int w = 0; w < NT / 32; w++)
            if (winner[w] >= 0 && (f < 0 || better(best[w], o))) {
                o = best[w];
                f = winner[w];
            }
        if (tid == 0) {
            const int64_t to = (int64_t)b * a.k + i;
            a.out[to] = f >= 0 ? (float)o.v : -INFINITY;
            a.parents[to] = f >= 0 ? b * a.W + o.w : -1;
            a.tokens[to] = f >= 0 ? token_of(o.key) : -1;
        }
        if (f >= 0 && f % NT == tid) {
            at[f]++;
            scan();
        }
        __syncthreads();
    }
}

// Runs of a row: enough for four CTAs an SM over all rows, of a part at least each.
struct Plan {
    int splits, parts;  // runs, and parts of a run
    size_t keys_bytes, sums_bytes;
};
Plan make_plan(int64_t B, int64_t W, int64_t V, int64_t k, int sms) {
    const int64_t parts = (V + PART - 1) / PART, rows = B * W;
    int64_t splits = (4 * (int64_t)sms + rows - 1) / rows;
    if (splits > parts) splits = parts;
    if (splits > 64) splits = 64;
    if (splits < 1) splits = 1;
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
