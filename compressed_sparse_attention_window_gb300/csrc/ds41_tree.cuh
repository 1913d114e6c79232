// ds41_tree.cuh - what the kernels of ds41_tree_attn_fwd share: their
// arguments, a sequence's limits, which keys a row sees, and the end of a row's
// softmax.
#pragma once

#include "ds41_dense.cuh"

namespace ds41 {
namespace tree {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
constexpr float RESCALE_LOG2 = 4.0f;

struct Args {
    const uint16_t* q;
    int64_t q_tok, q_head;
    PagedKv kv;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu_q;
    const int64_t* mask;
    int max_pages, mask_words, max_len;
    const float* sink;
    uint16_t* o;
    float* lse;
    int64_t Tq;
    int max_q, nh, kvh, hd, G;
    float scale_log2;
    int64_t window;
    // the split of the keys: chunk keys a split; partial results when splits > 1:
    // part [splits][Tq][nh][hd], part_ml [splits][Tq][nh] (reference, sum)
    int chunk, splits;
    float* part;
    float2* part_ml;
    unsigned int* status;
};

// A sequence, checked: its queries q0 .. q0 + n - 1 and its `len` keys.
struct Seq {
    int q0, n, len;
    bool ok;
};
__device__ __forceinline__ Seq load_seq(const Args& a, int b) {
    Seq s;
    s.q0 = a.cu_q[b];
    const int64_t n = (int64_t)a.cu_q[b + 1] - s.q0;
    s.len = a.lens[b];
    s.n = (int)n;
    s.ok = s.q0 >= 0 && n >= 0 && n <= a.max_q && s.q0 + n <= a.Tq && s.len >= n &&
           s.len <= a.max_len && s.len <= (int64_t)a.max_pages * a.kv.page;
    return s;
}
// The first key that some row of the sequence may see, rounded down to a group
// of 16: no token stands before the last earlier row.
__device__ __forceinline__ int first_key(const Args& a, const Seq& s) {
    const int64_t lo = a.window ? (int64_t)s.len - s.n - a.window : 0;
    return lo > 0 ? (int)(lo & ~(int64_t)15) : 0;
}

// What one row sees: of the earlier keys (below pre) those behind lo, of the
// drafted ones those up to chain_last, or those whose bit is set.
struct RowView {
    int64_t lo;
    int pre;
    int chain_last;
    const int64_t* bits;
};
__device__ __forceinline__ RowView row_view(const Args& a, const Seq& s, int t) {
    RowView w;
    w.bits = nullptr;
    w.pre = s.len - s.n;
    w.chain_last = w.pre + t;
    int d = t;
    if (a.mask) {
        w.bits = a.mask + (int64_t)(s.q0 + t) * a.mask_words;
        if (a.window) {
            d = -1;
            for (int i = 0; i * 64 < s.n; i++) {
                uint64_t m = (uint64_t)w.bits[i];
                if (s.n - 64 * i < 64) m &= (1ull << (s.n - 64 * i)) - 1;
                d += __popcll(m);
            }
        }
    }
    w.lo = a.window ? (int64_t)w.pre + d - a.window : -1;
    return w;
}
__device__ __forceinline__ bool seen(const RowView& w, int j, int len) {
    if (j < w.pre) return j > w.lo;
    if (j >= len) return false;
    if (!w.bits) return j <= w.chain_last;
    const int u = j - w.pre;
    return (w.bits[u >> 6] >> (u & 63)) & 1;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The end of a row: the sink joins the denominator; O times factor is the
// output.  A row that sees nothing (m = -inf) has factor 0.
struct Final {
    float factor, lse;
};
__device__ __forceinline__ Final finish(const Args& a, int head, float m, float l) {
    const float snk = a.sink ? a.sink[head] * LOG2E : -INFINITY;
    const float top = fmaxf(m, snk);
    const float base = top == -INFINITY ? 0.0f : top;
    const float f = exp2f(m - base);
    const float den = l * f + exp2f(snk - base);
    Final r;
    r.factor = den == 0.0f ? 0.0f : f / den;
    r.lse = (base + log2f(den)) * LN2;
    return r;
}

}  // namespace tree
}  // namespace ds41
