// ds41_tree.cuh - what the kernels of ds41_tree_attn_fwd share: their
// arguments, a sequence's limits, which keys a row sees, and the end of a row's
// softmax.
#pragma once

#include "ds41_dense.cuh"
#include "ds41_softmax_tc.cuh"

namespace ds41 {
namespace tree {

using tc::bf16x2;
using tc::ex2;

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
    // the split of the keys: chunk keys a split from the first one on (rounded
    // down to `align`), `per` partial results each; with parts > 1:
    // part [parts][Tq][nh][hd], part_ml [parts][Tq][nh] (reference in log2, sum)
    int chunk, align, per, parts;
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
// The first key that some row of the sequence may see, rounded down: no token
// stands before the last earlier row.
__device__ __forceinline__ int first_key(const Args& a, const Seq& s) {
    const int64_t lo = a.window ? (int64_t)s.len - s.n - a.window : 0;
    return lo > 0 ? (int)(lo & ~(int64_t)(a.align - 1)) : 0;
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

// The tensor-core kernel, for more than 16 rows per key/value head; pair: two
// tiles of 128 rows a CTA, else one (of at most 128 rows, two partial results).
int launch_many(const Args& a, bool pair, int row_tiles, int64_t B, const char* name,
                cudaStream_t st);

}  // namespace tree
}  // namespace ds41
