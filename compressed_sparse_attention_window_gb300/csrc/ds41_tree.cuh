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
    // the work: see `Share`
    int block, align;  // keys of a block; first keys are multiples of align, at most a page
    int tile_rows;     // rows of a tile
    int row_tiles;                // of the most drafted tokens
    int workers;
    float* part;                  // [workers][2][tile_rows][hd]
    float2* part_ml;              // [workers][2][tile_rows]: reference (log2), sum
    int2* ends;                   // [B][kvh][row_tiles]: first and last worker of a unit
    int B;
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
// The first key that is looked at: the first that some row of the sequence does see,
// rounded down within its page, as pages wholly before it have left the window and may
// be gone from the table, or be another sequence's.  A token with an empty mask row
// stands one place before the others; it is looked for only where that key is in
// another page (or group of rows).  (Loops that are not unrolled: nothing reaches them
// without a mask and a window, and every warp fetches past them.)
__device__ __forceinline__ int first_key(const Args& a, const Seq& s) {
    const int64_t at = a.window ? (int64_t)s.len - s.n - a.window + 1 : 0;
    if (at <= 0) return 0;
    if (a.mask && (at & (a.align - 1)) == 0) {
        const int64_t* bits = a.mask + (int64_t)s.q0 * a.mask_words;
#pragma unroll 1
        for (int t = 0; t < s.n; t++, bits += a.mask_words) {
            uint64_t any = 0;
#pragma unroll 1
            for (int i = 0; i * 64 < s.n; i++)
                any |= (uint64_t)bits[i] << (s.n - 64 * i < 64 ? 64 * (i + 1) - s.n : 0);
            if (any == 0) return (int)at - a.align;
        }
    }
    return (int)(at & ~(int64_t)(a.align - 1));
}

__device__ __forceinline__ int blocks_of(const Args& a, const Seq& s, int first) {
    return (s.len - first + a.block - 1) / a.block;
}
__device__ __forceinline__ int tiles_of(const Args& a, const Seq& s) {
    return (s.n * a.G + a.tile_rows - 1) / a.tile_rows;
}

// How the work is shared.  A unit is a tile of rows of one (sequence, key/value
// head); it has a number of key blocks that only the device knows.  All blocks
// of all units, in order (sequence, head, tile of rows, block), are dealt to the
// workers (CTAs) in equal runs, so that sequences of different lengths leave no
// worker with more than its share.  A run covers whole units and at most a part
// of one at each of its ends; whole units go straight to the output, parts to
// the worker's two slots of the workspace (slot 0: a unit that an earlier worker
// began, slot 1: one that a later worker goes on with), to be joined.
struct Share {
    int b;         // sequence of the run's first block
    int64_t at;    // that block, counted within the sequence
    int64_t left;  // blocks of the run
};
// Every thread of the CTA calls it; `report` (one worker) raises DS41_E_INDEX
// for sequences that break their limits.  sh: 2 * NT / 32 + 4 int64 of shared memory.
template <int NT>
__device__ __forceinline__ Share find_share(const Args& a, int64_t* sh, bool report) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (a.B + NT - 1) / NT;
    const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; b++) {
        const Seq s = load_seq(a, b);
        if (s.ok && s.n > 0)
            mine += (int64_t)blocks_of(a, s, first_key(a, s)) * tiles_of(a, s) * a.kvh;
        if (!s.ok && report) raise_status(a.status, DS41_E_INDEX);
    }
    int64_t sum = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, sum, off);
        if (lane >= off) sum += v;
    }
    if (lane == 31) sh[warp] = sum;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int i = 0; i < NT / 32; i++) {
        if (i < warp) before += sh[i];
        total += sh[i];
    }
    // with fewer blocks than workers the last workers have none (and not some in
    // between: the parts of a unit are with consecutive workers)
    const int64_t n = min((int64_t)a.workers, total), w = blockIdx.x;
    const int64_t x0 = w < n ? total * w / n : 0, x1 = w < n ? total * (w + 1) / n : 0;
    int64_t* out = sh + NT / 32;
    const int64_t start = before + sum - mine;
    if (x1 > x0 && x0 >= start && x0 < start + mine) {
        int64_t rem = x0 - start;
        int b = b0;
        for (; b < b1; b++) {
            const Seq s = load_seq(a, b);
            int64_t n = 0;
            if (s.ok && s.n > 0)
                n = (int64_t)blocks_of(a, s, first_key(a, s)) * tiles_of(a, s) * a.kvh;
            if (rem < n) break;
            rem -= n;
        }
        out[0] = b;
        out[1] = rem;
    }
    __syncthreads();
    Share r;
    r.b = x1 > x0 ? (int)out[0] : 0;
    r.at = x1 > x0 ? out[1] : 0;
    r.left = x1 - x0;
    return r;
}

// The next piece of a worker's run: blocks first .. first + count - 1 of a unit
// with n_blocks of them.  Uniform over the CTA; false when the run is done.
struct Piece {
    Seq s;
    int b, h, tile, first, count, n_blocks;
    int key;  // its first
};
__device__ __forceinline__ bool next_piece(const Args& a, Share& w, Piece& p) {
    if (w.left <= 0) return false;
    for (;; w.b++, w.at = 0) {
        if (w.b >= a.B) return false;
        p.s = load_seq(a, w.b);
        if (!p.s.ok || p.s.n == 0) continue;
        const int key = first_key(a, p.s);
        p.n_blocks = blocks_of(a, p.s, key);
        const int tiles = tiles_of(a, p.s);
        const int64_t unit = w.at / p.n_blocks;
        if (unit >= (int64_t)tiles * a.kvh) continue;
        p.b = w.b;
        p.h = (int)(unit / tiles);
        p.tile = (int)(unit % tiles);
        p.first = (int)(w.at - unit * p.n_blocks);
        p.key = key + p.first * a.block;
        p.count = (int)min((int64_t)(p.n_blocks - p.first), w.left);
        w.at += p.count;
        w.left -= p.count;
        return true;
    }
}
__device__ __forceinline__ bool is_whole(const Piece& p) { return p.count == p.n_blocks; }
// the slot of a piece that is not whole
__device__ __forceinline__ int64_t slot_of(const Piece& p) {
    return 2 * (int64_t)blockIdx.x + (p.first == 0 ? 1 : 0);
}
// one thread: which workers a unit's first and last block are with
__device__ __forceinline__ void note_ends(const Args& a, const Piece& p) {
    int2* e = a.ends + ((int64_t)p.b * a.kvh + p.h) * a.row_tiles + p.tile;
    if (p.first == 0) e->x = blockIdx.x;
    if (p.first + p.count == p.n_blocks) e->y = blockIdx.x;
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

// The tensor-core kernel, for more than 16 rows per key/value head, in tiles of
// 256 rows, or of 128 where no sequence has more.
int launch_many(const Args& a, const char* name, cudaStream_t st);

}  // namespace tree
}  // namespace ds41
