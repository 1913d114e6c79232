// ds41_block_prompt.cu - attention of packed prompts over the blocks that were picked for
// each token and key/value head, on the 5th-generation tensor cores.
//
// Mathematics.  As ds41_prompt_attn.cu: S = q K^T, p_j = 2^(c S_j - c m), l += sum p_j, O += p V
// with a lazily moved reference m per row, over the keys of the blocks that the row's token
// lists, up to its own place.
//
// Rows and keys.  A tile of 128 rows is TT tokens times the G heads of a group, an item two
// such tiles (2 TT neighbouring tokens), as there.  A tile's keys are the union of its
// tokens' blocks, packed: 128 keys of an MMA block (a record) are as many picked blocks
// (units of at most 128 keys) side by side, each copied by TMA to its own rows.  A row masks
// the units that its token does not list.  The blocks that both tiles list come first, in
// records that both read from one copy; then each tile walks the records of its own,
// the two side by side, so that the tensor core works on one while the softmax of the
// other runs.
//
// Why the union.  The two products of 128 rows and a unit of 64 keys take 512 cycles for the
// whole tile; token by token (16 rows at most, on mma.sync) the unit's K and V would have to
// be read from shared memory once for each token that lists it, 256 cycles each time: the
// union is ahead as soon as two tokens of a tile list the same block, as neighbours mostly do.
//
// Two kernels.  plan_kernel makes the items' records: a table of masks in shared memory (a word
// for 32 tokens and each block), filled from the tokens' lists, is walked in order; what is
// not empty becomes a slot of a record (its first row, and which tokens list it).
// block_prompt_kernel is the kernel of ds41_prompt_attn.cu with the records in place of a range of
// keys.
//
// What bounds it.  A tile's chain of scores, softmax and products, with the other tile's between
// (tensor pipe half busy), and the union's surplus over a token's own blocks.  (Chunk of 8192
// tokens behind 24576, 32 blocks of 64 rows each, alike for 32 tokens one after another, 32
// heads of 128 over 8: 354 us, the plan 19 of them; over all rows 2310.  Six prompts of up to
// 2001 tokens whose lists have nothing in common, 16 heads of 64 over 2: 75 us, over all rows
// 61.)
#include "ds41_prompt.cuh"

namespace ds41 {
namespace bp {

using namespace pa;

// An item: one head group of one pair of tiles of one sequence.  Its records: those of both
// tiles, of tile 0 alone, of tile 1 alone.  Step i: both tiles on record i, or behind
// those each on its own next one.
struct Item {
    int grp;             // head group, -1: nothing
    int q0, n, k0, len;  // its sequence's queries and keys
    int t0;              // first token of tile 0
    int both, own[2];    // records
    int tail, tail_end;  // rows of V behind the last key, in the record of
    int tail_step, tail_tile;
    int id, spare[2];
    __device__ __forceinline__ int steps(int t) const { return both + (t ? own[1] : own[0]); }
    __device__ __forceinline__ int steps() const { return both + max(own[0], own[1]); }
    __device__ __forceinline__ int record(int t, int i) const {
        return i + (t && i >= both ? own[0] : 0);
    }
};
static_assert(sizeof(Item) == 64, "four 16-byte pieces");

constexpr uint32_t ROW = 0x3fffffffu;  // a unit's word: its first row; this: none
constexpr int PLAN = 256;              // threads of plan_kernel
constexpr int SORTED = 64;             // sequences whose pairs it puts in order, at most
constexpr int TABLE = 8192;            // words of its table, at most

struct Params {
    const int32_t* cu_q;
    const int32_t* cu_k;
    const int32_t* idx;
    const float* sink;
    uint16_t* o;
    float* lse;
    int64_t Tq, Tk;
    int B, max_q, max_k, nh, kvh, hd, topk;
    int G, TT, subs;
    int pairs;              // of tiles, at most
    int shift, unit_shift;  // log2 of a block's keys, of a unit's
    int words;              // of a unit's mask: 2 TT tokens
    int rec_words, max_rec;
    int table;              // words of plan_kernel's
    float c;
    Item* items;
    uint32_t* recs;         // [item][max_rec][rec_words]: the units' words, their masks
    unsigned int* status;
};

// exclusive prefix of v over the CTA, and the sum.  sh: PLAN / 32 ints
__device__ __forceinline__ int prefix(int v, int* sh, int& sum) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) sh[warp] = x;
    __syncthreads();
    int before = 0;
    sum = 0;
#pragma unroll
    for (int w = 0; w < PLAN / 32; w++) {
        if (w < warp) before += sh[w];
        sum += sh[w];
    }
    __syncthreads();
    return before + x - v;
}

__global__ void __launch_bounds__(PLAN) plan_kernel(const Params p) {
    pdl_wait();
    pdl_trigger();
    extern __shared__ uint32_t table[];
    __shared__ int sh[PLAN / 32], pairs_of[SORTED], units_of[3];  // (both tiles', tile 0's, tile 1's)
    __shared__ __align__(16) Item it;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, id = blockIdx.x;
    // (head group by head group: what is under way at a time reads the keys of one or two, which
    // the L2 holds)
    const int grp = id / p.pairs, w = id - grp * p.pairs, h = grp / p.subs;
    if (tid == 0) {
        it = Item{};
        it.grp = -1;
        it.id = id;
    }
    if (tid < 3) units_of[tid] = 0;
    __syncthreads();
    // sequence b's pairs of tiles
    auto load = [&](int b, int& q0, int& n, int& k0, int& len) {
        q0 = n = k0 = len = 0;
        if (b < p.B) {
            q0 = p.cu_q[b];
            k0 = p.cu_k[b];
            const int64_t ln = (int64_t)p.cu_q[b + 1] - q0, lk = (int64_t)p.cu_k[b + 1] - k0;
            if (q0 >= 0 && ln >= 0 && ln <= p.max_q && q0 + ln <= p.Tq && k0 >= 0 && lk >= ln &&
                lk <= p.max_k && k0 + lk <= p.Tk) {
                n = (int)ln;
                len = (int)lk;
            } else if (id == 0) {
                raise_status(p.status, DS41_E_INDEX);
            }
        }
        return (n + 2 * p.TT - 1) / (2 * p.TT);
    };
    auto take = [&](int q0, int n, int k0, int len, int pair) {
        it.grp = grp;
        it.q0 = q0;
        it.n = n;
        it.k0 = k0;
        it.len = len;
        it.t0 = pair * 2 * p.TT;
    };
    // the sequence and the pair: all sequences' latest first, as their lists are the longest (six
    // prompts of 1175 .. 2001 tokens: 75 us, sequence by sequence 84; more than 64 sequences
    // are taken one after the other)
    if (p.B > 1 && p.B <= SORTED) {
        int q0, n, k0, len;
        const int mine = load(tid, q0, n, k0, len);
        if (tid < SORTED) pairs_of[tid] = mine;
        __syncthreads();
        // how many pairs are at place x of their sequence or behind it
        auto behind = [&](int x) {
            int sum = 0;
            for (int b = 0; b < p.B; b++) sum += max(0, pairs_of[b] - x);
            return sum;
        };
        // the last place at which there are more than w
        int at = 0;
        int span = (int)((min((int64_t)p.max_q, p.Tq) + 2 * p.TT - 1) / (2 * p.TT));
        for (int step; span > 0; span = step) {
            step = (span + PLAN - 1) / PLAN;
            const int yes = __syncthreads_count(tid * step < span && behind(at + tid * step) > w);
            at = yes ? at + (yes - 1) * step : -1;
            if (at < 0 || step == 1) break;
        }
        if (at >= 0) {
            int sum;
            const int rank = prefix(mine > at, sh, sum);
            if (mine > at && rank == w - behind(at + 1)) take(q0, n, k0, len, at);
        }
    } else {
        for (int b0 = 0, base = 0; b0 < p.B; b0 += PLAN) {
            int q0, n, k0, len, sum;
            const int mine = load(b0 + tid, q0, n, k0, len);
            const int at = base + prefix(mine, sh, sum);
            if (w >= at && w < at + mine) take(q0, n, k0, len, at + mine - 1 - w);
            base += sum;
            if (w < base && id != 0) break;
        }
    }
    __syncthreads();
    if (it.grp < 0) {
        if (tid == 0) p.items[id].grp = -1;
        return;
    }
    const int toks = min(2 * p.TT, it.n - it.t0), p0 = it.len - it.n + it.t0;
    const int32_t* lists = p.idx + ((int64_t)(it.q0 + it.t0) * p.kvh + h) * p.topk;
    const int blocks = ((p0 + toks - 1) >> p.shift) + 1, W = p.words;
    const int range = p.table / W;
    const int per = 1 << (p.shift - p.unit_shift);
    const int nu_shift = 7 - p.unit_shift, nu = 1 << nu_shift;
    uint32_t* recs = p.recs + (int64_t)id * p.max_rec * p.rec_words;
    // the masks of the blocks from r0 on: a warp for a token, its list 32 entries at a time
    auto fill = [&](int r0, int size, bool report) {
        for (int x = tid; x < size * W; x += PLAN) table[x] = 0;
        __syncthreads();
        constexpr int U = 4, NW = PLAN / 32;  // tokens of a warp at a time
        for (int tok0 = warp; tok0 < toks; tok0 += U * NW) {
            int x[U];
#pragma unroll
            for (int u = 0; u < U; u++)
                x[u] = tok0 + u * NW < toks && lane < p.topk
                           ? lists[(int64_t)(tok0 + u * NW) * p.kvh * p.topk + lane]
                           : -1;
#pragma unroll
            for (int u = 0; u < U; u++) {
                const int tok = tok0 + u * NW;
                if (tok >= toks) break;
                const int32_t* list = lists + (int64_t)tok * p.kvh * p.topk;
                const int cur = (p0 + tok) >> p.shift;
                for (int i0 = 0, last = -1;; ) {
                    int before = __shfl_up_sync(0xffffffffu, x[u], 1);
                    if (lane == 0) before = last;
                    last = __shfl_sync(0xffffffffu, x[u], 31);
                    // it ends at the first entry that does not rise or lies past its token
                    const unsigned bad = __ballot_sync(0xffffffffu, x[u] <= before || x[u] > cur);
                    const int end = bad ? __ffs(bad) - 1 : 32;
                    if (lane < end && x[u] >= r0 && x[u] < r0 + size)
                        atomicOr(&table[(x[u] - r0) * W + (tok >> 5)], 1u << (tok & 31));
                    if (report && lane == end && x[u] != -1) raise_status(p.status, DS41_E_INDEX);
                    i0 += 32;
                    if (bad || i0 >= p.topk) break;
                    x[u] = i0 + lane < p.topk ? list[i0 + lane] : -1;
                }
            }
        }
        __syncthreads();
    };
    // which tiles list block r0 + x: 0 neither, 1 tile 0, 2 tile 1, 3 both
    auto tiles_of = [&](int x, int size) {
        uint32_t tiles = 0;
        if (x < size)
            for (int y = 0; y < W; y++) {
                const uint32_t m = table[x * W + y], low = low_bits(p.TT - 32 * y);
                tiles |= (m & low ? 1u : 0u) | (m & ~low ? 2u : 0u);
            }
        return tiles;
    };
    // the units of each kind
    for (int r0 = 0; r0 < blocks; r0 += range) {
        const int size = min(range, blocks - r0);
        fill(r0, size, r0 == 0);
        uint32_t mine = 0;  // (three counts in one word: at most 32 blocks a thread, two units each)
        for (int x = tid; x < size; x += PLAN) {
            const uint32_t tiles = tiles_of(x, size);
            // (a block's second unit may lie behind the last key)
            const int n = per == 1 || ((r0 + x) << p.shift) + KB < it.len ? per : 1;
            if (tiles) mine += (uint32_t)n << (10 * (tiles == 3 ? 0 : tiles));
        }
#pragma unroll
        for (int k = 0; k < 3; k++) {
            const int n = __reduce_add_sync(0xffffffffu, (mine >> (10 * k)) & 1023);
            if (lane == 0 && n) atomicAdd(&units_of[k], n);
        }
        __syncthreads();
    }
    // The units of both tiles that do not fill a record (their first ones: the last may end behind
    // the last key) go to the tiles' own records where that saves a step.
    auto recs_of = [&](int units) { return (units + nu - 1) >> nu_shift; };
    const int most = max(units_of[1], units_of[2]), over = units_of[0] & (nu - 1);
    const int moved = units_of[0] > over && recs_of(most + over) == recs_of(most) ? over : 0;
    const int n_both = recs_of(units_of[0] - moved), n_own[2] = {recs_of(units_of[1] + moved),
                                                                 recs_of(units_of[2] + moved)};
    const int base[3] = {0, n_both, n_both + n_own[0]};
    // into their records
    int found[3] = {0, 0, 0};  // blocks so far
    for (int r0 = 0; r0 < blocks; r0 += range) {
        const int size = min(range, blocks - r0);
        if (blocks > range) fill(r0, size, false);
        for (int x0 = 0; x0 < size; x0 += PLAN) {
            const int x = x0 + tid;
            const uint32_t tiles = tiles_of(x, size);
            // (three counts of at most 256 in one word)
            const int kind = tiles == 3 ? 0 : (int)tiles;
            int sums;
            const int before = prefix(tiles ? 1 << (10 * kind) : 0, sh, sums);
            const int at = (kind == 0 ? found[0] : kind == 1 ? found[1] : found[2]) +
                           ((before >> (10 * kind)) & 1023);
#pragma unroll
            for (int k = 0; k < 3; k++) found[k] += (sums >> (10 * k)) & 1023;
            if (!tiles) continue;
            for (int k = 0; k < per; k++) {
                const int row = ((r0 + x) << p.shift) + (k << p.unit_shift);
                if (row >= it.len) break;  // (behind the last key: only the last block's)
                int u = at * per + k;
                auto put = [&](int first, int u) {
                    const int slot = u & (nu - 1);
                    uint32_t* to = recs + (int64_t)(first + (u >> nu_shift)) * p.rec_words;
                    to[slot] = (uint32_t)row;
                    for (int y = 0; y < W; y++) to[nu + slot * W + y] = table[x * W + y];
                };
                if (kind == 0 && u < moved) {
                    put(base[1], units_of[1] + u);
                    put(base[2], units_of[2] + u);
                    continue;
                }
                u -= kind == 0 ? moved : 0;
                const int rec = u >> nu_shift, slot = u & (nu - 1);
                put(kind == 0 ? base[0] : kind == 1 ? base[1] : base[2], u);
                if (row + (1 << p.unit_shift) > it.len) {
                    it.tail = (slot << p.unit_shift) + it.len - row;
                    it.tail_end = (slot + 1) << p.unit_shift;
                    it.tail_step = rec + (kind ? base[1] : 0);
                    it.tail_tile = kind == 2;
                }
            }
        }
        __syncthreads();
    }
    // slots behind a kind's last unit
#pragma unroll
    for (int kind = 0; kind < 3; kind++) {
        const int n = units_of[kind] + (kind ? moved : -moved), slots = recs_of(n) << nu_shift;
        for (int u = n + tid; u < slots; u += PLAN) {
            uint32_t* to = recs + (int64_t)(base[kind] + (u >> nu_shift)) * p.rec_words;
            const int slot = u & (nu - 1);
            to[slot] = ROW;
            for (int y = 0; y < W; y++) to[nu + slot * W + y] = 0;
        }
    }
    if (tid == 0) {
        it.both = n_both;
        it.own[0] = n_own[0];
        it.own[1] = n_own[1];
    }
    __syncthreads();
    if (tid < 4)
        reinterpret_cast<int4*>(p.items + id)[tid] = reinterpret_cast<const int4*>(&it)[tid];
}

// One thread's row of 128 scores, as softmax_block, with masks that are mostly whole words of
// 32 keys: a word's maximum and sum count or not, and its weights are kept or cleared,
// whatever its scores hold.  Only where some row of the warp sees a part of a word (its own
// block, or half a word of a block of 16) are scores masked key by key first.  The
// weights are worked out a word at a time in a loop, the scores read once more from tensor
// memory: unrolled, with all scores in registers, the code streams through the instruction
// caches at every step.  Weights are rounded to bf16, as the values are, for the second product (off
// by 2^-8 of themselves: outputs 2.3e-3 from 64 bits at most, with weights in 32 bits 1.7e-3).
// (8192 tokens over 32768 keys: 354 us; unrolled 389; with a second
// instance that masks throughout, for the few steps that need it, 416.)
template <int D>
__device__ __forceinline__ void softmax_words(uint32_t tm_s, uint32_t tm_o, bool have_o,
                                              const uint32_t (&vis)[4], bool parts, float c,
                                              bool live, RowState& st) {
    float top = -INFINITY;
    {
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; i++) tc_ld32(tm_s + 32 * i, s[i]);
        tc_wait_ld();
        if (parts) {
#pragma unroll
            for (int i = 0; i < 4; i++) {
                prepare32<false, true>(s[i], nullptr, vis[i]);
                tc_st32(tm_s + 32 * i, s[i]);
            }
            tc_wait_st();
        }
#pragma unroll
        for (int i = 0; i < 4; i++) top = fmaxf(top, vis[i] ? max32(s[i]) : -INFINITY);
    }
    // (-inf - -inf is NaN: no move)
    const bool move = (top - st.m) * c > SM_RESCALE_LOG2 && live;
    if (__any_sync(0xffffffffu, move)) {
        const float f = move ? ex2((st.m - top) * c) : 1.0f;
        if (move) st.m = top;
        st.l *= f;
        if (have_o) rescale<D>(tm_o, f);
    }
    float base = st.m == -INFINITY ? 0.0f : st.m * c, less = 0.0f;
    if (fabsf(base) > 0x1p22f) {
        // c m itself is rounded by more than a fraction of one power of two: take
        // the differences first
        less = st.m;
        base = 0.0f;
    }
    const bool far = __any_sync(0xffffffffu, less != 0.0f);
    const uint32_t seen =
        (vis[0] ? 1u : 0u) | (vis[1] ? 2u : 0u) | (vis[2] ? 4u : 0u) | (vis[3] ? 8u : 0u);
#pragma unroll 1
    for (int i = 0; i < 4; i++) {
        uint32_t s[32], pk[16];
        tc_ld32(tm_s + 32 * i, s);
        tc_wait_ld();
        if (far) {
#pragma unroll
            for (int e = 0; e < 32; e++) s[e] = __float_as_uint(u2f(s[e]) - less);
        }
        uint64_t part[2] = {0, 0};
        weights32<false, false>(s, pk, c, base, nullptr, 0, part);
        float x, y;
        unf2(add2(part[0], part[1]), x, y);
        const bool on = (seen >> i) & 1;
        st.l += on ? x + y : 0.0f;
#pragma unroll
        for (int e = 0; e < 16; e++) pk[e] &= on ? 0xffffffffu : 0u;
        tc_st16(tm_s + 16 * i, pk);
    }
    tc_wait_st();
}

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    block_prompt_kernel(const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k,
                        const __grid_constant__ CUtensorMap map_v, const Params p) {
    using C = Cfg<D>;
    constexpr int ITEMS = 4;  // items looked up ahead
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(sm);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
    uint64_t* b_q = bars;                      // an item's queries landed [QB]
    uint64_t* b_qe = b_q + C::QB;              // and have been used [QB]
    uint64_t* b_full = b_qe + C::QB;           // stage landed
    uint64_t* b_empty = b_full + C::STAGES;    // stage read
    uint64_t* b_s = b_empty + C::STAGES;       // S_t in tensor memory [2]
    uint64_t* b_p = b_s + 2;                   // P_t in tensor memory, O_t rescaled [2]
    uint64_t* b_o = b_p + 2;                   // O_t complete [2]
    uint64_t* b_oe = b_o + 2;                  // O_t read [2]
    uint64_t* b_tail = b_oe + 2;               // the V block that ends behind the last key landed
    uint64_t* b_fix = b_tail + 1;              // its rows behind the last key are zero
    uint64_t* b_item = b_fix + 1;              // an item is known [ITEMS]
    uint64_t* b_iteme = b_item + ITEMS;        // and every role is through with it
    uint64_t* b_clc = b_iteme + ITEMS;         // the answer to a request for another item
    uint64_t* b_end = b_clc + 1;               // every product is complete
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b_end + 1);
    volatile int* abort_f = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile uint32_t* tail_stage = tmem_slot + 2;  // where the V behind whose rows b_tail asks is
    Item* items = reinterpret_cast<Item*>(tmem_slot + 4);
    static_assert((2 * C::QB + 2 * C::STAGES + 12 + 2 * ITEMS) * 8 + 16 + ITEMS * sizeof(Item) <=
                      624,
                  "barrier area");
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;

    if (threadIdx.x == 32) {
        for (int i = 0; i < C::QB; i++) {
            mbar_init(&b_q[i], 1);
            mbar_init(&b_qe[i], 1);
        }
        for (int i = 0; i < C::STAGES; i++) {
            mbar_init(&b_full[i], 1);
            mbar_init(&b_empty[i], 1);
        }
        for (int t = 0; t < 2; t++) {
            mbar_init(&b_s[t], 1);
            mbar_init(&b_p[t], 4);
            mbar_init(&b_o[t], 1);
            mbar_init(&b_oe[t], 4);
        }
        mbar_init(b_tail, 1);
        mbar_init(b_fix, 1);
        for (int i = 0; i < ITEMS; i++) {
            mbar_init(&b_item[i], 1);
            mbar_init(&b_iteme[i], 11);
        }
        mbar_init(b_clc, 1);
        mbar_init(b_end, 1);
        *abort_f = 0;
        mbar_init_fence();
    }
    if (warp == 1) {
        asm volatile(
            "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(
                smem_u32(tmem_slot))
            : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    // rows of the query tiles that no copy fills
    const int used = p.TT * p.G;
    if (used < ROWS) {
        const int per = (ROWS - used) * 8;  // 16-byte pieces of one 64-column block
        for (int x = threadIdx.x; x < C::QB * 2 * C::NB * per; x += THREADS)
            *reinterpret_cast<uint4*>(sm + C::Q_OFF + (x / per) * C::BLK + used * 128 +
                                      (x % per) * 16) = make_uint4(0, 0, 0, 0);
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
    pdl_wait();
    const int nu = KB >> p.unit_shift;
    // the next item of this warp's walk; false at the end (or when a wait gave up)
    auto next_item = [&](int k, Item& it) {
        if (!warp_wait(&b_item[k % ITEMS], (k / ITEMS) & 1, abort_f, p.status)) return false;
        const Item& x = items[k % ITEMS];
        it.grp = uniform(x.grp);
        it.q0 = uniform(x.q0);
        it.n = uniform(x.n);
        it.k0 = uniform(x.k0);
        it.len = uniform(x.len);
        it.t0 = uniform(x.t0);
        it.both = uniform(x.both);
        it.own[0] = uniform(x.own[0]);
        it.own[1] = uniform(x.own[1]);
        it.tail = uniform(x.tail);
        it.tail_end = uniform(x.tail_end);
        it.tail_step = uniform(x.tail_step);
        it.tail_tile = uniform(x.tail_tile);
        it.id = uniform(x.id);
        return it.grp >= 0;
    };
    auto done_item = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_iteme[k % ITEMS]);
    };
    auto records = [&](const Item& it) { return p.recs + (int64_t)it.id * p.max_rec * p.rec_words; };
    // the units of tile t's step i, one a lane (none behind the last)
    auto units = [&](const uint32_t* recs, const Item& it, int t, int i) {
        return i < it.steps(t) && lane < nu ? recs[(int64_t)it.record(t, i) * p.rec_words + lane]
                                            : ROW;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
        if (warp == 0) {
            uint32_t n = 0, nq = 0;
            bool ok = true;
            Item it;
            for (int k = 0; ok && next_item(k, it); k++) {
                const int steps = it.steps();
                if (steps > 0) {
                    const int head0 = it.grp * p.G, kvh = it.grp / p.subs, qb = nq % C::QB;
                    const uint32_t* recs = records(it);
                    // the tiles' units of this step, the next and the one after that
                    uint32_t now[2], next[2], ahead[2];
#pragma unroll
                    for (int t = 0; t < 2; t++) {
                        now[t] = ROW;
                        next[t] = units(recs, it, t, 0);
                        ahead[t] = units(recs, it, t, 1);
                    }
                    if (nq >= C::QB)
                        ok = warp_wait(&b_qe[qb], ((nq / C::QB) - 1) & 1, abort_f, p.status);
                    if (ok) {
                        if (lane == 0) {
                            uint32_t q_tiles = 0;
#pragma unroll
                            for (int t = 0; t < 2; t++) q_tiles += it.steps(t) > 0;
                            mbar_arrive_expect_tx(&b_q[qb], q_tiles * C::NB * (uint32_t)used * 128);
#pragma unroll
                            for (int t = 0; t < 2; t++)
                                if (it.steps(t) > 0)
                                    for (int x = 0; x < C::NB; x++)
                                        tma_load_3d(sbase + C::Q_OFF + (2 * qb + t) * C::TILE +
                                                        x * C::BLK,
                                                    &map_q, 64 * x, head0,
                                                    it.q0 + it.t0 + t * p.TT, &b_q[qb]);
                        }
                        nq++;
                    }
                    // lane l copies unit l % nu, columns 64 (l / nu) ..
                    const int slot = lane % nu, x = lane / nu;
                    auto load = [&](uint32_t unit, const CUtensorMap* map) {
                        const uint32_t word = __shfl_sync(0xffffffffu, unit, slot);
                        // (behind the last unit: rows that do not exist, read as zeros)
                        const int row = word == ROW ? (int)p.Tk : it.k0 + (int)word;
                        const uint32_t st = n % C::STAGES, use = n / C::STAGES;
                        if (use > 0)
                            ok = ok && warp_wait(&b_empty[st], (use - 1) & 1, abort_f, p.status);
                        if (!ok) return;
                        if (lane == 0) mbar_arrive_expect_tx(&b_full[st], C::TILE);
                        __syncwarp();
                        if (x < C::NB)
                            tma_load_3d(sbase + C::KV_OFF + st * C::TILE + x * C::BLK +
                                            ((slot << p.unit_shift) * 128),
                                        map, 64 * x, kvh, row, &b_full[st]);
                        n++;
                    };
                    // in the order in which the products want them (step -1: the first keys)
                    for (int i = -1; i < steps && ok; i++) {
#pragma unroll
                        for (int t = 0; t < 2; t++) {
                            if (i >= 0 && i < it.steps(t) && (t == 0 || i >= it.both))
                                load(now[t], &map_v);
                            if (i + 1 < it.steps(t) && (t == 0 || i + 1 >= it.both))
                                load(next[t], &map_k);
                        }
#pragma unroll
                        for (int t = 0; t < 2; t++) {
                            now[t] = next[t];
                            next[t] = ahead[t];
                            ahead[t] = units(recs, it, t, i + 3);
                        }
                    }
                }
                done_item(k);
            }
            // everything that was started lands before the CTA ends
            __syncwarp();
            if (lane == 0) {
                for (uint32_t x = nq > C::QB ? nq - C::QB : 0; x < nq; x++)
                    drain_bar(&b_q[x % C::QB], (x / C::QB) & 1, p.status);
                for (uint32_t x = n > C::STAGES ? n - C::STAGES : 0; x < n; x++)
                    drain_bar(&b_full[x % C::STAGES], (x / C::STAGES) & 1, p.status);
            }
        } else if (warp == 1) {
            constexpr uint32_t IDESC_S = idesc_bf16(128, KB, 0, 0);
            constexpr uint32_t IDESC_O = idesc_bf16(128, D, 0, 1);
            const uint32_t kd = desc_lo(sbase + C::KV_OFF, 16);
            const uint32_t vd = desc_lo(sbase + C::KV_OFF, C::BLK);
            uint32_t n = 0, nq = 0, tails = 0, done_p[2] = {0, 0}, outs[2] = {0, 0};
            auto wait_stage = [&](uint32_t n) {
                const bool r =
                    warp_wait(&b_full[n % C::STAGES], (n / C::STAGES) & 1, abort_f, p.status);
                tc_fence_after();
                return r;
            };
            auto stage_off = [&](uint32_t n) { return ((n % C::STAGES) * C::TILE) >> 4; };
            bool ok = true;
            Item it;
            for (int k = 0; ok && next_item(k, it); k++) {
                const int both = it.both, own0 = it.own[0], own1 = it.own[1];
                if (both + own0 + own1 > 0) {
                    const int qb = nq % C::QB;
                    const uint32_t qd = desc_lo(sbase + C::Q_OFF + 2 * qb * C::TILE, 16);
                    ok = warp_wait(&b_q[qb], (nq / C::QB) & 1, abort_f, p.status);
                    nq++;
                    // Tile t's scores on stage k.  (free: nobody else reads the stage)
                    auto scores = [&](int t, uint32_t k, bool free) {
                        mma_scores<D, IDESC_S>(tmem + TM_S + 128 * t, qd + ((t * C::TILE) >> 4),
                                               kd + stage_off(k));
                        tc_commit(&b_s[t]);
                        if (free) tc_commit(&b_empty[k % C::STAGES]);
                    };
                    // Tile t's step i: the output on stage v (if mine), then the next scores on
                    // stage k (if then).
                    // (late: nobody has waited for that stage yet)
                    auto step = [&](int t, int i, bool mine, uint32_t v, bool free_v, bool last,
                                    bool then, uint32_t k, bool free_k, bool end, bool late) {
                        if (ok && mine && it.tail > 0 && i == it.tail_step && t == it.tail_tile) {
                            if (lane == 0) {
                                *tail_stage = v % C::STAGES;
                                mbar_arrive(b_tail);
                            }
                            ok = warp_wait(b_fix, tails & 1, abort_f, p.status);
                            tails++;
                            tc_fence_after();
                        }
                        if (ok && mine) {
                            // the last item's outputs have been read
                            if (i == 0 && outs[t] > 0)
                                ok = warp_wait(&b_oe[t], (outs[t] - 1) & 1, abort_f, p.status);
                            ok = ok && warp_wait(&b_p[t], done_p[t] & 1, abort_f, p.status);
                            done_p[t]++;
                            tc_fence_after();
                        }
                        if (ok && elect_one()) {
                            if (mine) {
                                mma_output<D, IDESC_O>(tmem + TM_O + 128 * t, tmem + TM_S + 128 * t,
                                                       vd + stage_off(v), i > 0);
                                if (last) tc_commit(&b_o[t]);
                                if (free_v) tc_commit(&b_empty[v % C::STAGES]);
                            }
                        }
                        __syncwarp();
                        if (ok && late && then) ok = wait_stage(k);
                        if (ok && elect_one()) {
                            if (then) scores(t, k, free_k);
                            if (end) tc_commit(&b_qe[qb]);  // the last scores
                        }
                        __syncwarp();
                        if (mine && last) outs[t]++;
                    };
                    // the first scores
                    const bool any0 = own0 > 0, any1 = own1 > 0;
                    if (both > 0) {
                        ok = ok && wait_stage(n);
                        if (ok && elect_one()) {
                            scores(0, n, false);
                            scores(1, n, true);
                        }
                    } else {
                        ok = ok && (!any0 || wait_stage(n)) && (!any1 || wait_stage(n + any0));
                        if (ok && elect_one()) {
                            if (any0) scores(0, n, true);
                            if (any1) scores(1, n + any0, true);
                        }
                    }
                    const int steps = it.steps();
                    if (ok && steps == 1 && elect_one()) tc_commit(&b_qe[qb]);
                    __syncwarp();
                    // (stages are waited for before the weights: nothing stands between their
                    // arrival and the products.  Their numbers follow from the step's.)
                    for (int i = 0; i < both && ok; i++) {
                        const bool more = i + 1 < both;
                        const uint32_t v = n + 2 * i + 1, k0 = v + 1, k1 = more ? k0 : k0 + any0;
                        ok = wait_stage(v) && (!(more || any0) || wait_stage(k0)) &&
                             (more || !any1 || wait_stage(k1));
                        step(0, i, true, v, false, !more && !any0, more || any0, k0, !more, false,
                             false);
                        step(1, i, true, v, true, !more && !any1, more || any1, k1, true,
                             i + 2 == steps, false);
                    }
                    n += 2 * both + any0 + any1;
                    for (int m = 0; m + both < steps && ok; m++) {
                        const bool a0 = m < own0, c0 = m + 1 < own0;
                        const bool a1 = m < own1, c1 = m + 1 < own1;
                        const uint32_t k0 = n + a0, v1 = k0 + c0, k1 = v1 + a1;
                        const int i = both + m;
                        ok = !a0 || wait_stage(n);
                        step(0, i, a0, n, true, !c0, c0, k0, true, false, true);
                        ok = ok && (!a1 || wait_stage(v1));
                        step(1, i, a1, v1, true, !c1, c1, k1, true, i + 2 == steps, true);
                        n = k1 + c1;
                    }
                }
                done_item(k);
            }
        } else if (warp == 2) {
            // zero the V rows behind the last key
            uint32_t tails = 0;
            bool ok = true;
            Item it;
            for (int k = 0; ok && next_item(k, it); k++) {
                if (it.tail > 0) {
                    ok = warp_wait(b_tail, tails & 1, abort_f, p.status);
                    tails++;
                    if (!ok) break;
                    uint8_t* v = sm + C::KV_OFF + (uint32_t)uniform((int)*tail_stage) * C::TILE;
                    for (int x = lane; x < (it.tail_end - it.tail) * C::NB * 8; x += 32) {
                        const int r = it.tail + x / (C::NB * 8), piece = x % (C::NB * 8);
                        *reinterpret_cast<uint4*>(v + (piece / 8) * C::BLK + r * 128 +
                                                  (piece % 8) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                    __syncwarp();
                    if (lane == 0) mbar_arrive(b_fix);
                }
                done_item(k);
            }
        } else {
            // the items: this CTA's own, then those that it takes over
            const uint32_t response = sbase + C::BAR_OFF + 640 - 16;
            int id = blockIdx.x;
            bool ok = true;
            for (int k = 0, asked = 0; ok && id >= 0;) {
                if (lane == 0) take_over(response, b_clc);
                int4 piece = make_int4(-1, 0, 0, 0);
                if (lane < 4) piece = reinterpret_cast<const int4*>(p.items + id)[lane];
                if (uniform(piece.x) >= 0) {  // (grp, of lane 0's piece)
                    if (k >= ITEMS)
                        ok = warp_wait(&b_iteme[k % ITEMS], ((k / ITEMS) - 1) & 1, abort_f,
                                       p.status);
                    if (ok && lane < 4) {
                        int* to = reinterpret_cast<int*>(&items[k % ITEMS]) + 4 * lane;
                        to[0] = piece.x;
                        to[1] = piece.y;
                        to[2] = piece.z;
                        to[3] = piece.w;
                    }
                    __syncwarp();
                    if (ok && lane == 0) mbar_arrive(&b_item[k % ITEMS]);
                    k++;
                }
                // (an answer that is on its way is waited for in any case)
                const bool here = __all_sync(
                    0xffffffffu, drain_bar(b_clc, asked & 1, p.status));
                asked++;
                id = here ? taken_over(response) : -1;
                __syncwarp();
                if (id < 0 || !ok) {
                    if (ok && k >= ITEMS)
                        ok = warp_wait(&b_iteme[k % ITEMS], ((k / ITEMS) - 1) & 1, abort_f,
                                       p.status);
                    if (lane == 0) {
                        items[k % ITEMS].grp = -1;
                        mbar_arrive(&b_item[k % ITEMS]);
                    }
                    break;
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;\n");
        const int t = (warp - 4) >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tm_s = tmem + lanes + TM_S + 128 * t, tm_o = tmem + lanes + TM_O + 128 * t;
        const int row = 32 * (warp & 3) + lane;
        const int tok = row / p.G, gh = row - tok * p.G;
        const float c = p.c;
        uint32_t ph = 0, outs = 0;
        bool ok = true;
        Item it;
        for (int k = 0; ok && next_item(k, it); k++) {
            const int count = max(0, min(p.TT, it.n - it.t0 - t * p.TT));  // tokens of the tile
            const bool live = tok < count;
            const bool idle = !__any_sync(0xffffffffu, live);
            const int steps = it.steps(t);
            const int pos = it.len - it.n + it.t0 + t * p.TT + tok;  // the last key it sees
            const int bit = live ? t * p.TT + tok : 0;
            // Step i's record, a word a lane (a step ahead; longer ones are read when wanted).
            const bool held = p.rec_words <= 32;
            auto fetch = [&](int i) {
                return held && i < steps && lane < p.rec_words
                           ? records(it)[(int64_t)it.record(t, i) * p.rec_words + lane]
                           : 0u;
            };
            // The row's view of it: the keys of the units that its token lists, up to its place.
            auto look = [&](int i, uint32_t word, uint32_t (&vis)[4]) {
                const uint32_t* rec = records(it) + (int64_t)it.record(t, i) * p.rec_words;
                auto at = [&](int x) { return held ? __shfl_sync(0xffffffffu, word, x) : rec[x]; };
                auto keys = [&](int unit, int off) {  // of a unit from key off on
                    const uint32_t mask = at(nu + unit * p.words + (bit >> 5));
                    const int n = pos - (int)at(unit) - off + 1;
                    return low_bits(live && ((mask >> (bit & 31)) & 1) ? n : 0);
                };
                if (p.unit_shift >= 5) {
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        const int unit = (32 * x) >> p.unit_shift;
                        vis[x] = keys(unit, 32 * x - (unit << p.unit_shift));
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < 4; x++)
                        vis[x] = (keys(2 * x, 0) & 0xffffu) | keys(2 * x + 1, 0) << 16;
                }
            };
            uint32_t word = fetch(0);
            RowState st;
            for (int i = 0; i < steps; i++) {
                uint32_t vis[4];
                look(i, word, vis);
                word = fetch(i + 1);
                const bool parts = __any_sync(  // (a word that is neither 0 nor all ones)
                    0xffffffffu, vis[0] + 1 > 1 || vis[1] + 1 > 1 || vis[2] + 1 > 1 ||
                                     vis[3] + 1 > 1);
                ok = warp_wait(&b_s[t], ph & 1, abort_f, p.status);
                if (!ok) break;
                ph++;
                tc_fence_after();
                // (where none of the warp's rows exists, whatever its scores hold weighs no one)
                if (!idle) softmax_words<D>(tm_s, tm_o, i > 0, vis, parts, c, live, st);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_p[t]);
            }
            if (!ok) break;
            // the sink is one more term of the denominator
            const int head = it.grp * p.G + gh;
            const RowEnd end = row_end(st.reference(c), st.l,
                                       live && p.sink ? p.sink[head] : -INFINITY);
            const int64_t at = (int64_t)(it.q0 + it.t0 + t * p.TT + tok) * p.nh + head;
            if (live && p.lse) p.lse[at] = end.lse;
            if (count > 0) {
                const bool any = steps > 0;
                if (any) {
                    ok = warp_wait(&b_o[t], outs & 1, abort_f, p.status);
                    if (!ok) break;
                    outs++;
                    tc_fence_after();
                }
                // (offsets from the tile's first row: at most 128 tokens of 4096 heads)
                uint16_t* dst = p.o + (int64_t)(it.q0 + it.t0 + t * p.TT) * p.nh * p.hd;
                store_rows<D>(tm_o, any, end.factor, dst,
                              live ? (tok * p.nh + head) * p.hd : -1, p.hd, [&] {
                                  tc_fence_before();
                                  __syncwarp();
                                  if (any && lane == 0) mbar_arrive(&b_oe[t]);
                              });
            }
            done_item(k);
        }
    }

    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        // The softmax warps have seen every output complete, unless a wait gave up: then what
        // this warp issued may still be running.
        if (*abort_f) {
            if (elect_one()) tc_commit(b_end);
            __syncwarp();
            drain_bar(b_end, 0, p.status);
        }
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem)
                     : "memory");
    }
}

// The shape of a call's work and its scratch.
struct Plan {
    int G, TT, subs, words, unit_shift, rec_words, max_rec;
    int64_t items;
    size_t items_bytes, recs_bytes;
    size_t bytes() const { return items_bytes + recs_bytes; }
};
Plan make_plan(int64_t B, int64_t Tq, int64_t max_q, int64_t max_k, int64_t topk, int64_t block,
               int64_t nh, int64_t kvh) {
    Plan pl;
    pl.G = heads_of_tile(nh / kvh, &pl.subs);
    pl.TT = ROWS / pl.G;
    pl.words = (2 * pl.TT + 31) / 32;
    const int64_t unit = block < KB ? block : KB;
    pl.unit_shift = 0;
    while ((1 << pl.unit_shift) < unit) pl.unit_shift++;
    const int64_t nu = KB / unit;
    pl.rec_words = (int)(nu * (1 + pl.words));
    // blocks of an item: as many as there are, or as its tokens can list
    const int64_t toks = 2 * pl.TT < max_q ? 2 * pl.TT : max_q;
    int64_t blocks = (max_k + block - 1) / block;
    if (toks * topk < blocks) blocks = toks * topk;
    // (three kinds of them, each with a record that is not full; units of both tiles that move to
    // the tiles' own records free one, and the shorter of those may need one more)
    pl.max_rec = (int)((blocks * (block / unit) + nu - 1) / nu) + 2;
    // every sequence has at most one pair of tiles that is not full
    pl.items = (Tq / (2 * pl.TT) + B) * kvh * pl.subs;
    pl.items_bytes = (size_t)pl.items * sizeof(Item);
    pl.recs_bytes = (size_t)pl.items * pl.max_rec * pl.rec_words * 4;
    return pl;
}

int check_sizes(const char* name, int64_t B, int64_t Tq, int64_t max_q, int64_t max_k, int64_t topk,
                int64_t block) {
    const int64_t lim = int64_t(1) << 31;
    DS41_REQUIRE(block >= 16 && block <= 256 && (block & (block - 1)) == 0, DS41_E_ARG,
                 "%s: blocks of %lld rows (a power of two of 16 .. 256)", name, (long long)block);
    DS41_REQUIRE(topk >= 1 && topk <= 1024, DS41_E_ARG, "%s: topk=%lld (1 .. 1024)", name,
                 (long long)topk);
    DS41_REQUIRE(B >= 0 && B < 65536 && Tq >= 0 && Tq < lim && max_q >= 0 && max_q < lim &&
                     max_k >= 0 && max_k <= 32768 * block,
                 DS41_E_RANGE, "%s: B=%lld Tq=%lld max_q=%lld max_k=%lld (at most 32768 blocks)",
                 name, (long long)B, (long long)Tq, (long long)max_q, (long long)max_k);
    return DS41_OK;
}

}  // namespace bp
}  // namespace ds41

using namespace ds41;

extern "C" size_t ds41_block_prompt_attn_workspace_bytes(int64_t B, int64_t Tq, int64_t max_q,
                                                         int64_t max_k, int64_t topk,
                                                         int64_t block, int64_t nh, int64_t kvh) {
    const char* name = "ds41_block_prompt_attn_workspace_bytes";
    if (check_heads(name, nh, kvh, 16, 1.0f, 0) ||
        bp::check_sizes(name, B, Tq, max_q, max_k, topk, block) || B == 0 || Tq == 0 || max_q == 0)
        return 0;
    return bp::make_plan(B, Tq, max_q, max_k, topk, block, nh, kvh).bytes();
}

extern "C" int ds41_block_prompt_attn_fwd(const ds41_bf16* q, int64_t q_tok, int64_t q_head,
                                          const ds41_bf16* k, int64_t k_tok, int64_t k_head,
                                          const ds41_bf16* v, int64_t v_tok, int64_t v_head,
                                          const int32_t* cu_q, const int32_t* cu_k,
                                          const int32_t* idx, int64_t topk, int64_t block,
                                          int64_t B, int64_t Tq, int64_t Tk, int64_t max_q,
                                          int64_t max_k, int64_t nh, int64_t kvh, int64_t hd,
                                          float scale, const float* sink, ds41_bf16* o, float* lse,
                                          void* ws, size_t ws_bytes, ds41_stream_t stream) {
    const char* name = "ds41_block_prompt_attn_fwd";
    if (int rc = check_heads(name, nh, kvh, hd, scale, 0)) return rc;
    if (int rc = bp::check_sizes(name, B, Tq, max_q, max_k, topk, block)) return rc;
    const int64_t lim = int64_t(1) << 31;
    DS41_REQUIRE(Tk >= 0 && Tk < lim, DS41_E_RANGE, "%s: Tk=%lld", name, (long long)Tk);
    if (B == 0 || Tq == 0 || max_q == 0) return DS41_OK;
    DS41_REQUIRE(q && o && cu_q && cu_k && idx && (Tk == 0 || (k && v)), DS41_E_ARG,
                 "%s: q, k, v, cu_q, cu_k, idx and o must be non-null", name);
    DS41_REQUIRE(aligned16(q) && aligned16(k) && aligned16(v) && aligned16(o) &&
                     aligned_to(cu_q, 4) && aligned_to(cu_k, 4) && aligned_to(idx, 4) &&
                     aligned_to(sink, 4) && aligned_to(lse, 4),
                 DS41_E_ARG, "%s: q, k, v and o must be 16-byte aligned", name);
    DS41_REQUIRE(good_strides(q_tok, q_head, hd) &&
                     (Tk == 0 ||
                      (good_strides(k_tok, k_head, hd) && good_strides(v_tok, v_head, hd))),
                 DS41_E_ARG, "%s: strides must be multiples of 8 and at least hd", name);
    const bp::Plan pl = bp::make_plan(B, Tq, max_q, max_k, topk, block, nh, kvh);
    DS41_REQUIRE(pl.items < lim, DS41_E_RANGE, "%s: Tq=%lld B=%lld kvh=%lld", name, (long long)Tq,
                 (long long)B, (long long)kvh);
    DS41_REQUIRE(ws && aligned16(ws) && ws_bytes >= pl.bytes(), DS41_E_WORKSPACE,
                 "%s: needs %zu bytes of workspace, got %zu", name, pl.bytes(), ws ? ws_bytes : 0);
    bp::Params p{};
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.idx = idx;
    p.sink = sink;
    p.o = o;
    p.lse = lse;
    p.Tq = Tq;
    p.Tk = Tk;
    p.B = (int)B;
    p.max_q = (int)max_q;
    p.max_k = (int)max_k;
    p.nh = (int)nh;
    p.kvh = (int)kvh;
    p.hd = (int)hd;
    p.topk = (int)topk;
    p.G = pl.G;
    p.TT = pl.TT;
    p.subs = pl.subs;
    p.pairs = (int)(pl.items / (kvh * pl.subs));
    while ((1 << p.shift) < block) p.shift++;
    p.unit_shift = pl.unit_shift;
    p.words = pl.words;
    p.rec_words = pl.rec_words;
    p.max_rec = pl.max_rec;
    p.c = scale * tc::SM_LOG2E;
    p.items = static_cast<bp::Item*>(ws);
    p.recs = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + pl.items_bytes);
    if (int rc = status_word(&p.status)) return rc;
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    if (int rc = tc::get_encode(&enc)) return rc;
    CUtensorMap mq, mk, mv;
    const int unit = 1 << pl.unit_shift;
    if (int rc = pa::make_map_heads(enc, &mq, q, Tq, nh, hd, q_tok, q_head, pl.G, pl.TT)) return rc;
    if (Tk > 0) {
        if (int rc = pa::make_map_heads(enc, &mk, k, Tk, kvh, hd, k_tok, k_head, 1, unit)) return rc;
        if (int rc = pa::make_map_heads(enc, &mv, v, Tk, kvh, hd, v_tok, v_head, 1, unit)) return rc;
    } else {
        mk = mv = mq;  // never read
    }
    cudaStream_t st = (cudaStream_t)stream;
    const dim3 grid((unsigned)pl.items);
    // (no larger than the blocks need: more CTAs fit an SM)
    const int64_t words = ((max_k + block - 1) / block) * pl.words;
    p.table = (int)(words < bp::TABLE ? (words > 0 ? words : pl.words) : bp::TABLE);
    if (int rc = launch_pdl(bp::plan_kernel, grid, dim3(bp::PLAN), (size_t)p.table * 4, st, name, p))
        return rc;
    auto kern = hd <= 64 ? bp::block_prompt_kernel<64> : bp::block_prompt_kernel<128>;
    const size_t smem = hd <= 64 ? pa::Cfg<64>::SMEM : pa::Cfg<128>::SMEM;
    if (int rc = hd <= 64 ? allow_smem<bp::block_prompt_kernel<64>>((int)smem, name)
                          : allow_smem<bp::block_prompt_kernel<128>>((int)smem, name))
        return rc;
    return launch_pdl(kern, grid, dim3(pa::THREADS), smem, st, name, mq, mk, mv, p);
}
