// ds41_prompt_attn.cu - causal attention over packed prompts with grouped
// heads, on the 5th-generation tensor cores.
//
// Mathematics.  Per query row and key block of 128, in units of log2 with
// c = scale log2(e):
//   S = q K^T,  p_j = 2^(c S_j - c m),  l += sum p_j,  O += p V
// with a reference m that follows the running maximum of the row; whenever m
// moves from m0 to m1, l and O are scaled by 2^(c (m0 - m1)).  At the end
// o = O / (l + 2^(sink - c m)).  m need not be the exact maximum, only close
// enough that nothing overflows: it moves when a block exceeds it by 2^8, so O
// is rescaled on the first blocks of a row, if at all.
//
// Rows.  The query heads that share a key/value head see the same keys, so a
// tile of 128 rows is TT tokens times the G heads of a group (row = token * G +
// head; G = 4: 32 tokens), and a CTA holds two such tiles over one stream of
// key/value blocks.
//
// Design.  One persistent CTA per SM walks its items (a pair of tiles of one head
// group), warp-specialised: warp 0 issues the TMA copies (an item's two query
// tiles, then its K and V blocks through a ring of stages), warp 1 issues the
// MMAs, warp 3 looks the items up some ahead, warps 4..7 and 8..11 compute the
// softmax of tile 0 and of tile 1, a thread per row, and write the outputs.  No
// role waits for another at an item's end: the next item's queries and keys
// arrive and its first scores are computed while the last one's outputs are
// written.  S_t (128 columns of f32) and O_t live in tensor
// memory; the weights go back as bf16 into the columns of S_t and are the A
// operand of the second product from there, so neither S nor P touches shared
// memory.  Issue order PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1): while the softmax of
// one tile runs, the tensor core works on the other.  A commit after QK_t(j+1)
// also covers PV_t(j), so a softmax thread that has seen S_t(j+1) may rescale
// its row of O_t itself: no fourth role, no further barrier.
//
// What bounds it.  Long prompts: the products.  A pair of blocks takes 2700 cycles
// where the tensor core's rate alone would allow 2048, as 128 x 128 products with
// both operands in shared memory read it at its full rate (16384 tokens of 32 heads
// of 128 over 8: 1.32 ms, 1660 TFLOP/s).  Short ones: the ends of the items, where
// the tensor core waits for first scores and last outputs (seven prompts of 415 ..
// 2000 tokens: 150 us, 9 items a CTA); with a window, whose items are two blocks
// long, one chain of scores, softmax, product and output (chunks of 4096 and 1440
// tokens, window 128, 64 heads of 64 over 8: 60 us).
#include "ds41_dense.cuh"
#include "ds41_softmax_tc.cuh"

namespace ds41 {
namespace pa {

using namespace tc;

constexpr int KB = 128;         // keys per block
constexpr int ROWS = 128;       // rows per tile
constexpr int THREADS = 384;

template <int D>
struct Cfg {
    static constexpr int NB = D / 64;                   // 64-column blocks of a row
    static constexpr uint32_t BLK = 128 * 128;          // [128 rows][64 columns] bf16
    static constexpr uint32_t TILE = NB * BLK;          // a query tile, or a K or V block
    static constexpr int STAGES = D == 128 ? 5 : 9;
    static constexpr int QB = D == 128 ? 1 : 2;         // items whose queries are held
    static constexpr uint32_t Q_OFF = 0;                // two query tiles each
    static constexpr uint32_t KV_OFF = QB * 2 * TILE;
    static constexpr uint32_t BAR_OFF = KV_OFF + STAGES * TILE;
    static constexpr uint32_t SMEM = BAR_OFF + 640 + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
};

// tensor memory columns: S_0 S_1 O_0 O_1
constexpr uint32_t TM_S = 0, TM_O = 256;

struct Params {
    const int32_t* cu_q;
    const int32_t* cu_k;
    const float* sink;
    uint16_t* o;
    float* lse;
    int64_t Tq, Tk, window;
    int B, max_q, nh, hd;
    int G;        // heads of a tile
    int TT;       // tokens of a tile
    int n_groups; // key/value heads times tiles' head groups per key/value head
    int subs;     // head groups per key/value head
    float c;      // scale * log2(e)
    unsigned int* status;
};

// An item: one head group of one pair of tiles of one sequence.
struct Item {
    int grp;        // head group, -1: no more items
    int q0, n;      // its sequence's queries
    int k0, len;    // and keys
    int t0;         // first token of tile 0
};
constexpr int ITEMS = 4;  // items looked up ahead

// the lowest n bits (none for n <= 0, all for n >= 32)
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// The key blocks [lo, hi) that some row of tile t sees; count = its tokens.
struct Range {
    int lo, hi, count, p_first;
};
__device__ __forceinline__ Range tile_range(const Item& it, const Params& p, int t) {
    Range r;
    const int first = it.t0 + t * p.TT;
    r.count = max(0, min(p.TT, it.n - first));
    r.p_first = first + it.len - it.n;
    r.lo = r.hi = 0;
    if (r.count > 0) {
        const int64_t last = r.p_first + (int64_t)r.count - 1;
        if (last >= 0) {
            r.hi = (int)(last / KB) + 1;
            const int64_t lo = p.window ? max((int64_t)0, r.p_first - p.window + 1) : 0;
            r.lo = (int)(lo / KB);
        }
    }
    return r;
}

// A CTA that is through with an item takes over one whose CTA has not started yet:
// the grid has a CTA for every item, and the launch queue is the list of what is
// left, longest first, so the SMs end together (items dealt out beforehand left
// one of them 7% more blocks than the average of a 16384-token prompt).
__device__ __forceinline__ void take_over(uint32_t response, uint64_t* bar) {
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    mbar_arrive_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
        "[%0], [%1];\n" ::"r"(response),
        "r"(smem_u32(bar))
        : "memory");
}
// the answer: the CTA's index, or -1: all have started
__device__ __forceinline__ int taken_over(uint32_t response) {
    uint32_t got, x;
    asm volatile(
        "{\n.reg .pred p;\n.reg .b128 r;\nld.shared.b128 r, [%2];\n"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
        "selp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
        : "=r"(got), "=r"(x)
        : "r"(response)
        : "memory");
    return got ? (int)x : -1;
}

// Walks the sequences, 32 at a time (a whole warp): flat index w -> sequence and
// pair of tiles (indices mostly rise from call to call; one that does not starts
// over).  A sequence that breaks its limits has no tiles.  The tiles of a sequence
// come in falling order: the longest first.
struct Finder {
    int b0 = -32, base = 0, end = 0;  // sequences b0 .. b0 + 31 have pairs base .. end - 1
    int q0, n, k0, len, tiles, sum;   // this lane's sequence; sum: inclusive prefix of tiles
    __device__ __forceinline__ bool find(const Params& p, int w, bool report, int lane, Item& it) {
        if (w < base) {
            b0 = -32;
            base = end = 0;
        }
        while (w >= end) {
            b0 += 32;
            if (b0 >= p.B) {
                b0 -= 32;
                return false;
            }
            const int b = b0 + lane;
            q0 = n = k0 = len = tiles = 0;
            if (b < p.B) {
                q0 = p.cu_q[b];
                k0 = p.cu_k[b];
                const int64_t ln = (int64_t)p.cu_q[b + 1] - q0, lk = (int64_t)p.cu_k[b + 1] - k0;
                if (q0 >= 0 && ln >= 0 && ln <= p.max_q && q0 + ln <= p.Tq && k0 >= 0 && lk >= 0 &&
                    k0 + lk <= p.Tk) {
                    n = (int)ln;
                    len = (int)lk;
                    tiles = (n + 2 * p.TT - 1) / (2 * p.TT);
                } else if (report) {
                    raise_status(p.status, DS41_E_INDEX);
                }
            }
            sum = tiles;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, off);
                if (lane >= off) sum += v;
            }
            base = end;
            end = base + __shfl_sync(0xffffffffu, sum, 31);
        }
        const unsigned mine =
            __ballot_sync(0xffffffffu, w >= base + sum - tiles && w < base + sum);
        const int src = __ffs(mine) - 1;
        it.q0 = __shfl_sync(0xffffffffu, q0, src);
        it.n = __shfl_sync(0xffffffffu, n, src);
        it.k0 = __shfl_sync(0xffffffffu, k0, src);
        it.len = __shfl_sync(0xffffffffu, len, src);
        it.t0 = (base + __shfl_sync(0xffffffffu, sum, src) - 1 - w) * 2 * p.TT;
        return true;
    }
};

// What every role derives from an item: the tiles' key blocks, their union
// [jlo, jhi), and the keys of the last block when it is not full (the rest of its
// V rows belong to another sequence, or to nobody).
struct Span {
    Range rg[2];
    int jlo, jhi, tail;
    __device__ __forceinline__ Span(const Item& it, const Params& p)
        : rg{tile_range(it, p, 0), tile_range(it, p, 1)} {
        jlo = rg[0].lo;
        jhi = rg[0].hi;
        if (rg[1].hi > rg[1].lo) {
            jlo = rg[0].hi > rg[0].lo ? min(jlo, rg[1].lo) : rg[1].lo;
            jhi = max(jhi, rg[1].hi);
        }
        tail = jhi * KB > it.len ? it.len - (jhi - 1) * KB : 0;
    }
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap map_q,
                       const __grid_constant__ CUtensorMap map_k,
                       const __grid_constant__ CUtensorMap map_v, const Params p) {
    pdl_wait();
    using C = Cfg<D>;
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
    Item* items = reinterpret_cast<Item*>(tmem_slot + 2);
    static_assert((2 * C::QB + 2 * C::STAGES + 12 + 2 * ITEMS) * 8 + 8 + ITEMS * sizeof(Item) <=
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
        return it.grp >= 0;
    };
    auto done_item = [&](int k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&b_iteme[k % ITEMS]);
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;\n");
        if (warp == 0) {
            uint32_t n = 0, nq = 0;
            bool ok = true;
            Item it;
            for (int k = 0; ok && next_item(k, it); k++) {
                const Span sp(it, p);
                if (sp.jhi > sp.jlo && lane == 0) {
                    const int head0 = it.grp * p.G, kvh = it.grp / p.subs, qb = nq % C::QB;
                    if (nq >= C::QB)
                        ok = wait_bar(&b_qe[qb], ((nq / C::QB) - 1) & 1, abort_f, p.status);
                    if (ok) {
                        uint32_t q_tiles = 0;
                        for (int t = 0; t < 2; t++) q_tiles += sp.rg[t].hi > sp.rg[t].lo;
                        mbar_arrive_expect_tx(&b_q[qb], q_tiles * C::NB * (uint32_t)used * 128);
                        for (int t = 0; t < 2; t++)
                            if (sp.rg[t].hi > sp.rg[t].lo)
                                for (int x = 0; x < C::NB; x++)
                                    tma_load_3d(sbase + C::Q_OFF + (2 * qb + t) * C::TILE +
                                                    x * C::BLK,
                                                &map_q, 64 * x, head0, it.q0 + it.t0 + t * p.TT,
                                                &b_q[qb]);
                        nq++;
                    }
                    for (int j = sp.jlo; j < sp.jhi && ok; j++) {
                        for (int kv = 0; kv < 2 && ok; kv++) {
                            const uint32_t st = n % C::STAGES, use = n / C::STAGES;
                            if (use > 0)
                                ok = wait_bar(&b_empty[st], (use - 1) & 1, abort_f, p.status);
                            if (!ok) break;
                            mbar_arrive_expect_tx(&b_full[st], C::TILE);
                            for (int x = 0; x < C::NB; x++)
                                tma_load_3d(sbase + C::KV_OFF + st * C::TILE + x * C::BLK,
                                            kv ? &map_v : &map_k, 64 * x, kvh, it.k0 + j * KB,
                                            &b_full[st]);
                            n++;
                        }
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                done_item(k);
            }
            // everything that was started lands before the CTA ends
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
            uint32_t ring0 = 0, nq = 0, tails = 0, done_p[2] = {0, 0}, outs[2] = {0, 0};
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
                const Span sp(it, p);
                const int jlo = sp.jlo, jhi = sp.jhi;
                if (jhi > jlo) {
                    const int qb = nq % C::QB;
                    const uint32_t qd = desc_lo(sbase + C::Q_OFF + 2 * qb * C::TILE, 16);
                    ok = warp_wait(&b_q[qb], (nq / C::QB) & 1, abort_f, p.status) &&
                         wait_stage(ring0);
                    nq++;
                    if (ok && elect_one()) {
#pragma unroll
                        for (int t = 0; t < 2; t++)
                            if (jlo >= sp.rg[t].lo && jlo < sp.rg[t].hi) {
                                mma_scores<D, IDESC_S>(tmem + TM_S + 128 * t,
                                                       qd + ((t * C::TILE) >> 4),
                                                       kd + stage_off(ring0));
                                tc_commit(&b_s[t]);
                            }
                        tc_commit(&b_empty[ring0 % C::STAGES]);
                        if (jhi == jlo + 1) tc_commit(&b_qe[qb]);
                    }
                    __syncwarp();
                    for (int j = jlo; j < jhi && ok; j++) {
                        const uint32_t nv = ring0 + 2 * (uint32_t)(j - jlo) + 1, nk = nv + 1;
                        // (both before the waits for the weights: nothing stands between
                        // their arrival and the products)
                        ok = wait_stage(nv) && (j + 1 >= jhi || wait_stage(nk));
                        if (ok && j == jhi - 1 && sp.tail > 0) {
                            if (lane == 0) mbar_arrive(b_tail);
                            ok = warp_wait(b_fix, tails & 1, abort_f, p.status);
                            tails++;
                            tc_fence_after();
                        }
#pragma unroll
                        for (int t = 0; t < 2; t++) {
                            const bool now = j >= sp.rg[t].lo && j < sp.rg[t].hi;
                            const bool next = j + 1 >= sp.rg[t].lo && j + 1 < sp.rg[t].hi;
                            if (ok && now) {
                                // the last item's outputs have been read
                                if (j == sp.rg[t].lo && outs[t] > 0)
                                    ok = warp_wait(&b_oe[t], (outs[t] - 1) & 1, abort_f, p.status);
                                ok = ok && warp_wait(&b_p[t], done_p[t] & 1, abort_f, p.status);
                                done_p[t]++;
                                tc_fence_after();
                            }
                            if (ok && elect_one()) {
                                if (now) {
                                    mma_output<D, IDESC_O>(tmem + TM_O + 128 * t,
                                                           tmem + TM_S + 128 * t,
                                                           vd + stage_off(nv), j > sp.rg[t].lo);
                                    if (j + 1 == sp.rg[t].hi) tc_commit(&b_o[t]);
                                }
                                if (t == 1) tc_commit(&b_empty[nv % C::STAGES]);
                                if (next) {
                                    mma_scores<D, IDESC_S>(tmem + TM_S + 128 * t,
                                                           qd + ((t * C::TILE) >> 4),
                                                           kd + stage_off(nk));
                                    tc_commit(&b_s[t]);
                                }
                            }
                            __syncwarp();
                            if (now && j + 1 == sp.rg[t].hi) outs[t]++;
                        }
                        if (ok && j + 1 < jhi && elect_one()) {
                            tc_commit(&b_empty[nk % C::STAGES]);
                            if (j + 2 == jhi) tc_commit(&b_qe[qb]);  // the last scores
                        }
                        __syncwarp();
                    }
                    ring0 += 2 * (uint32_t)(jhi - jlo);
                }
                done_item(k);
            }
        } else if (warp == 2) {
            // zero the V rows behind the last key
            uint32_t ring0 = 0, tails = 0;
            bool ok = true;
            Item it;
            for (int k = 0; ok && next_item(k, it); k++) {
                const Span sp(it, p);
                if (sp.jhi > sp.jlo) {
                    ring0 += 2 * (uint32_t)(sp.jhi - sp.jlo);
                    if (sp.tail > 0) {
                        ok = warp_wait(b_tail, tails & 1, abort_f, p.status);
                        tails++;
                        if (!ok) break;
                        uint8_t* v = sm + C::KV_OFF + ((ring0 - 1) % C::STAGES) * C::TILE;
                        for (int x = lane; x < (KB - sp.tail) * C::NB * 8; x += 32) {
                            const int r = sp.tail + x / (C::NB * 8), piece = x % (C::NB * 8);
                            *reinterpret_cast<uint4*>(v + (piece / 8) * C::BLK + r * 128 +
                                                      (piece % 8) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(b_fix);
                    }
                }
                done_item(k);
            }
        } else {
            // the items: this CTA's own, then those that it takes over
            const uint32_t response = sbase + C::BAR_OFF + 640 - 16;
            Finder f;
            int id = blockIdx.x;
            bool ok = true;
            for (int k = 0, asked = 0; ok && id >= 0;) {
                if (lane == 0) take_over(response, b_clc);
                Item it;
                const int w = id / p.n_groups;
                if (f.find(p, w, false, lane, it)) {
                    it.grp = id - w * p.n_groups;
                    if (k >= ITEMS)
                        ok = warp_wait(&b_iteme[k % ITEMS], ((k / ITEMS) - 1) & 1, abort_f,
                                       p.status);
                    if (ok && lane == 0) {
                        items[k % ITEMS] = it;
                        mbar_arrive(&b_item[k % ITEMS]);
                    }
                    k++;
                }
                if (id == 0) {  // whoever has the first item reports the bad sequences
                    Finder all;
                    while (all.find(p, 0x7fffffff, true, lane, it)) {
                    }
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
            const Range r = tile_range(it, p, t);
            const bool live = tok < r.count;
            const bool idle = !__any_sync(0xffffffffu, live);
            const int64_t pos = (int64_t)r.p_first + tok;              // the last key it sees
            const int64_t before = p.window ? pos - p.window : -1;     // the last key before those
            const int64_t p_last = (int64_t)r.p_first + r.count - 1;
            RowState st;
            for (int j = r.lo; j < r.hi; j++, ph++) {
                ok = warp_wait(&b_s[t], ph & 1, abort_f, p.status);
                if (!ok) break;
                tc_fence_after();
                const int64_t j0 = (int64_t)j * KB;
                const bool masked =
                    j0 + KB - 1 > r.p_first || (p.window && j0 <= p_last - p.window);
                if (idle) {
                    // none of the warp's rows exists: whatever its scores hold weighs no one
                } else if (masked) {
                    const int hi = (int)max((int64_t)-1, min((int64_t)KB, pos - j0));
                    const int lo = (int)max((int64_t)-1, min((int64_t)KB, before - j0));
                    uint32_t vis[4];
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        vis[i] = low_bits(hi + 1 - 32 * i) & ~low_bits(lo + 1 - 32 * i);
                    softmax_block<D, true>(tm_s, tm_o, j > r.lo, vis, c, live, st);
                } else {
                    const uint32_t all[4] = {};
                    softmax_block<D, false>(tm_s, tm_o, j > r.lo, all, c, live, st);
                }
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
            if (r.count > 0) {
                const bool any = r.hi > r.lo;
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

// [tokens][heads][hd] with strides in elements; a box of 64 columns x box_h
// heads x box_t tokens, 128-byte swizzle, zeros outside.
int make_map_heads(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* ptr,
                   int64_t tokens, int64_t heads, int64_t hd, int64_t tok, int64_t head, int box_h,
                   int box_t) {
    cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)tok * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)box_h, (cuuint32_t)box_t};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(DS41_E_CUDA, "cuTensorMapEncodeTiled (heads) failed (%d)", (int)r);
    return DS41_OK;
}

}  // namespace pa
}  // namespace ds41

using namespace ds41;

extern "C" int ds41_prompt_attn_fwd(const ds41_bf16* q, int64_t q_tok, int64_t q_head,
                                    const ds41_bf16* k, int64_t k_tok, int64_t k_head,
                                    const ds41_bf16* v, int64_t v_tok, int64_t v_head,
                                    const int32_t* cu_q, const int32_t* cu_k, int64_t B, int64_t Tq,
                                    int64_t Tk, int64_t max_q, int64_t nh, int64_t kvh, int64_t hd,
                                    float scale, int64_t window, const float* sink, ds41_bf16* o,
                                    float* lse, ds41_stream_t stream) {
    const char* name = "ds41_prompt_attn_fwd";
    if (int rc = check_heads(name, nh, kvh, hd, scale, window)) return rc;
    const int64_t lim = int64_t(1) << 31;
    DS41_REQUIRE(B >= 0 && B < 65536 && Tq >= 0 && Tq < lim && Tk >= 0 && Tk < lim && max_q >= 0 &&
                     max_q < lim,
                 DS41_E_RANGE, "%s: B=%lld Tq=%lld Tk=%lld max_q=%lld", name, (long long)B,
                 (long long)Tq, (long long)Tk, (long long)max_q);
    if (B == 0 || Tq == 0 || max_q == 0) return DS41_OK;
    DS41_REQUIRE(q && o && cu_q && cu_k && (Tk == 0 || (k && v)), DS41_E_ARG,
                 "%s: q, k, v, cu_q, cu_k and o must be non-null", name);
    DS41_REQUIRE(aligned16(q) && aligned16(k) && aligned16(v) && aligned16(o) &&
                     aligned_to(cu_q, 4) && aligned_to(cu_k, 4) && aligned_to(sink, 4) &&
                     aligned_to(lse, 4),
                 DS41_E_ARG, "%s: q, k, v and o must be 16-byte aligned", name);
    DS41_REQUIRE(good_strides(q_tok, q_head, hd) &&
                     (Tk == 0 ||
                      (good_strides(k_tok, k_head, hd) && good_strides(v_tok, v_head, hd))),
                 DS41_E_ARG, "%s: strides must be multiples of 8 and at least hd", name);
    pa::Params p{};
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.sink = sink;
    p.o = o;
    p.lse = lse;
    p.Tq = Tq;
    p.Tk = Tk;
    p.window = finite_window(window);
    p.B = (int)B;
    p.max_q = (int)max_q;
    p.nh = (int)nh;
    p.hd = (int)hd;
    p.c = scale * tc::SM_LOG2E;
    // heads per tile: the whole group, or its largest divisor that fits
    int G = (int)(nh / kvh);
    p.subs = 1;
    if (G > pa::ROWS) {
        int d = pa::ROWS;
        while (G % d) d--;
        p.subs = G / d;
        G = d;
    }
    p.G = G;
    p.TT = pa::ROWS / G;
    p.n_groups = (int)kvh * p.subs;
    if (int rc = status_word(&p.status)) return rc;
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    if (int rc = tc::get_encode(&enc)) return rc;
    CUtensorMap mq, mk, mv;
    if (int rc = pa::make_map_heads(enc, &mq, q, Tq, nh, hd, q_tok, q_head, G, p.TT)) return rc;
    if (Tk > 0) {
        if (int rc = pa::make_map_heads(enc, &mk, k, Tk, kvh, hd, k_tok, k_head, 1, pa::KB))
            return rc;
        if (int rc = pa::make_map_heads(enc, &mv, v, Tk, kvh, hd, v_tok, v_head, 1, pa::KB))
            return rc;
    } else {
        mk = mv = mq;  // never read
    }
    // every sequence has at most one tile pair that is not full
    const int64_t pairs = Tq / (2 * p.TT) + B;
    const int64_t blocks = pairs * p.n_groups;
    DS41_REQUIRE(blocks < lim, DS41_E_RANGE, "%s: Tq=%lld B=%lld kvh=%lld", name, (long long)Tq,
                 (long long)B, (long long)kvh);
    auto kern = hd <= 64 ? pa::prompt_attn_kernel<64> : pa::prompt_attn_kernel<128>;
    const size_t smem = hd <= 64 ? pa::Cfg<64>::SMEM : pa::Cfg<128>::SMEM;
    if (int rc = hd <= 64 ? allow_smem<pa::prompt_attn_kernel<64>>((int)smem, name)
                          : allow_smem<pa::prompt_attn_kernel<128>>((int)smem, name))
        return rc;
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(pa::THREADS), smem, (cudaStream_t)stream,
                      name, mq, mk, mv, p);
}
