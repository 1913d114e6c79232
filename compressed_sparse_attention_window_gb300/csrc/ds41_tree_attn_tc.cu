// ds41_tree_attn_tc.cu - attention of drafted tokens over a paged cache on the
// 5th-generation tensor cores, for more than a handful of rows per key/value
// head.
//
// Mathematics: that of ds41_tree_attn.cu, in blocks of 128 keys and 128 rows (a
// row: a drafted token and one of the G query heads that share the key/value
// head).
//
// Design.  One CTA per SM works through its run of the key blocks of all
// sequences (Share in ds41_tree.cuh).  It has two streams t = 0, 1, each with its
// own scores S_t and output O_t in tensor memory and its own softmax warpgroup (a
// thread per row), so that the tensor core works on one while the other's
// softmax runs; the issue order is PV_0 QK_0 PV_1 QK_1 as in the prompt kernel.
// What the streams are depends on the rows:
// * PAIR, more than 128 rows: two tiles of 128 rows over the same key blocks (each
//   block is loaded and widened once for 256 rows);
// * else: one tile of rows, the even key blocks to stream 0 and the odd ones to
//   stream 1, joined through shared memory at the end.
//
// A bf16 cache arrives by TMA, page by page, in the layout the products want.  An
// e4m3 cache has to be widened (the products take one operand type): its codes
// arrive as bulk copies, one for each run of rows of a page, and four warps turn
// them into f16 (exact, two codes an instruction; bf16 takes four) and store them
// swizzled.  The threads' 16-code pieces are dealt so that neither side has bank
// conflicts: eight lanes take four pieces of a row and the other four of the next
// row, which are 128 contiguous bytes of codes modulo 128 and eight different
// bank groups of the swizzled tile.  The queries become f16 with an exponent per
// row, the scales stay outside the products: ks multiplies the scores, vs the
// weights.
//
// What bounds it.  No single unit: a block of 128 e4m3 keys takes 96 KB through
// shared memory to be read and widened, 96 KB for the products' operands, and the
// scaled softmax 2700 cycles of its warps (1430 without scales); with one tile of rows
// the widening warps are as busy, 1150 cycles for a block's K and for its V.  The
// copies' waits look at every second use of a stage and are right because stages are
// freed in the ring's order.  8 trees of up to
// 16 tokens over 16384 keys, 32 heads of 128 over 8: 91 us; 4 of 64 over 32768, 64
// heads: 221 us.
#include "ds41_internal.cuh"
#include "ds41_tree.cuh"

namespace ds41 {
namespace tree {

using namespace tc;

constexpr int KB = 128;  // keys per block
constexpr int SCN = 8;   // blocks whose scales and visibility are held

// warps 0 K copies, 1 MMA, 2 V copies, 3 the next step, 4..7 and 8..11 softmax,
// 12..15 widening (e4m3)
template <int D, bool E4M3, bool PAIR>
struct TcCfg {
    static constexpr int THREADS = E4M3 ? 512 : 384;
    static constexpr int NB = D / 64;
    static constexpr uint32_t BLK = 128 * 128;
    static constexpr uint32_t TILE = NB * BLK;               // a K or V block, 16 bits a value
    static constexpr int QT = PAIR ? 2 : 1;                  // tiles of rows
    static constexpr int STAGES = E4M3 ? 3 : 4;
    static constexpr int CODES = PAIR ? 3 : 5;               // tiles of codes in flight
    static constexpr uint32_t CTILE = E4M3 ? KB * D : 0;
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t KV_OFF = QT * TILE;
    static constexpr uint32_t C_OFF = KV_OFF + STAGES * TILE;
    static constexpr uint32_t SC_OFF = C_OFF + CODES * CTILE;
    // per held block: 4 words of real keys and for e4m3 ks [128], vs [128]
    static constexpr uint32_t SC_BYTES = (E4M3 ? 1024 : 0) + 16;
    static constexpr uint32_t QE_OFF = SC_OFF + SCN * SC_BYTES;  // the queries' exponents
    static constexpr uint32_t BAR_OFF = QE_OFF + (E4M3 ? QT * 128 : 0);
    static constexpr uint32_t SMEM = BAR_OFF + 1024 + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
    static constexpr int LA = PAIR ? 1 : 2;  // K blocks ahead of the V blocks
    // the other stream's rows at the end of a piece (no tile is in use then)
    static constexpr int XP = D + 4;
    static_assert(PAIR || 128 * XP * 4 <= STAGES * TILE, "exchange area");
};

// The ring holds K and V blocks in the order in which they are used: the first
// LA K blocks, then V_i, K_{i+LA} for i = 0 ..
template <int LA>
__device__ __forceinline__ int pos_k(int j) {
    return j < LA ? j : LA + 2 * (j - LA) + 1;
}
template <int LA>
__device__ __forceinline__ int pos_v(int j, int n) {
    return min(LA, n) + j + min(j, max(0, n - LA));
}
// Which of the keys j .. j + 31 a row sees.
__device__ __forceinline__ uint32_t low_bits(int64_t n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
__device__ __forceinline__ uint32_t seen_word(const RowView& w, int n_drafted, int j) {
    const uint32_t earlier = low_bits((int64_t)w.pre - j);
    uint32_t r = earlier & ~low_bits(w.lo + 1 - j);
    if (earlier != 0xffffffffu) {
        uint32_t d;
        if (!w.bits) {
            d = low_bits((int64_t)w.chain_last + 1 - j);
        } else {
            const int u = j - w.pre;  // the drafted token of the first key
            if (u < 0) {
                d = u <= -32 ? 0u : (uint32_t)((uint64_t)w.bits[0] << -u);
            } else if (u >= n_drafted) {
                d = 0;
            } else {
                const int i = u >> 6, sh = u & 63;
                d = (uint32_t)((uint64_t)w.bits[i] >> sh);
                if (sh > 32 && (i + 1) * 64 < n_drafted)
                    d |= (uint32_t)((uint64_t)w.bits[i + 1] << (64 - sh));
            }
        }
        r |= d & ~earlier;
    }
    return r;
}

// A step of the CTA's walk through its pieces, in shared memory (two: one thread
// plans the next while the roles work on the present): the piece, and what the
// barriers have seen before it: entries of the ring, blocks, blocks and ends of
// each stream, V blocks with rows behind the last key.  The roles read what they
// need when they need it: held in registers through the key loop it would push
// the softmax warps' scores into local memory, which shared memory of this size
// leaves hardly any cache for.
struct Step {
    Piece pc;
    int more;                    // 0: the walk is over
    int rows, r0, k0, k1, n_blocks, tail;  // tail: keys of the last block
    int nt[2];                   // blocks of each stream
    int ring0, blocks0, used0[2], ends0[2], tails0;
};
template <int QT>
__device__ __forceinline__ void plan_step(const Args& a, Share& share, const Step& was, Step& w) {
    constexpr bool PAIR = QT == 2;
    Piece pc;
    w.more = next_piece(a, share, pc) ? 1 : 0;
    if (!w.more) return;
    w.pc = pc;
    w.rows = pc.s.n * a.G;
    w.r0 = pc.tile * QT * 128;
    w.k0 = pc.key;
    w.k1 = min(pc.s.len, w.k0 + pc.count * KB);
    w.n_blocks = pc.count;
    w.tail = (w.k1 - w.k0) - (pc.count - 1) * KB;
    w.nt[0] = PAIR ? pc.count : (pc.count + 1) / 2;
    w.nt[1] = PAIR ? (w.rows - w.r0 > 128 ? pc.count : 0) : pc.count / 2;
    w.ring0 = was.ring0 + 2 * was.n_blocks;
    w.blocks0 = was.blocks0 + was.n_blocks;
    for (int t = 0; t < 2; t++) {
        w.used0[t] = was.used0[t] + was.nt[t];
        w.ends0[t] = was.ends0[t] + (was.nt[t] > 0);
    }
    w.tails0 = was.tails0 + (was.n_blocks > 0 && was.tail < KB);
    note_ends(a, pc);
}

template <int D, bool E4M3, bool PAIR>
__global__ void __launch_bounds__(TcCfg<D, E4M3, PAIR>::THREADS, 1)
    tree_many_kernel(const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const Args a) {
    pdl_wait();
    using C = TcCfg<D, E4M3, PAIR>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    uint8_t* sm = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const uint32_t sbase = smem_u32(sm);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::BAR_OFF);
    uint64_t* b_full = bars;                  // a K or V block is in its stage
    uint64_t* b_empty = b_full + C::STAGES;   // it has been used
    uint64_t* b_code = b_empty + C::STAGES;   // a tile of codes has arrived
    uint64_t* b_codee = b_code + C::CODES;    // it has been read
    uint64_t* b_sc = b_codee + C::CODES;      // a block's scales and real keys are there
    uint64_t* b_sce = b_sc + SCN;             // they have been read
    uint64_t* b_s = b_sce + SCN;              // S_t in tensor memory [2]
    uint64_t* b_p = b_s + 2;                  // P_t in tensor memory, O_t rescaled [2]
    uint64_t* b_o = b_p + 2;                  // O_t complete [2]
    uint64_t* b_tail = b_o + 2;               // the V block with the last key landed
    uint64_t* b_fix = b_tail + 1;             // its rows behind the last key are zero
    uint64_t* b_end = b_fix + 1;              // every product is complete
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b_end + 2);
    volatile int* abort_f = reinterpret_cast<volatile int*>(tmem_slot + 1);
    int64_t* sh = reinterpret_cast<int64_t*>(tmem_slot + 2);
    Step* steps = reinterpret_cast<Step*>(sh + C::THREADS / 32 + 4);
    static_assert((2 * C::STAGES + 2 * C::CODES + 2 * SCN + 10) * 8 + 8 +
                          (C::THREADS / 32 + 4) * 8 + 2 * sizeof(Step) <= 1024,
                  "barrier area");
    const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; i++) {
            mbar_init(&b_full[i], E4M3 ? 4 : 1);
            mbar_init(&b_empty[i], 1);
        }
        for (int i = 0; i < C::CODES; i++) {
            mbar_init(&b_code[i], 1);
            mbar_init(&b_codee[i], 4);
        }
        for (int i = 0; i < SCN; i++) {
            mbar_init(&b_sc[i], 1);
            mbar_init(&b_sce[i], PAIR ? 8 : 4);
        }
        for (int t = 0; t < 2; t++) {
            mbar_init(&b_s[t], 1);
            mbar_init(&b_p[t], 4);
            mbar_init(&b_o[t], 1);
        }
        mbar_init(b_tail, 1);
        mbar_init(b_fix, 1);
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
    tc_fence_before();
    Share share = find_share<C::THREADS>(a, sh, blockIdx.x == 0);  // (synchronises)
    tc_fence_after();
    const uint32_t tmem = (uint32_t)uniform((int)*tmem_slot);
    constexpr uint32_t TM_S = 0, TM_O = 256;
    // Every role walks the same pieces; all of them meet where a piece begins (its
    // queries are in shared memory), for one tile of rows again where its streams
    // end, and where it ends.  The roles' code is kept apart so that each has its
    // own share of the register file (128 a thread at launch, 168 on bf16).
    if (threadIdx.x == 96) {
        steps[1].n_blocks = steps[1].ring0 = steps[1].blocks0 = steps[1].tails0 = 0;
        steps[1].nt[0] = steps[1].nt[1] = 0;
        for (int t = 0; t < 2; t++) steps[1].used0[t] = steps[1].ends0[t] = 0;
        plan_step<C::QT>(a, share, steps[1], steps[0]);
    }
    __syncthreads();
    bool ok = true;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(E4M3 ? 72 : 88));
        for (int turn = 0; steps[turn & 1].more; turn++) {
            const Step& w = steps[turn & 1];
            const int32_t* table = a.table + (int64_t)uniform(w.pc.b) * a.max_pages;
            const int h = uniform(w.pc.h);
            const int k0 = uniform(w.k0), k1 = uniform(w.k1);
            const int n_blocks = uniform(w.n_blocks), n_ring = 2 * n_blocks;
            const int ring0 = uniform(w.ring0), blocks0 = uniform(w.blocks0);
            const int tail = uniform(w.tail), tails0 = uniform(w.tails0);
            const int nt[2] = {uniform(w.nt[0]), uniform(w.nt[1])};
            const int used0[2] = {uniform(w.used0[0]), uniform(w.used0[1])};
            auto uses = [&](int t, int j) { return PAIR ? nt[t] > 0 : (j & 1) == t; };
            __syncthreads();
            if (threadIdx.x == 96) plan_step<C::QT>(a, share, w, steps[(turn + 1) & 1]);
            if ((warp == 0 || warp == 2) && ok) {
                // pages -> stages (bf16) or code tiles (e4m3): warp 0 the K blocks,
                // and which keys are real, warp 2 the V blocks (one warp takes 1500
                // cycles for a block's K and as many for its V)
                const int kv = warp >> 1;
                constexpr int DEPTH = E4M3 ? C::CODES : C::STAGES;
                uint64_t* const arrived = E4M3 ? b_code : b_full;
                uint64_t* const freed = E4M3 ? b_codee : b_empty;
                const int shift = min(a.kv.page_shift, 7), per = 1 << shift;  // rows of a copy
                const int copies = KB >> shift;
                const bool copier = lane < copies;
                const uint8_t* const src = kv ? a.kv.v : a.kv.k;
                const int64_t head_rows = (int64_t)h * a.kv.page;
                const int64_t page_rows = (int64_t)a.kvh * a.kv.page;
                // lane i < copies: the page of the rows it copies, looked up a block ahead
                auto page_of = [&](int j) {
                    const int key = k0 + j * KB + lane * per;
                    return copier && key < k1 ? table[key >> a.kv.page_shift] : -1;
                };
                int next = page_of(0), sent = 0;
                for (; sent < n_blocks; sent++) {
                    const int j = sent, e = kv ? pos_v<C::LA>(j, n_blocks) : pos_k<C::LA>(j);
                    const int ge = ring0 + e, st = ge % DEPTH, use = ge / DEPTH;
                    const int page = next;
                    next = page_of(j + 1);
                    const int gb = blocks0 + j, sl = gb % SCN;
                    if (use > 0) ok = warp_wait(&freed[st], (use - 1) & 1, abort_f, a.status);
                    if (ok && kv == 0 && gb >= SCN)
                        ok = warp_wait(&b_sce[sl], ((gb / SCN) - 1) & 1, abort_f, a.status);
                    if (!ok) break;
                    const int key0 = k0 + j * KB, key = key0 + lane * per;
                    const int n = copier ? max(0, min(per, k1 - key)) : 0;
                    const bool real = page >= 0 && page < a.kv.n_pages;
                    const bool lost = n > 0 && !real;
                    const bool plain = __all_sync(0xffffffffu, !copier || (n == per && real));
                    if (lost && kv == 0) raise_status(a.status, DS41_E_INDEX);
                    uint8_t* const sc = sm + C::SC_OFF + sl * C::SC_BYTES;
                    uint8_t* const dst = sm + C::C_OFF + st * C::CTILE;
                    uint32_t bytes = (uint32_t)(KB * a.hd), sbytes = 2 * KB * 4;
                    const uint32_t mine = real ? (uint32_t)(n * a.hd) : 0u;
                    const uint32_t smine = real ? (uint32_t)((n + 3) / 4 * 16) : 0u;
                    if (!plain) {
                        const uint32_t good = __ballot_sync(0xffffffffu, n > 0 && real);
                        if (kv == 0 && lane < 4) {
                            // word i: which of the keys 32 i .. are real
                            uint32_t word = 0;
                            for (int x = 0; x < 32; x += 16)
                                if ((good >> ((32 * lane + x) >> shift)) & 1) word |= 0xffffu << x;
                            reinterpret_cast<uint32_t*>(sc)[lane] =
                                word & low_bits((int64_t)k1 - key0 - 32 * lane);
                        }
                        if (E4M3) {
                            bytes = __reduce_add_sync(0xffffffffu, mine);
                            sbytes = 2 * __reduce_add_sync(0xffffffffu, smine);
                            // rows that no copy fills are zero: no product meets a NaN
                            for (int i = 0; i < copies; i++) {
                                const int have = __shfl_sync(0xffffffffu, real ? n : 0, i);
                                for (int x = lane; x < (per - have) * a.hd / 16; x += 32)
                                    *reinterpret_cast<uint4*>(dst + (i * per + have) * a.hd +
                                                              x * 16) = make_uint4(0, 0, 0, 0);
                            }
                        }
                    } else if (kv == 0 && lane < 4) {
                        reinterpret_cast<uint32_t*>(sc)[lane] = 0xffffffffu;
                    }
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive_expect_tx(&arrived[st], E4M3 ? bytes : C::TILE);
                        if (kv == 0) {
                            if (E4M3) mbar_arrive_expect_tx(&b_sc[sl], sbytes);
                            else mbar_arrive(&b_sc[sl]);
                        }
                    }
                    __syncwarp();
                    const int off = key & (a.kv.page - 1);
                    if (E4M3) {
                        if (mine) {
                            const int64_t row = page * page_rows + head_rows + off;
                            bulk_g2s(dst + lane * per * a.hd, src + row * a.hd, mine, &arrived[st]);
                            if (kv == 0) {
                                bulk_g2s(sc + 16 + lane * per * 4, a.kv.ks + row, smine, &b_sc[sl]);
                                bulk_g2s(sc + 528 + lane * per * 4, a.kv.vs + row, smine,
                                         &b_sc[sl]);
                            }
                        }
                    } else if (copier) {
                        // a page that does not exist reads as zeros (a coordinate
                        // past the tensor)
                        const int z = (int)(n > 0 && real ? (int64_t)page * a.kvh + h
                                                          : a.kv.n_pages * a.kvh);
#pragma unroll
                        for (int x = 0; x < C::NB; x++)
                            tma_load_3d(sbase + C::KV_OFF + st * C::TILE + x * C::BLK +
                                            lane * per * 128,
                                        kv ? &map_v : &map_k, 64 * x, off, z, &arrived[st]);
                    }
                }
                if (warp == 2 && !E4M3 && tail < KB && ok) {
                    // the V rows behind the last key hold whatever an earlier user left
                    const int ge = ring0 + pos_v<C::LA>(n_blocks - 1, n_blocks);
                    ok = warp_wait(b_tail, tails0 & 1, abort_f, a.status);
                    if (ok) {
                        uint8_t* v = sm + C::KV_OFF + (ge % C::STAGES) * C::TILE;
                        for (int x = lane; x < (KB - tail) * C::NB * 8; x += 32) {
                            const int r = tail + x / (C::NB * 8), piece = x % (C::NB * 8);
                            *reinterpret_cast<uint4*>(v + (piece / 8) * C::BLK + r * 128 +
                                                      (piece % 8) * 16) = make_uint4(0, 0, 0, 0);
                        }
                        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                        __syncwarp();
                        if (lane == 0) mbar_arrive(b_fix);
                    }
                }
                // everything that was started lands before the piece ends (a stage that
                // the other warp has filled since says so by itself)
                for (int j = max(0, sent - DEPTH); j < sent; j++) {
                    const int e = kv ? pos_v<C::LA>(j, n_blocks) : pos_k<C::LA>(j);
                    const int ge = ring0 + e;
                    if (!ok || e >= n_ring - DEPTH)
                        drain_bar(&arrived[ge % DEPTH], (ge / DEPTH) & 1, a.status);
                }
            } else if (warp == 1 && ok) {
                constexpr uint32_t IDESC_S =
                    E4M3 ? idesc_f16(128, KB, 0, 0) : idesc_bf16(128, KB, 0, 0);
                constexpr uint32_t IDESC_O =
                    E4M3 ? idesc_f16(128, D, 0, 1) : idesc_bf16(128, D, 0, 1);
                const uint32_t qd = desc_lo(sbase + C::Q_OFF, 16);
                const uint32_t kd = desc_lo(sbase + C::KV_OFF, 16);
                const uint32_t vd = desc_lo(sbase + C::KV_OFF, C::BLK);
                int done_p[2] = {0, 0};
                auto wait_entry = [&](int e) {
                    const int ge = ring0 + e;
                    const bool r =
                        warp_wait(&b_full[ge % C::STAGES], (ge / C::STAGES) & 1, abort_f, a.status);
                    tc_fence_after();
                    return r;
                };
                auto stage_of = [&](int e) { return (ring0 + e) % C::STAGES; };
                auto stage_off = [&](int e) { return (stage_of(e) * C::TILE) >> 4; };
                auto scores = [&](int t, int e) {
                    mma_scores<D, IDESC_S>(tmem + TM_S + 128 * t,
                                           qd + ((PAIR ? t * C::TILE : 0) >> 4), kd + stage_off(e));
                    tc_commit(&b_s[t]);
                };
                for (int j = 0; j < min(C::LA, n_blocks) && ok; j++) {
                    ok = wait_entry(j);
                    if (ok && elect_one()) {
#pragma unroll
                        for (int t = 0; t < 2; t++)
                            if (uses(t, j)) scores(t, j);
                        tc_commit(&b_empty[stage_of(j)]);
                    }
                    __syncwarp();
                }
                for (int j = 0; j < n_blocks && ok; j++) {
                    const int ev = pos_v<C::LA>(j, n_blocks);
                    const bool more = j + C::LA < n_blocks;
                    const int ek = pos_k<C::LA>(j + C::LA);
                    ok = wait_entry(ev);
                    if (ok && !E4M3 && tail < KB && j == n_blocks - 1) {
                        if (lane == 0) mbar_arrive(b_tail);
                        ok = warp_wait(b_fix, tails0 & 1, abort_f, a.status);
                        tc_fence_after();
                    }
                    bool have_k = false;
#pragma unroll
                    for (int t = 0; t < 2; t++) {
                        const bool now = uses(t, j), next = more && uses(t, j + C::LA);
                        if (ok && now) {
                            ok = warp_wait(&b_p[t], (used0[t] + done_p[t]) & 1, abort_f, a.status);
                            done_p[t]++;
                            tc_fence_after();
                        }
                        if (ok && elect_one()) {
                            if (now) {
                                mma_output<D, IDESC_O>(tmem + TM_O + 128 * t, tmem + TM_S + 128 * t,
                                                       vd + stage_off(ev), done_p[t] > 1);
                                if (done_p[t] == nt[t]) tc_commit(&b_o[t]);
                            }
                            if (t == 1) tc_commit(&b_empty[stage_of(ev)]);
                        }
                        __syncwarp();
                        if (ok && next) {
                            if (!have_k) ok = wait_entry(ek);
                            have_k = true;
                            if (ok && elect_one()) scores(t, ek);
                            __syncwarp();
                        }
                    }
                    if (ok && more && elect_one()) tc_commit(&b_empty[stage_of(ek)]);
                    __syncwarp();
                }
            }
            if (!PAIR) __syncthreads();
            __syncthreads();
            if (*abort_f) ok = false;
        }
    } else if (E4M3 && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 40;\n");
        const int tid = threadIdx.x - 384;
        constexpr int PIECES = KB * D / 16 / 128;  // 16-code pieces a thread has of a tile
        constexpr int RPP = 128 / PIECES;          // rows from a piece to the next
        int r_in, ch;
        if (D == 128) {
            const int p = tid >> 3, odd = (tid >> 2) & 1;  // pair of rows and half
            r_in = (p >> 1) * 2 + odd;
            ch = (tid & 3) + 4 * (odd ^ (p & 1));
        } else {
            r_in = tid >> 2;
            ch = tid & 3;
        }
        const bool in_row = ch * 16 < a.hd;
        const uint32_t src_off = (uint32_t)(r_in * a.hd + ch * 16);
        const int c0 = (ch & 3) * 2;
        // (RPP is a multiple of 8, so r & 7 is that of r_in)
        const uint32_t dst0 =
            (ch >> 2) * C::BLK + r_in * 128 + (uint32_t)((c0 ^ (r_in & 7)) << 4);
        const uint32_t dst1 =
            (ch >> 2) * C::BLK + r_in * 128 + (uint32_t)(((c0 + 1) ^ (r_in & 7)) << 4);
        for (int turn = 0; steps[turn & 1].more; turn++) {
            const Step& w = steps[turn & 1];
            const int n_ring = 2 * uniform(w.n_blocks), ring0 = uniform(w.ring0);
            __syncthreads();
            for (int e = 0; e < n_ring && ok; e++) {
                const int ge = ring0 + e, cs = ge % C::CODES, st = ge % C::STAGES;
                ok = warp_wait(&b_code[cs], (ge / C::CODES) & 1, abort_f, a.status);
                if (!ok) break;
                if (ge >= C::STAGES) {
                    ok = warp_wait(&b_empty[st], ((ge / C::STAGES) - 1) & 1, abort_f, a.status);
                    if (!ok) break;
                }
                const uint8_t* from = sm + C::C_OFF + cs * C::CTILE + src_off;
                uint8_t* to = sm + C::KV_OFF + st * C::TILE;
                // four pieces at a time: the widening warps live on few registers
#pragma unroll 1
                for (int x0 = 0; x0 < PIECES; x0 += 4) {
                    uint4 w[4];
#pragma unroll
                    for (int x = 0; x < 4; x++)
                        w[x] = in_row
                                   ? *reinterpret_cast<const uint4*>(from + (x0 + x) * RPP * a.hd)
                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int x = 0; x < 4; x++) {
                        uint32_t out[8];
                        e4m3x4_to_f16(w[x].x, out[0], out[1]);
                        e4m3x4_to_f16(w[x].y, out[2], out[3]);
                        e4m3x4_to_f16(w[x].z, out[4], out[5]);
                        e4m3x4_to_f16(w[x].w, out[6], out[7]);
                        *reinterpret_cast<uint4*>(to + dst0 + (x0 + x) * RPP * 128) =
                            make_uint4(out[0], out[1], out[2], out[3]);
                        *reinterpret_cast<uint4*>(to + dst1 + (x0 + x) * RPP * 128) =
                            make_uint4(out[4], out[5], out[6], out[7]);
                    }
                }
                // (the codes have been read: the copies that follow wait for this)
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&b_full[st]);
                    mbar_arrive(&b_codee[cs]);
                }
            }
            if (!PAIR) __syncthreads();
            __syncthreads();
            if (*abort_f) ok = false;
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(E4M3 ? 200 : 208));
        for (int turn = 0; steps[turn & 1].more; turn++) {
            const Step& w = steps[turn & 1];
            {
                // the queries, 128-byte swizzled; rows that do not exist are zero.  A
                // thread has one 16-byte piece of every (256 * 8 / D)-th row, four in
                // flight
                constexpr int CPR = D / 8, STEP = 256 / CPR;
                const int tid = threadIdx.x - 128, ch = tid % CPR;
                const uint16_t* q0 =
                    a.q + w.pc.s.q0 * a.q_tok + (int64_t)w.pc.h * a.G * a.q_head + ch * 8;
                const int rows = w.rows - w.r0;
#pragma unroll 1
                for (int k = tid / CPR; k < C::QT * 128; k += 4 * STEP) {
                    uint4 v[4];
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const int r = k + u * STEP;
                        const uint32_t rr = (uint32_t)(w.r0 + r), t = rr / (uint32_t)a.G;
                        v[u] = make_uint4(0, 0, 0, 0);
                        if (r < rows && ch * 8 < a.hd)
                            v[u] = *reinterpret_cast<const uint4*>(q0 + t * a.q_tok +
                                                                   (rr - t * a.G) * a.q_head);
                    }
#pragma unroll
                    for (int u = 0; u < 4; u++) {
                        const int r = k + u * STEP;
                        if (E4M3) {  // D / 8 lanes have a row
                            const uint32_t m2 =
                                __vmaxu2(__vmaxu2(v[u].x & 0x7fff7fffu, v[u].y & 0x7fff7fffu),
                                         __vmaxu2(v[u].z & 0x7fff7fffu, v[u].w & 0x7fff7fffu));
                            uint32_t mb = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
                            for (int off = D / 16; off > 0; off >>= 1)
                                mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, off));
                            const int e = query_exponent(mb);
                            const float down = exp2f((float)-e);
                            v[u] = make_uint4(
                                bf16x2_to_f16x2(v[u].x, down), bf16x2_to_f16x2(v[u].y, down),
                                bf16x2_to_f16x2(v[u].z, down), bf16x2_to_f16x2(v[u].w, down));
                            if (ch == 0) reinterpret_cast<int8_t*>(sm + C::QE_OFF)[r] = (int8_t)e;
                        }
                        *reinterpret_cast<uint4*>(sm + C::Q_OFF + (r >> 7) * C::TILE +
                                                  (ch >> 3) * C::BLK + (r & 127) * 128 +
                                                  (((ch & 7) ^ (r & 7)) << 4)) = v[u];
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            __syncthreads();

            // what a stream leaves: reference (log2), sum; its rows are in tensor memory
            float end_m = -INFINITY, end_l = 0.0f;
            if (ok) {
                const int t = (warp - 4) >> 2;
                const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
                const uint32_t tm_s = tmem + lanes + TM_S + 128 * t;
                const uint32_t tm_o = tmem + lanes + TM_O + 128 * t;
                const int row = w.r0 + (PAIR ? 128 * t : 0) + 32 * (warp & 3) + lane;
                const bool live = row < w.rows;
                const bool idle = !__any_sync(0xffffffffu, live);  // none of the warp's rows is
                const RowView view = row_view(a, w.pc.s, min(row, w.rows - 1) / a.G);
                const int nt = uniform(w.nt[t]), n_blocks = uniform(w.n_blocks);
                const int k0 = uniform(w.k0), blocks0 = uniform(w.blocks0);
                const int used0 = uniform(w.used0[t]);
                float c = a.scale_log2;
                if (E4M3)
                    c = fmaxf(c * exp2f((float)reinterpret_cast<const int8_t*>(
                                      sm + C::QE_OFF)[(PAIR ? 128 * t : 0) + 32 * (warp & 3) + lane]),
                              SM_C_MIN);
                RowState st;
                for (int j = PAIR ? 0 : t, i = 0; j < n_blocks; j += PAIR ? 1 : 2, i++) {
                    const int gb = blocks0 + j, sl = gb % SCN;
                    ok = warp_wait(&b_sc[sl], (gb / SCN) & 1, abort_f, a.status);
                    if (ok && nt > 0)
                        ok = warp_wait(&b_s[t], (used0 + i) & 1, abort_f, a.status);
                    if (!ok) break;
                    if (nt > 0 && !idle) {
                        tc_fence_after();
                        const float* sc =
                            reinterpret_cast<const float*>(sm + C::SC_OFF + sl * C::SC_BYTES);
                        const uint4 real = *reinterpret_cast<const uint4*>(sc);
                        const int j0 = k0 + j * KB;
                        // one choice for the warp: its lanes load from tensor memory together
                        const bool any = __any_sync(
                            0xffffffffu, (real.x & real.y & real.z & real.w) != 0xffffffffu ||
                                             j0 + KB > view.pre || j0 <= view.lo);
                        uint32_t vis[4] = {};
                        if (any) {
                            vis[0] = real.x & seen_word(view, w.pc.s.n, j0);
                            vis[1] = real.y & seen_word(view, w.pc.s.n, j0 + 32);
                            vis[2] = real.z & seen_word(view, w.pc.s.n, j0 + 64);
                            vis[3] = real.w & seen_word(view, w.pc.s.n, j0 + 96);
                        }
                        float vmax = 0.0f;
                        if (E4M3) {
                            // the largest scale of a real key (fmaxf passes over NaN; the sign of one
                            // that is not this library's has no part in it)
                            const uint32_t w = lane < 16 ? (lane < 8 ? real.x : real.y)
                                                         : (lane < 24 ? real.z : real.w);
                            const float4 v4 = *reinterpret_cast<const float4*>(sc + 132 + 4 * lane);
                            const int b4 = 4 * (lane & 7);
                            if ((w >> b4) & 1) vmax = fmaxf(vmax, fabsf(v4.x));
                            if ((w >> (b4 + 1)) & 1) vmax = fmaxf(vmax, fabsf(v4.y));
                            if ((w >> (b4 + 2)) & 1) vmax = fmaxf(vmax, fabsf(v4.z));
                            if ((w >> (b4 + 3)) & 1) vmax = fmaxf(vmax, fabsf(v4.w));
#pragma unroll
                            for (int off = 16; off > 0; off >>= 1)
                                vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
                        }
                        if (E4M3 && any)
                            softmax_block_scaled<D, true>(tm_s, tm_o, i > 0, vis, c, sc + 4,
                                                          sc + 132, vmax, live, st);
                        else if (E4M3)
                            softmax_block_scaled<D, false>(tm_s, tm_o, i > 0, vis, c, sc + 4,
                                                           sc + 132, vmax, live, st);
                        else if (any)
                            softmax_block<D, true>(tm_s, tm_o, i > 0, vis, c, live, st);
                        else
                            softmax_block<D, false>(tm_s, tm_o, i > 0, vis, c, live, st);
                        tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if (nt > 0) mbar_arrive(&b_p[t]);
                        mbar_arrive(&b_sce[sl]);
                    }
                }
                if (nt > 0 && ok) ok = warp_wait(&b_o[t], w.ends0[t] & 1, abort_f, a.status);
                // (the exchange below lies in the ring: the other stream's last products
                // have to have read it too)
                if (!PAIR && t == 1 && nt > 0 && ok)
                    ok = warp_wait(&b_o[0], w.ends0[0] & 1, abort_f, a.status);
                tc_fence_after();
                end_m = st.reference(c);
                end_l = st.l;
                if (!PAIR && t == 1 && nt > 0 && ok) {
                    // to the other stream, through the ring (nothing of it is in use)
                    float* x = reinterpret_cast<float*>(sm + C::KV_OFF) +
                               (32 * (warp & 3) + lane) * C::XP;
                    x[D] = end_m;
                    x[D + 1] = end_l;
#pragma unroll 1
                    for (int d = 0; d < D; d += 16) {
                        uint32_t ov[16];
                        tc_ld16(tm_o + d, ov);
                        tc_wait_ld();
#pragma unroll
                        for (int e = 0; e < 16; e += 4)
                            *reinterpret_cast<uint4*>(x + d + e) =
                                make_uint4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                    }
                }
            }
            if (!PAIR) __syncthreads();
            if (warp < (PAIR ? 12 : 8) && ok) {
                const int t = (warp - 4) >> 2, row_in = 32 * (warp & 3) + lane;
                const uint32_t tm_o = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + TM_O + 128 * t;
                const int row = w.r0 + 128 * t + row_in;
                const bool live = row < w.rows;
                const int held = min(row, w.rows - 1);
                const int tok = held / a.G, head = w.pc.h * a.G + held % a.G;
                const int64_t at = (int64_t)(w.pc.s.q0 + tok) * a.nh + head;
                const bool whole = is_whole(w.pc);
                const float* x = reinterpret_cast<const float*>(sm + C::KV_OFF) + row_in * C::XP;
                const bool both = !PAIR && w.nt[1] > 0;
                float f = 1.0f, fx = 0.0f, m = end_m, l = end_l;
                if (both) {
                    m = fmaxf(end_m, x[D]);
                    const float base = m == -INFINITY ? 0.0f : m;
                    f = exp2f(end_m - base);
                    fx = exp2f(x[D] - base);
                    l = f * end_l + fx * x[D + 1];
                }
                if (whole) {
                    const RowEnd end = row_end(m, l, a.sink ? a.sink[head] : -INFINITY);
                    if (live && a.lse) a.lse[at] = end.lse;
                    f *= end.factor;
                    fx *= end.factor;
                }
                const int64_t slot = slot_of(w.pc) * a.tile_rows + 128 * t + row_in;
                if (live && !whole) a.part_ml[slot] = make_float2(m, l);
                if (w.nt[t] > 0) {
#pragma unroll 1
                    for (int d = 0; d < D; d += 16) {
                        uint32_t ov[16];
                        float v[16];
                        tc_ld16(tm_o + d, ov);
                        tc_wait_ld();
                        if (!live || d >= a.hd) continue;
#pragma unroll
                        for (int e = 0; e < 16; e++) v[e] = u2f(ov[e]) * f;
                        if (both) {
#pragma unroll
                            for (int e = 0; e < 16; e += 4) {
                                const float4 y = *reinterpret_cast<const float4*>(x + d + e);
                                v[e] += y.x * fx;
                                v[e + 1] += y.y * fx;
                                v[e + 2] += y.z * fx;
                                v[e + 3] += y.w * fx;
                            }
                        }
                        if (whole) {
                            uint4* dst = reinterpret_cast<uint4*>(a.o + at * a.hd + d);
#pragma unroll
                            for (int e = 0; e < 16; e += 8)
                                dst[e / 8] =
                                    make_uint4(bf16x2(v[e], v[e + 1]), bf16x2(v[e + 2], v[e + 3]),
                                               bf16x2(v[e + 4], v[e + 5]), bf16x2(v[e + 6], v[e + 7]));
                        } else {
                            float4* dst = reinterpret_cast<float4*>(a.part + slot * a.hd + d);
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                dst[e / 4] = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                        }
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            }
            // tensor memory, the queries and the ring are free for the next piece
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
            if (*abort_f) ok = false;
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
            drain_bar(b_end, 0, a.status);
        }
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem)
                     : "memory");
    }
}

namespace {

// [n_pages * kvh][page][hd] bf16, a box of 64 columns x min(page, 128) rows
int make_map_pages(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* ptr,
                   const PagedKv& kv) {
    cuuint64_t dims[3] = {(cuuint64_t)kv.hd, (cuuint64_t)kv.page,
                          (cuuint64_t)(kv.n_pages * kv.kvh)};
    cuuint64_t strides[2] = {(cuuint64_t)kv.hd * 2, (cuuint64_t)kv.hd * kv.page * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)(kv.page < KB ? kv.page : KB), 1u};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(DS41_E_CUDA, "cuTensorMapEncodeTiled (pages) failed (%d)", (int)r);
    return DS41_OK;
}

template <int D, bool E4M3, bool PAIR>
int launch_many_as(const Args& a, const char* name, cudaStream_t st) {
    using C = TcCfg<D, E4M3, PAIR>;
    CUtensorMap mk = {}, mv = {};
    if (!E4M3) {
        PFN_cuTensorMapEncodeTiled_v12000 enc;
        if (int rc = get_encode(&enc)) return rc;
        if (int rc = make_map_pages(enc, &mk, a.kv.k, a.kv)) return rc;
        if (int rc = make_map_pages(enc, &mv, a.kv.v, a.kv)) return rc;
    }
    auto kern = tree_many_kernel<D, E4M3, PAIR>;
    if (int rc = allow_smem<tree_many_kernel<D, E4M3, PAIR>>((int)C::SMEM, name)) return rc;
    return launch_pdl(kern, dim3((unsigned)a.workers), dim3(C::THREADS), C::SMEM, st, name, mk, mv,
                      a);
}

}  // namespace

int launch_many(const Args& a, const char* name, cudaStream_t st) {
    const bool e = a.kv.ks != nullptr, pair = a.tile_rows == 256;
    if (a.hd <= 64)
        return e ? (pair ? launch_many_as<64, true, true>(a, name, st)
                         : launch_many_as<64, true, false>(a, name, st))
                 : (pair ? launch_many_as<64, false, true>(a, name, st)
                         : launch_many_as<64, false, false>(a, name, st));
    return e ? (pair ? launch_many_as<128, true, true>(a, name, st)
                     : launch_many_as<128, true, false>(a, name, st))
             : (pair ? launch_many_as<128, false, true>(a, name, st)
                     : launch_many_as<128, false, false>(a, name, st));
}

}  // namespace tree
}  // namespace ds41
