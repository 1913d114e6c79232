// ds41_tree_attn_tc.cu - attention of drafted tokens over a paged cache on the
// 5th-generation tensor cores, for more than a handful of rows per key/value
// head.
//
// Mathematics: that of ds41_tree_attn.cu, in blocks of 128 keys and 128 rows (a
// row: a drafted token and one of the G query heads that share the key/value
// head).
//
// Design.  A CTA runs two streams t = 0, 1, each with its own scores S_t and
// output O_t in tensor memory and its own softmax warpgroup (a thread per row),
// so that the tensor core works on one while the other's softmax runs; the issue
// order is PV_0 QK_0 PV_1 QK_1 as in the prompt kernel.  What the streams are
// depends on the rows:
// * more than 128 rows: two tiles of 128 rows over the same key blocks (each
//   block is loaded and widened once for 256 rows);
// * up to 128 rows: one tile of rows, the even key blocks to stream 0 and the
//   odd ones to stream 1, joined at the end like two splits.
// The keys are split over CTAs (chunks), partial results joined by the second
// kernel of the few-row path.
//
// A bf16 cache arrives by TMA, page by page, in the layout the products want.  An
// e4m3 cache has to be widened (the products take one operand type): four warps
// fetch the codes with cp.async, every thread its own pieces, some tiles ahead,
// so no barrier stands between a piece's arrival and its use, turn them into f16
// (exact, two codes an instruction; bf16 takes four) and store them swizzled.
// The threads' pieces are dealt so that eight lanes store into eight different
// bank groups (rows r and r + 1 side by side, their halves crossed) and the code
// buffer is private to each thread, so neither side has bank conflicts.  The
// queries become f16 with an exponent per row, the scales stay outside the
// products: ks multiplies the scores, vs the weights.
#include "ds41_internal.cuh"
#include "ds41_softmax_tc.cuh"
#include "ds41_tree.cuh"

namespace ds41 {
namespace tree {

using namespace tc;

constexpr int KB = 128;  // keys per block
constexpr int SCN = 4;   // blocks whose scales and visibility are held

// warps 0 TMA, 1 MMA, 2 tail, 4..7 and 8..11 softmax, 12..15 widening (e4m3)
template <int D, bool E4M3, bool PAIR>
struct TcCfg {
    static constexpr int THREADS = E4M3 ? 512 : 384;
    static constexpr int NB = D / 64;
    static constexpr uint32_t BLK = 128 * 128;
    static constexpr uint32_t TILE = NB * BLK;               // a K or V block in bf16
    static constexpr int QT = PAIR ? 2 : 1;                  // tiles of rows
    static constexpr int STAGES = E4M3 ? 3 : 4;
    static constexpr int CODES = PAIR ? 3 : 5;               // tiles of codes in flight
    static constexpr uint32_t CTILE = E4M3 ? KB * D : 0;
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t KV_OFF = QT * TILE;
    static constexpr uint32_t C_OFF = KV_OFF + STAGES * TILE;
    static constexpr uint32_t SC_OFF = C_OFF + CODES * CTILE;
    // per held block: 4 words of real keys, and for e4m3 the largest vs of each
    // 32 keys, ks [128], vs [128]
    static constexpr uint32_t SC_BYTES = (E4M3 ? 1024 + 16 : 0) + 16;
    static constexpr uint32_t QE_OFF = SC_OFF + SCN * SC_BYTES;  // the queries' exponents
    static constexpr uint32_t BAR_OFF = QE_OFF + (E4M3 ? QT * 128 : 0);
    static constexpr uint32_t SMEM = BAR_OFF + 512 + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
    static constexpr int LA = PAIR ? 1 : 2;  // K blocks ahead of the V blocks
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
    uint64_t* b_sc = b_empty + C::STAGES;     // a block's scales and real keys are there
    uint64_t* b_sce = b_sc + SCN;             // they have been read
    uint64_t* b_s = b_sce + SCN;              // S_t in tensor memory [2]
    uint64_t* b_p = b_s + 2;                  // P_t in tensor memory, O_t rescaled [2]
    uint64_t* b_o = b_p + 2;                  // O_t complete [2]
    uint64_t* b_tail = b_o + 2;               // the V block with the last key landed
    uint64_t* b_fix = b_tail + 1;             // its rows behind the last key are zero
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(b_fix + 1);
    volatile int* abort_f = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((2 * C::STAGES + 2 * SCN + 8) * 8 + 8 <= 512, "barrier area");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int split = blockIdx.x, h = blockIdx.y % a.kvh, rt = blockIdx.y / a.kvh, b = blockIdx.z;
    const Seq s = load_seq(a, b);
    if (!s.ok) {
        if (threadIdx.x == 0) raise_status(a.status, DS41_E_INDEX);
        return;
    }
    const int rows = s.n * a.G, r0 = rt * C::QT * 128;
    if (r0 >= rows) return;
    const int k0 = first_key(a, s) + split * a.chunk, k1 = min(s.len, k0 + a.chunk);
    if (k0 >= k1) return;
    const int n_blocks = (k1 - k0 + KB - 1) / KB;
    const int tail = (k1 - k0) - (n_blocks - 1) * KB;  // keys of the last block
    const int32_t* table = a.table + (int64_t)b * a.max_pages;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; i++) {
            mbar_init(&b_full[i], E4M3 ? 4 : 1);
            mbar_init(&b_empty[i], 1);
        }
        for (int i = 0; i < SCN; i++) {
            mbar_init(&b_sc[i], E4M3 ? 4 : 1);
            mbar_init(&b_sce[i], PAIR && rows - r0 > 128 ? 8 : 4);
        }
        for (int t = 0; t < 2; t++) {
            mbar_init(&b_s[t], 1);
            mbar_init(&b_p[t], 4);
            mbar_init(&b_o[t], 1);
        }
        mbar_init(b_tail, 1);
        mbar_init(b_fix, 1);
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
    // the queries, 128-byte swizzled; rows that do not exist are zero
    for (int x = threadIdx.x; x < C::QT * 128 * (D / 8); x += C::THREADS) {
        const int r = x / (D / 8), ch = x % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r0 + r < rows && ch * 8 < a.hd) {
            const int t = (r0 + r) / a.G;
            v = *reinterpret_cast<const uint4*>(
                a.q + (s.q0 + t) * a.q_tok + (h * a.G + (r0 + r) % a.G) * a.q_head + ch * 8);
        }
        if (E4M3) {  // D / 8 lanes have a row
            const uint32_t m2 = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                         __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
            uint32_t mb = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
            for (int off = D / 16; off > 0; off >>= 1)
                mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, off));
            const int e = query_exponent(mb);
            const float down = exp2f((float)-e);
            v = make_uint4(bf16x2_to_f16x2(v.x, down), bf16x2_to_f16x2(v.y, down),
                           bf16x2_to_f16x2(v.z, down), bf16x2_to_f16x2(v.w, down));
            if (ch == 0) reinterpret_cast<int8_t*>(sm + C::QE_OFF)[r] = (int8_t)e;
        }
        *reinterpret_cast<uint4*>(sm + C::Q_OFF + (r >> 7) * C::TILE + (ch >> 3) * C::BLK +
                                  (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
    }
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    constexpr uint32_t TM_S = 0, TM_O = 256;
    // stream t uses block j
    const int nt[2] = {PAIR ? n_blocks : (n_blocks + 1) / 2,
                       PAIR ? (rows - r0 > 128 ? n_blocks : 0) : n_blocks / 2};
    auto uses = [&](int t, int j) { return PAIR ? nt[t] > 0 : (j & 1) == t; };
    auto block_of = [&](int t, int i) { return PAIR ? i : 2 * i + t; };
    const int n_ring = 2 * n_blocks;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(E4M3 ? 72 : 88));
        if (warp == 0 && !E4M3) {
            // pages -> stages, and which keys are real
            bool ok = true;
            uint32_t armed[C::STAGES] = {};
            for (int e = 0; e < n_ring && ok; e++) {
                // ring entry e: K block or V block
                int j, kv;
                const int lead = min(C::LA, n_blocks);
                if (e < lead) {
                    j = e;
                    kv = 0;
                } else {
                    const int x = e - lead, both = 2 * max(0, n_blocks - C::LA);
                    kv = x < both ? (x & 1) ^ 1 : 1;
                    j = x < both ? (kv ? x / 2 : x / 2 + C::LA) : x - both / 2;
                }
                const int st = e % C::STAGES, use = e / C::STAGES;
                if (use > 0) ok = warp_wait(&b_empty[st], (use - 1) & 1, abort_f, a.status);
                if (!ok) break;
                const int key0 = k0 + j * KB;
                // lane i: the page of the 16 keys from key0 + 16 i on
                int64_t pg = -1;
                const int key = key0 + 16 * (lane & 7);
                if (key < k1) {
                    pg = table[key >> a.kv.page_shift];
                    if (pg < 0 || pg >= a.kv.n_pages) {
                        pg = -1;
                        if (kv == 0) raise_status(a.status, DS41_E_INDEX);
                    }
                }
                if (kv == 0) {
                    const int sl = j % SCN;
                    if (j >= SCN) ok = warp_wait(&b_sce[sl], ((j / SCN) - 1) & 1, abort_f, a.status);
                    if (!ok) break;
                    const uint32_t good = __ballot_sync(0xffffffffu, pg >= 0) & 0xffu;
                    if (lane < 4) {
                        uint32_t w = ((good >> (2 * lane)) & 1 ? 0xffffu : 0u) |
                                     ((good >> (2 * lane + 1)) & 1 ? 0xffff0000u : 0u);
                        w &= low_bits((int64_t)k1 - key0 - 32 * lane);
                        reinterpret_cast<uint32_t*>(sm + C::SC_OFF + sl * C::SC_BYTES)[lane] = w;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&b_sc[sl]);
                }
                if (lane == 0) mbar_arrive_expect_tx(&b_full[st], C::TILE);
                armed[st]++;
                __syncwarp();
                // a copy takes min(page, 128) rows of one page; a page that does
                // not exist reads as zeros (a coordinate past the tensor)
                const int per = min(a.kv.page, KB), copies = KB / per;
                const int src = lane < copies ? lane * per / 16 : 0;
                const int64_t cp = __shfl_sync(0xffffffffu, pg, src);
                if (lane < copies) {
                    const int64_t z = cp >= 0 ? cp * a.kvh + h : a.kv.n_pages * a.kvh;
                    const int off = (key0 + lane * per) & (a.kv.page - 1);
                    for (int x = 0; x < C::NB; x++)
                        tma_load_3d(sbase + C::KV_OFF + st * C::TILE + x * C::BLK +
                                        lane * per * 128,
                                    kv ? &map_v : &map_k, 64 * x, off, (int)z, &b_full[st]);
                }
            }
            for (int st = 0; st < C::STAGES; st++)
                if (armed[st]) drain_bar(&b_full[st], (armed[st] - 1) & 1, a.status);
        } else if (warp == 1) {
            constexpr uint32_t IDESC_S = E4M3 ? idesc_f16(128, KB, 0, 0) : idesc_bf16(128, KB, 0, 0);
            constexpr uint32_t IDESC_O = E4M3 ? idesc_f16(128, D, 0, 1) : idesc_bf16(128, D, 0, 1);
            const uint64_t qd = sdesc(sbase + C::Q_OFF, 16, 1024);
            const uint64_t kd = sdesc(sbase + C::KV_OFF, 16, 1024);
            const uint64_t vd = sdesc(sbase + C::KV_OFF, C::BLK, 1024);
            int done_p[2] = {0, 0};
            auto wait_entry = [&](int e) {
                const bool ok =
                    warp_wait(&b_full[e % C::STAGES], (e / C::STAGES) & 1, abort_f, a.status);
                tc_fence_after();
                return ok;
            };
            auto stage_off = [&](int e) { return ((e % C::STAGES) * C::TILE) >> 4; };
            auto scores = [&](int t, int e) {
                mma_scores<D, IDESC_S>(tmem + TM_S + 128 * t,
                                       qd + ((PAIR ? t * C::TILE : 0) >> 4), kd + stage_off(e));
                tc_commit(&b_s[t]);
            };
            bool ok = true;
            for (int j = 0; j < min(C::LA, n_blocks) && ok; j++) {
                ok = wait_entry(j);
                if (ok && elect_one()) {
#pragma unroll
                    for (int t = 0; t < 2; t++)
                        if (uses(t, j)) scores(t, j);
                    tc_commit(&b_empty[j % C::STAGES]);
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
                    ok = warp_wait(b_fix, 0, abort_f, a.status);
                    tc_fence_after();
                }
                bool have_k = false;
#pragma unroll
                for (int t = 0; t < 2; t++) {
                    const bool now = uses(t, j), next = more && uses(t, j + C::LA);
                    if (ok && now) {
                        ok = warp_wait(&b_p[t], done_p[t] & 1, abort_f, a.status);
                        done_p[t]++;
                        tc_fence_after();
                    }
                    if (ok && elect_one()) {
                        if (now) {
                            mma_output<D, IDESC_O>(tmem + TM_O + 128 * t, tmem + TM_S + 128 * t,
                                                   vd + stage_off(ev), done_p[t] > 1);
                            if (done_p[t] == nt[t]) tc_commit(&b_o[t]);
                        }
                        if (t == 1) tc_commit(&b_empty[ev % C::STAGES]);
                    }
                    __syncwarp();
                    if (ok && next) {
                        if (!have_k) ok = wait_entry(ek);
                        have_k = true;
                        if (ok && elect_one()) scores(t, ek);
                        __syncwarp();
                    }
                }
                if (ok && more && elect_one()) tc_commit(&b_empty[ek % C::STAGES]);
                __syncwarp();
            }
        } else if (warp == 2 && !E4M3 && tail < KB) {
            // the V rows behind the last key hold whatever an earlier user left
            const int ev = pos_v<C::LA>(n_blocks - 1, n_blocks);
            if (warp_wait(b_tail, 0, abort_f, a.status)) {
                uint8_t* v = sm + C::KV_OFF + (ev % C::STAGES) * C::TILE;
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
    } else if (E4M3 && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;\n");
        const int tid = threadIdx.x - 384;
        constexpr int PIECES = KB * D / 16 / 128;  // 16-code pieces a thread has of a tile
        // piece x of this thread: row and which of the row's pieces.  Eight lanes
        // take four pieces of a row and the other four of the next.
        auto piece = [&](int x, int& r, int& ch) {
            if (D == 128) {
                const int p = x * 16 + (tid >> 3);  // 0 .. 127: pair of rows, and which half
                const int odd = (tid >> 2) & 1;
                r = (p >> 1) * 2 + odd;
                ch = (tid & 3) + 4 * (odd ^ (p & 1));
            } else {
                r = x * 32 + (tid >> 2);
                ch = tid & 3;
            }
        };
        // entry e of the ring -> block j, K or V
        auto entry = [&](int e, int& j, int& kv) {
            const int lead = min(C::LA, n_blocks);
            if (e < lead) {
                j = e;
                kv = 0;
            } else {
                const int x = e - lead, both = 2 * max(0, n_blocks - C::LA);
                kv = x < both ? (x & 1) ^ 1 : 1;
                j = x < both ? (kv ? x / 2 : x / 2 + C::LA) : x - both / 2;
            }
        };
        // lane i < 8: the page of the 16 keys from key 16 i of entry e's block on
        auto pages = [&](int e) {
            int j, kv, pg = -1;
            entry(e, j, kv);
            const int key = k0 + j * KB + 16 * (lane & 7);
            if (e < n_ring && key < k1) pg = table[key >> a.kv.page_shift];
            return pg;
        };
        // what of an address does not change: the place in a group of 16 (32) keys
        int r_in, ch_in;
        piece(0, r_in, ch_in);
        const int in_group = r_in * a.hd + ch_in * 16;
        const bool in_row = ch_in * 16 < a.hd;
        const int64_t page_bytes = (int64_t)a.kv.page * a.hd, pages_bytes = page_bytes * a.kvh;
        constexpr int RPP = 128 / PIECES;  // rows from a piece to the next
        auto fetch = [&](int e, int pgs) {
            if (e < n_ring) {
                int j, kv;
                entry(e, j, kv);
                const uint32_t dst = sbase + C::C_OFF + (e % C::CODES) * C::CTILE + tid * 16;
                const uint8_t* src = (kv ? a.kv.v : a.kv.k) + h * page_bytes;
                const int key0 = k0 + j * KB;
#pragma unroll
                for (int x = 0; x < PIECES; x++) {
                    // (a piece's rows lie in one group of 16 keys, so in one page)
                    const int grp = (x * RPP + r_in) / 16;
                    const int pg = __shfl_sync(0xffffffffu, pgs, grp);
                    const int key = key0 + x * RPP + r_in;
                    const bool in = key < k1 && in_row && pg >= 0 && pg < a.kv.n_pages;
                    const int off = ((key0 + 16 * grp) & (a.kv.page - 1)) * a.hd +
                                    in_group + (x * RPP - 16 * grp) * a.hd;
                    cp_async16(dst + x * 2048, src + (in ? pg * pages_bytes + off : 0), in);
                }
            }
            cp_async_commit();
        };
        // the scales of block j's key tid, loaded a block ahead
        float ks = 0.0f, vs = 0.0f;
        bool real = false;
        auto scales = [&](int j) {
            const int key = k0 + j * KB + tid;
            ks = vs = 0.0f;
            real = false;
            if (j < n_blocks && key < k1) {
                const int64_t pg = table[key >> a.kv.page_shift];
                real = pg >= 0 && pg < a.kv.n_pages;
                if (real) {
                    const int64_t at = paged_row(a.kv, pg, h, key & (a.kv.page - 1));
                    ks = a.kv.ks[at];
                    vs = a.kv.vs[at];
                } else {
                    raise_status(a.status, DS41_E_INDEX);
                }
            }
        };
        for (int e = 0; e < C::CODES - 1; e++) fetch(e, pages(e));
        int ahead = pages(C::CODES - 1);
        scales(0);
        bool ok = true;
        for (int e = 0; e < n_ring && ok; e++) {
            int j, kv;
            entry(e, j, kv);
            fetch(e + C::CODES - 1, ahead);
            ahead = pages(e + C::CODES);
            const int st = e % C::STAGES, use = e / C::STAGES;
            if (use > 0) ok = warp_wait(&b_empty[st], (use - 1) & 1, abort_f, a.status);
            if (!ok) break;
            cp_async_wait<C::CODES - 1>();
            const uint8_t* from = sm + C::C_OFF + (e % C::CODES) * C::CTILE + tid * 16;
            uint8_t* to = sm + C::KV_OFF + st * C::TILE;
#pragma unroll
            for (int x = 0; x < PIECES; x++) {
                int r, ch;
                piece(x, r, ch);
                const uint4 w = *reinterpret_cast<const uint4*>(from + x * 2048);
                uint32_t out[8];
                e4m3x4_to_f16(w.x, out[0], out[1]);
                e4m3x4_to_f16(w.y, out[2], out[3]);
                e4m3x4_to_f16(w.z, out[4], out[5]);
                e4m3x4_to_f16(w.w, out[6], out[7]);
                uint8_t* row = to + (ch >> 2) * C::BLK + r * 128;
                const int c0 = (ch & 3) * 2;
                *reinterpret_cast<uint4*>(row + ((c0 ^ (r & 7)) << 4)) =
                    make_uint4(out[0], out[1], out[2], out[3]);
                *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (r & 7)) << 4)) =
                    make_uint4(out[4], out[5], out[6], out[7]);
            }
            asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&b_full[st]);
            if (kv == 0) {
                const int sl = j % SCN;
                if (j >= SCN) ok = warp_wait(&b_sce[sl], ((j / SCN) - 1) & 1, abort_f, a.status);
                if (!ok) break;
                float* sc = reinterpret_cast<float*>(sm + C::SC_OFF + sl * C::SC_BYTES);
                sc[8 + tid] = ks;
                sc[136 + tid] = vs;
                const uint32_t w = __ballot_sync(0xffffffffu, real);
                float vm = vs == vs ? fabsf(vs) : 0.0f;  // (a NaN scale asks for nothing)
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, off));
                if (lane == 0) {
                    reinterpret_cast<uint32_t*>(sc)[warp & 3] = w;
                    sc[4 + (warp & 3)] = vm;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&b_sc[sl]);
                scales(j + 1);
            }
        }
        cp_async_wait<0>();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(E4M3 ? 176 : 208));
        const int t = (warp - 4) >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tm_s = tmem + lanes + TM_S + 128 * t, tm_o = tmem + lanes + TM_O + 128 * t;
        const int row = r0 + (PAIR ? 128 * t : 0) + 32 * (warp & 3) + lane;
        const bool live = row < rows;
        const int tok = min(row, rows - 1) / a.G, head = h * a.G + min(row, rows - 1) % a.G;
        const RowView view = row_view(a, s, tok);
        float c = a.scale_log2;
        if (E4M3)
            c *= exp2f((float)reinterpret_cast<const int8_t*>(
                sm + C::QE_OFF)[(PAIR ? 128 * t : 0) + 32 * (warp & 3) + lane]);
        RowState st(E4M3);
        bool ok = true;
        for (int i = 0; i < nt[t]; i++) {
            const int j = block_of(t, i), sl = j % SCN;
            ok = warp_wait(&b_sc[sl], (j / SCN) & 1, abort_f, a.status) &&
                 warp_wait(&b_s[t], i & 1, abort_f, a.status);
            if (!ok) break;
            tc_fence_after();
            const float* sc = reinterpret_cast<const float*>(sm + C::SC_OFF + sl * C::SC_BYTES);
            const uint4 real = *reinterpret_cast<const uint4*>(sc);
            const int j0 = k0 + j * KB;
            const bool masked = (real.x & real.y & real.z & real.w) != 0xffffffffu ||
                                j0 + KB > view.pre || j0 <= view.lo;
            uint32_t vis[4] = {};
            // one choice for the warp: its lanes load from tensor memory together
            const bool any = __any_sync(0xffffffffu, masked);
            if (any) {
                vis[0] = real.x & seen_word(view, s.n, j0);
                vis[1] = real.y & seen_word(view, s.n, j0 + 32);
                vis[2] = real.z & seen_word(view, s.n, j0 + 64);
                vis[3] = real.w & seen_word(view, s.n, j0 + 96);
            }
            float vmax = 0.0f;
            if (E4M3) {
                const float4 v4 = *reinterpret_cast<const float4*>(sc + 4);
                vmax = fmaxf(fmaxf(v4.x, v4.y), fmaxf(v4.z, v4.w));
            }
            softmax_block<D, E4M3>(tm_s, tm_o, i > 0, any, vis, c, sc + 8, sc + 136, vmax, live,
                                   st);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&b_p[t]);
                mbar_arrive(&b_sce[sl]);
            }
        }
        if (nt[t] > 0 && ok) ok = warp_wait(&b_o[t], 0, abort_f, a.status);
        tc_fence_after();
        const int64_t at = (int64_t)(s.q0 + tok) * a.nh + head;
        const bool direct = PAIR && a.parts == 1;
        if (ok && (!PAIR || nt[t] > 0)) {
            // O is read by whole warps; a stream without blocks (ALT, one block)
            // still leaves its empty partial result
            const RowEnd end = direct ? row_end(st.reference(c), st.l,
                                                a.sink ? a.sink[head] : -INFINITY)
                                      : RowEnd{1.0f, 0.0f};
            const int64_t part = PAIR ? split : 2 * split + t;
            float* po = direct ? nullptr : a.part + (part * a.Tq * a.nh + at) * a.hd;
#pragma unroll 1
            for (int x = 0; x < D; x += 16) {
                uint32_t ov[16] = {};
                if (nt[t] > 0) {
                    tc_ld16(tm_o + x, ov);
                    tc_wait_ld();
                }
                if (!live || x >= a.hd) continue;
                if (direct) {
                    uint4* dst = reinterpret_cast<uint4*>(a.o + at * a.hd + x);
#pragma unroll
                    for (int e = 0; e < 16; e += 8)
                        dst[e / 8] = make_uint4(
                            bf16x2(u2f(ov[e]) * end.factor, u2f(ov[e + 1]) * end.factor),
                            bf16x2(u2f(ov[e + 2]) * end.factor, u2f(ov[e + 3]) * end.factor),
                            bf16x2(u2f(ov[e + 4]) * end.factor, u2f(ov[e + 5]) * end.factor),
                            bf16x2(u2f(ov[e + 6]) * end.factor, u2f(ov[e + 7]) * end.factor));
                } else {
#pragma unroll
                    for (int e = 0; e < 16; e += 4)
                        *reinterpret_cast<uint4*>(po + x + e) =
                            make_uint4(ov[e], ov[e + 1], ov[e + 2], ov[e + 3]);
                }
            }
            if (live && direct && a.lse) a.lse[at] = end.lse;
            if (live && !direct)
                a.part_ml[part * a.Tq * a.nh + at] =
                    make_float2(st.reference(c), st.l);
        }
    }

    pdl_trigger();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;\n" ::"r"(tmem)
                     : "memory");
}

namespace {

// [n_pages * kvh][page][hd] bf16, a box of 64 columns x min(page, 128) rows
int make_map_pages(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* ptr,
                   const PagedKv& kv) {
    cuuint64_t dims[3] = {(cuuint64_t)kv.hd, (cuuint64_t)kv.page, (cuuint64_t)(kv.n_pages * kv.kvh)};
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
int launch_many_as(const Args& a, int row_tiles, int64_t B, const char* name, cudaStream_t st) {
    using C = TcCfg<D, E4M3, PAIR>;
    CUtensorMap mk = {}, mv = {};
    if (!E4M3) {
        PFN_cuTensorMapEncodeTiled_v12000 enc;
        if (int rc = get_encode(&enc)) return rc;
        if (int rc = make_map_pages(enc, &mk, a.kv.k, a.kv)) return rc;
        if (int rc = make_map_pages(enc, &mv, a.kv.v, a.kv)) return rc;
    }
    auto kern = tree_many_kernel<D, E4M3, PAIR>;
    if (int rc = cuda_check(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 (int)C::SMEM),
                            name))
        return rc;
    const int splits = a.parts / a.per;
    return launch_pdl(kern, dim3((unsigned)splits, (unsigned)(a.kvh * row_tiles), (unsigned)B),
                      dim3(C::THREADS), C::SMEM, st, name, mk, mv, a);
}

}  // namespace

int launch_many(const Args& a, bool pair, int row_tiles, int64_t B, const char* name,
                cudaStream_t st) {
    const bool e = a.kv.ks != nullptr;
    if (a.hd <= 64)
        return e ? (pair ? launch_many_as<64, true, true>(a, row_tiles, B, name, st)
                         : launch_many_as<64, true, false>(a, row_tiles, B, name, st))
                 : (pair ? launch_many_as<64, false, true>(a, row_tiles, B, name, st)
                         : launch_many_as<64, false, false>(a, row_tiles, B, name, st));
    return e ? (pair ? launch_many_as<128, true, true>(a, row_tiles, B, name, st)
                     : launch_many_as<128, true, false>(a, row_tiles, B, name, st))
             : (pair ? launch_many_as<128, false, true>(a, row_tiles, B, name, st)
                     : launch_many_as<128, false, false>(a, row_tiles, B, name, st));
}

}  // namespace tree
}  // namespace ds41
