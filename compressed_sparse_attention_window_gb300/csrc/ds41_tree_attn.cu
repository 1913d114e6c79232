// ds41_tree_attn.cu - attention of drafted tokens (or of one token, plain
// decode) over a paged cache, few rows per key/value head.
//
// Mathematics.  One pass with a running reference m and sum l per row, in units
// of log2: t_j = scale log2(e) ks_j <q, k_j> (ks_j, vs_j: the row's scales, 1
// for bf16), p_j = 2^(t_j - m), l += p_j, O += (p_j vs_j) v_j, the weights
// rounded to 16 bits for the tensor cores.  m follows the running maximum lazily:
// it moves (and l and O are rescaled) when a score exceeds it by 2^8.  An e4m3
// cache runs on f16 products: its codes are exact in f16 (one instruction for
// two codes; bf16 takes four), the queries become f16 with an exponent per row,
// and l and O carry 2^-lr, which keeps the largest p_j vs_j that a row sees at 2^8 ..
// 2^15 of f16's range, and follows it alone: a row of values that weighs nothing may
// have any scale (RowState in ds41_softmax_tc.cuh).  The scales stay outside the
// products.
//
// Rows.  All queries of a (sequence, key/value head): tokens times the G heads
// that share it, 16 rows a CTA (the M of an m16n8k16 product).
//
// What bounds it.  Every cache row is read once for 16 rows of queries: HBM
// bandwidth, if enough is in flight and the conversion of codes keeps up.  So
// the key blocks of all sequences are dealt to the CTAs in equal runs (Share in
// ds41_tree.cuh), every warp streams its own 16-key groups (a group lies in one page, so
// its K and its V are one contiguous run each) through a private ring of
// cp.async stages, with no barrier between warps until the end, and the fragments
// are taken from shared memory with an order of hd (for Q K^T) and of the output
// columns (for P V) in which each lane's share is contiguous: the same order on
// both operands leaves the product unchanged.  The codes are widened in
// registers on the way into the products.  (48 sequences of one token over up to 8191
// keys, 64 heads of 128 over 8, e4m3: 95 us with the join, 5.0 TB/s.)
#include "ds41_few.cuh"
#include "ds41_internal.cuh"
#include "ds41_tree.cuh"

namespace ds41 {
namespace tree {

constexpr int WARPS = 4;
constexpr int NT = WARPS * 32;
using few::GROUP;
using few::k_piece;
using few::v_piece;
constexpr int BLOCK = WARPS * GROUP;  // keys of a block: a group for every warp

template <int HD, bool E4M3>
struct Cfg : few::Cfg<HD, E4M3> {
    static constexpr int SMEM = WARPS * Cfg::RING;
    static constexpr int MERGE = WARPS * 16 * Cfg::P * 4;  // the warps' results
    static constexpr int BYTES = SMEM > MERGE ? SMEM : MERGE;
};

template <int HD, bool E4M3>
__global__ void __launch_bounds__(NT, E4M3 ? 3 : 2) tree_few_kernel(const Args a) {
    pdl_wait();
    using C = Cfg<HD, E4M3>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t sh[2 * WARPS + 4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    Share share = find_share<NT>(a, sh, blockIdx.x == 0);
    Piece pc;
    while (next_piece(a, share, pc)) {
        const Seq s = pc.s;
        const int h = pc.h;
        const int rows = s.n * a.G;  // at most 16
        const int k0 = pc.key, k1 = min(s.len, k0 + pc.count * BLOCK);
        if (threadIdx.x == 0) note_ends(a, pc);

        uint8_t* ring = smem + warp * C::STAGES * C::STAGE;
        const int n_groups = (k1 - k0 + GROUP - 1) / GROUP;
        const int mine = (n_groups - warp + WARPS - 1) / WARPS;  // groups warp, warp + 4, ...
        const int32_t* table = a.table + (int64_t)pc.b * a.max_pages;
        unsigned bad = 0;  // stages whose page does not exist

        // what of the addresses does not change: a lane copies piece ch of the rows
        // r_in, r_in + RPI, ...
        constexpr int RPI = 32 / C::CH;
        const int r_in = lane / C::CH, ch = lane % C::CH;
        const int rb = a.hd * (E4M3 ? 1 : 2);  // bytes of a row in the cache
        const bool in_row = ch * 16 < rb;
        const int lane_off = r_in * rb + ch * 16, head_rows = h * a.kv.page;
        const uint32_t ring_u = smem_u32(ring);
        // (looked up a group ahead)
        auto page_of = [&](int i) {
            return i < mine ? table[(k0 + (i * WARPS + warp) * GROUP) >> a.kv.page_shift] : -1;
        };
        int page = page_of(0);
        auto fetch = [&](int i) {
            if (i < mine) {
                const int st = i % C::STAGES, j = k0 + (i * WARPS + warp) * GROUP;
                const int pg = page;
                page = page_of(i + 1);
                const bool ok = pg >= 0 && pg < a.kv.n_pages;
                if (!ok && lane == 0) raise_status(a.status, DS41_E_INDEX);
                bad = ok ? bad & ~(1u << st) : bad | (1u << st);
                const int64_t row =
                    ok ? (int64_t)pg * a.kvh * a.kv.page + (head_rows + (j & (a.kv.page - 1))) : 0;
                const uint32_t dst = ring_u + st * C::STAGE + lane / C::CH * C::RB;
                const uint8_t* kp = a.kv.k + row * rb + lane_off;
                const uint8_t* vp = a.kv.v + row * rb + lane_off;
                // rows behind the sequence's end are read as zeros, whatever they hold
                const int live = ok ? min(GROUP, k1 - j) : 0;
                if (live == GROUP && rb == C::RB) {
#pragma unroll
                    for (int x = 0; x < GROUP / RPI; x++) {
                        const int r = x * RPI + r_in;
                        const uint32_t to = dst + x * RPI * C::RB;
                        cp_async16(to + k_piece<C::RB>(r, ch) * 16, kp + x * RPI * C::RB, true);
                        cp_async16(to + GROUP * C::RB + v_piece<C::RB>(r, ch) * 16,
                                   vp + x * RPI * C::RB, true);
                    }
                } else {
#pragma unroll
                    for (int x = 0; x < GROUP / RPI; x++) {
                        const int r = x * RPI + r_in;
                        const uint32_t to = dst + x * RPI * C::RB;
                        const bool in = r < live && in_row;
                        const int off = in ? x * RPI * rb : -lane_off;
                        cp_async16(to + k_piece<C::RB>(r, ch) * 16, kp + off, in);
                        cp_async16(to + GROUP * C::RB + v_piece<C::RB>(r, ch) * 16, vp + off, in);
                    }
                }
                if (E4M3 && lane < 8) {
                    const float* src = (lane < 4 ? a.kv.ks : a.kv.vs) + row + (lane & 3) * 4;
                    cp_async16(ring_u + st * C::STAGE + 2 * GROUP * C::RB + lane * 16, src, ok);
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < C::STAGES - 1; i++) fetch(i);

        // the queries: rows g and g + 8 of the tile, hd in the order of the keys'
        // fragments (fp8: lane c owns bytes 16 c .. and 64 + 16 c .. of a row, bf16:
        // 16 c + 64 i ..; four elements a step)
        RowView view[2];
        uint32_t qf[HD / 16][4];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int r = min(g + 8 * i, rows - 1);
            const int t = r / a.G;
            view[i] = row_view(a, s, t);
            const uint16_t* qp = a.q + (s.q0 + t) * a.q_tok + (h * a.G + r % a.G) * a.q_head;
#pragma unroll
            for (int st = 0; st < HD / 16; st++) {
                const int d = E4M3 ? (c + 4 * (st / 4)) * 16 + 4 * (st % 4)
                                   : (c + 4 * (st / 2)) * 8 + 4 * (st % 2);
                const uint2 v =
                    d < a.hd ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0, 0);
                qf[st][i] = v.x;
                qf[st][i + 2] = v.y;
            }
        }
        float cr[2] = {a.scale_log2, a.scale_log2};
        if (E4M3) {
#pragma unroll
            for (int i = 0; i < 2; i++) {
                uint32_t m2 = 0;
#pragma unroll
                for (int st = 0; st < HD / 16; st++)
                    m2 = __vmaxu2(m2, __vmaxu2(qf[st][i] & 0x7fff7fffu,
                                               qf[st][i + 2] & 0x7fff7fffu));
                uint32_t mb = max(m2 & 0xffffu, m2 >> 16);  // four lanes have the row
                mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
                mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
                const int e = query_exponent(mb);
                const float down = exp2f((float)-e);
                cr[i] = fmaxf(cr[i] * exp2f((float)e), tc::SM_C_MIN);
#pragma unroll
                for (int st = 0; st < HD / 16; st++) {
                    qf[st][i] = bf16x2_to_f16x2(qf[st][i], down);
                    qf[st][i + 2] = bf16x2_to_f16x2(qf[st][i + 2], down);
                }
            }
        }
        // keys below `easy` are seen by both rows (and none lies at or before lo)
        const int easy = min(view[0].pre, view[1].pre);
        const int64_t lo = view[0].lo > view[1].lo ? view[0].lo : view[1].lo;

        float o[HD / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0, 0};
        float lr[2] = {0.0f, 0.0f}, vlim = 0.0f;
        float lim[2] = {tc::SM_RESCALE_LOG2, tc::SM_RESCALE_LOG2};
        float base[2] = {0.0f, 0.0f};  // c m + lr: what an exponent is reduced by
        for (int i = 0; i < mine; i++) {
            fetch(i + C::STAGES - 1);
            cp_async_wait<C::STAGES - 1>();
            __syncwarp();
            const int st = i % C::STAGES, j = k0 + (i * WARPS + warp) * GROUP;
            const uint8_t* kx = ring + st * C::STAGE;
            const uint8_t* vx = kx + GROUP * C::RB;
            const float* sx = reinterpret_cast<const float*>(kx + 2 * GROUP * C::RB);
            float sc[2][4] = {};
            // ---- S = Q K^T ----
#pragma unroll
            for (int x = 0; x < C::CH / 4; x++) {
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    const int r = n * 8 + g;
                    const uint4 kv = *reinterpret_cast<const uint4*>(
                        kx + r * C::RB + k_piece<C::RB>(r, c + 4 * x) * 16);
                    const uint32_t w[4] = {kv.x, kv.y, kv.z, kv.w};
                    if (E4M3) {
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const int q = 4 * x + e;
                            uint32_t lo16, hi16;
                            e4m3x4_to_f16(w[e], lo16, hi16);
                            mma_f16(sc[n], qf[q][0], qf[q][1], qf[q][2], qf[q][3], lo16, hi16);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            const int q = 2 * x + e;
                            mma_bf16(sc[n], qf[q][0], qf[q][1], qf[q][2], qf[q][3], w[2 * e],
                                     w[2 * e + 1]);
                        }
                    }
                }
            }
            // ---- softmax: this lane has rows g, g + 8 and keys 2c, 2c+1, 2c+8, 2c+9 ----
            float2 ks[2], vs[2];
            if (E4M3) {
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    ks[n] = *reinterpret_cast<const float2*>(sx + n * 8 + 2 * c);
                    vs[n] = *reinterpret_cast<const float2*>(sx + 16 + n * 8 + 2 * c);
#pragma unroll
                    for (int e = 0; e < 4; e++) sc[n][e] *= (e & 1) ? ks[n].y : ks[n].x;
                }
            }
            const bool masked = ((bad >> st) & 1) || j + GROUP > easy || j <= lo;
            if (masked) {
#pragma unroll
                for (int n = 0; n < 2; n++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (((bad >> st) & 1) ||
                            !seen(view[e >> 1], j + n * 8 + 2 * c + (e & 1), s.len))
                            sc[n][e] = -INFINITY;
            }
            float mx[2];
#pragma unroll
            for (int i2 = 0; i2 < 2; i2++)
                mx[i2] = fmaxf(fmaxf(sc[0][2 * i2], sc[0][2 * i2 + 1]),
                               fmaxf(sc[1][2 * i2], sc[1][2 * i2 + 1]));
            // (scales that no key needs may be NaN, which fmaxf skips, or anything: the look
            // at the group that follows is exact)
            float vm = 0.0f;
            if (E4M3)
                vm = fmaxf(fmaxf(fabsf(vs[0].x), fabsf(vs[0].y)),
                           fmaxf(fabsf(vs[1].x), fabsf(vs[1].y)));
            const bool look = (mx[0] - m[0]) * cr[0] > lim[0] || (mx[1] - m[1]) * cr[1] > lim[1];
            if (__any_sync(0xffffffffu, look || (E4M3 && vm > vlim))) {
                float up = 0.0f;
                if (E4M3) {
                    vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 1));
                    vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, 2));
                    up = tc::unit_limit(vm, vlim);
                }
#pragma unroll
                for (int i2 = 0; i2 < 2; i2++) {
                    float t = mx[i2], f = 1.0f;
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
                    t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2));
                    if (E4M3) {
                        // the largest weight of the keys that the row sees
                        float e = -INFINITY;
#pragma unroll
                        for (int n = 0; n < 2; n++) {
                            e = fmaxf(e, fmaf(sc[n][2 * i2] - t, cr[i2], tc::lg2(fabsf(vs[n].x))));
                            e = fmaxf(e,
                                      fmaf(sc[n][2 * i2 + 1] - t, cr[i2], tc::lg2(fabsf(vs[n].y))));
                        }
                        e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, 1));
                        e = fmaxf(e, __shfl_xor_sync(0xffffffffu, e, 2));
                        f = tc::move_unit(t, e, cr[i2], m[i2], lr[i2]);
                        lim[i2] = lr[i2] + up;
                    } else if ((t - m[i2]) * cr[i2] > tc::SM_RESCALE_LOG2) {
                        f = exp2f((m[i2] - t) * cr[i2]);
                        m[i2] = t;
                    }
                    l[i2] *= f;
#pragma unroll
                    for (int d = 0; d < HD / 8; d++) {
                        o[d][2 * i2] *= f;
                        o[d][2 * i2 + 1] *= f;
                    }
                    base[i2] = m[i2] == -INFINITY ? 0.0f : fmaf(m[i2], cr[i2], lr[i2]);
                }
            }
            uint32_t pf[4];
#pragma unroll
            for (int i2 = 0; i2 < 2; i2++) {
                float less = base[i2], at = 0.0f;
                if (fabsf(less) > 0x1p22f) {  // c m is rounded too far: the difference first
                    less = lr[i2];
                    at = m[i2];
                }
#pragma unroll
                for (int n = 0; n < 2; n++) {
                    const float p0 = ex2(fmaf(sc[n][2 * i2] - at, cr[i2], -less));
                    const float p1 = ex2(fmaf(sc[n][2 * i2 + 1] - at, cr[i2], -less));
                    l[i2] += p0 + p1;
                    if (!E4M3) {
                        pf[2 * n + i2] = bf16x2(p0, p1);
                        continue;
                    }
                    float w0 = p0 * vs[n].x, w1 = p1 * vs[n].y;
                    if (masked) {
                        // a row that is not seen weighs nothing, whatever its scale holds
                        if (sc[n][2 * i2] == -INFINITY) w0 = 0.0f;
                        if (sc[n][2 * i2 + 1] == -INFINITY) w1 = 0.0f;
                    }
                    pf[2 * n + i2] = tc::f16x2(w0, w1);
                }
            }
            // ---- O += P V: n-tile d holds the columns g HD/8 + d ----
            if (E4M3) {
                uint32_t w[4][HD / 32];
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int row = 2 * c + (r & 1) + 8 * (r >> 1);
                    if (HD == 128) {
                        *reinterpret_cast<uint4*>(w[r]) = *reinterpret_cast<const uint4*>(
                            vx + row * C::RB + v_piece<C::RB>(row, g) * 16);
                    } else {
                        *reinterpret_cast<uint2*>(w[r]) = *reinterpret_cast<const uint2*>(
                            vx + row * C::RB + v_piece<C::RB>(row, g >> 1) * 16 + (g & 1) * 8);
                    }
                }
#pragma unroll
                for (int d = 0; d < HD / 8; d += 2) {
                    // bytes d, d + 1 of two rows, side by side
                    const uint32_t sel = (d & 2) ? 0x7362u : 0x5140u;
                    uint32_t a0, a1, b0, b1;
                    e4m3x4_to_f16(__byte_perm(w[0][d / 4], w[1][d / 4], sel), a0, a1);
                    e4m3x4_to_f16(__byte_perm(w[2][d / 4], w[3][d / 4], sel), b0, b1);
                    mma_f16(o[d], pf[0], pf[1], pf[2], pf[3], a0, b0);
                    mma_f16(o[d + 1], pf[0], pf[1], pf[2], pf[3], a1, b1);
                }
            } else {
                uint32_t w[4][HD / 16];
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const int row = 2 * c + (r & 1) + 8 * (r >> 1);
#pragma unroll
                    for (int x = 0; x < HD / 64; x++)
                        *reinterpret_cast<uint4*>(w[r] + 4 * x) = *reinterpret_cast<const uint4*>(
                            vx + row * C::RB + v_piece<C::RB>(row, g * (HD / 64) + x) * 16);
                }
#pragma unroll
                for (int d = 0; d < HD / 8; d++) {
                    const uint32_t sel = (d & 1) ? 0x7632u : 0x5410u;
                    mma_bf16(o[d], pf[0], pf[1], pf[2], pf[3],
                             __byte_perm(w[0][d / 2], w[1][d / 2], sel),
                             __byte_perm(w[2][d / 2], w[3][d / 2], sel));
                }
            }
            __syncwarp();  // the stage is read before it is filled again
        }
        cp_async_wait<0>();
        __syncthreads();
        // ---- the warps' results: through shared memory, 16 rows ----
        constexpr int P = HD + 4;
        float* out = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            float* row = out + (warp * 16 + g + 8 * i) * P;
            if (c == 0) {
                row[HD] = m[i] == -INFINITY ? -INFINITY : fmaf(m[i], cr[i], lr[i]);
                row[HD + 1] = l[i];
            }
#pragma unroll
            for (int d = 0; d < HD / 8; d++) {
                row[2 * c * (HD / 8) + d] = o[d][2 * i];
                row[(2 * c + 1) * (HD / 8) + d] = o[d][2 * i + 1];
            }
        }
        __syncthreads();
        constexpr int PER = NT / 16;  // threads of a row
        const int r = threadIdx.x / PER, part = threadIdx.x % PER;
        if (r < rows) {
            float mm = -INFINITY, f[WARPS], ll = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; w++) mm = fmaxf(mm, out[(w * 16 + r) * P + HD]);
            const float base = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
            for (int w = 0; w < WARPS; w++) {
                f[w] = exp2f(out[(w * 16 + r) * P + HD] - base);
                ll += f[w] * out[(w * 16 + r) * P + HD + 1];
            }
            const int t = r / a.G, head = h * a.G + r % a.G;
            const int64_t at = (int64_t)(s.q0 + t) * a.nh + head;
            const bool whole = is_whole(pc);
            float inv = 1.0f;
            if (whole) {
                const tc::RowEnd end = tc::row_end(mm, ll, a.sink ? a.sink[head] : -INFINITY);
                inv = end.factor;
                if (a.lse && part == 0) a.lse[at] = end.lse;
            } else if (part == 0) {
                a.part_ml[slot_of(pc) * 16 + r] = make_float2(mm, ll);
            }
            float* po = a.part + (slot_of(pc) * 16 + r) * a.hd;
            for (int x = part * 4; x < a.hd; x += PER * 4) {
                float v[4] = {0, 0, 0, 0};
#pragma unroll
                for (int w = 0; w < WARPS; w++) {
                    const float4 ow = *reinterpret_cast<const float4*>(&out[(w * 16 + r) * P + x]);
                    v[0] += f[w] * ow.x;
                    v[1] += f[w] * ow.y;
                    v[2] += f[w] * ow.z;
                    v[3] += f[w] * ow.w;
                }
                if (whole)
                    *reinterpret_cast<uint2*>(a.o + at * a.hd + x) =
                        make_uint2(bf16x2(v[0] * inv, v[1] * inv), bf16x2(v[2] * inv, v[3] * inv));
                else
                    *reinterpret_cast<float4*>(po + x) = make_float4(v[0], v[1], v[2], v[3]);
            }
        }
        __syncthreads();  // the results are read before the rings are filled again
    }
    pdl_trigger();
}

// (token, head) by (token, head): where its unit was shared, the parts joined and
// the sink added.  PER warps take a row, every PER-th part each, eight parts' rows
// in flight: one where there are rows enough to fill the GPU (16384 rows of 4
// parts: 36 us with four warps each, 16 with one), four for a handful of rows of
// many parts (32 rows of 57: 27 us a call with one, 20 with four).
template <int PER>
__global__ void __launch_bounds__(NT) tree_join_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    __shared__ float4 acc[PER > 1 ? WARPS : 1][32];
    __shared__ float sums[WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int id = PER > 1 ? (int)blockIdx.x : (int)blockIdx.x * WARPS + warp;
    const Seq s = load_seq(a, blockIdx.y);
    if (!s.ok || id >= s.n * a.nh) return;
    const int t = id / a.nh, head = id % a.nh;
    const int r = t * a.G + head % a.G;
    const int2 ends =
        a.ends[((int64_t)blockIdx.y * a.kvh + head / a.G) * a.row_tiles + r / a.tile_rows];
    if (ends.x == ends.y) return;  // the one worker has written the output
    const int n = ends.y - ends.x + 1;
    // part 0 is its worker's slot 1, the others are slot 0
    const int64_t row0 = (2 * (int64_t)ends.x + 1) * a.tile_rows + r % a.tile_rows;
    const int64_t step = 2 * (int64_t)a.tile_rows, row1 = row0 - a.tile_rows;
    auto index = [&](int x) { return x == 0 ? row0 : row1 + x * step; };
    const int64_t at = (int64_t)s.q0 * a.nh + id;
    float m = -INFINITY, l = 0.0f;
    for (int x = lane; x < n; x += 32) m = fmaxf(m, a.part_ml[index(x)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
    const float base = m == -INFINITY ? 0.0f : m;
    float4 v = make_float4(0, 0, 0, 0);
    const bool mine = lane * 4 < a.hd;
#pragma unroll 8
    for (int x = PER > 1 ? warp : 0; x < n; x += PER) {
        const float2 ml = a.part_ml[index(x)];
        const float4 p =
            mine ? *reinterpret_cast<const float4*>(a.part + index(x) * a.hd + lane * 4)
                 : make_float4(0, 0, 0, 0);
        const float f = exp2f(ml.x - base);
        l += f * ml.y;
        v.x += f * p.x;
        v.y += f * p.y;
        v.z += f * p.z;
        v.w += f * p.w;
    }
    if (PER > 1) {
        acc[warp][lane] = v;
        if (lane == 0) sums[warp] = l;
        __syncthreads();
        if (warp > 0) return;
        l = sums[0];
#pragma unroll
        for (int w = 1; w < PER; w++) {
            l += sums[w];
            v.x += acc[w][lane].x;
            v.y += acc[w][lane].y;
            v.z += acc[w][lane].z;
            v.w += acc[w][lane].w;
        }
    }
    const tc::RowEnd end = tc::row_end(m, l, a.sink ? a.sink[head] : -INFINITY);
    if (a.lse && lane == 0) a.lse[at] = end.lse;
    if (mine)
        *reinterpret_cast<uint2*>(a.o + at * a.hd + lane * 4) =
            make_uint2(bf16x2(v.x * end.factor, v.y * end.factor),
                       bf16x2(v.z * end.factor, v.w * end.factor));
}

// The shape of a call's work: which kernel, its tiles and blocks, its workers.
// Up to 16 rows per key/value head the few-row kernel, three CTAs an SM (two on a
// bf16 cache, whose stages are twice as large); above, the tensor-core kernel,
// one CTA an SM (for 8 rows it takes 213 us where the few-row kernel takes 95, 48
// sequences of 8191 e4m3 keys).  Above 128 rows two tiles share a block's loads
// (4 sequences of 512 rows over 32768 keys: 217 us, 231 a tile at a time).  Never more
// workers than blocks at the longest lengths.
struct Plan {
    bool many;
    int block, align, tile_rows, row_tiles, workers;
    size_t part_bytes, ml_bytes, ends_bytes;
    size_t bytes() const { return part_bytes + ml_bytes + ends_bytes; }
};
Plan make_plan(int64_t B, int64_t max_q, int64_t max_len, int64_t nh, int64_t kvh, int64_t hd,
               int64_t window, int fmt, int sms) {
    Plan p;
    const int64_t rows = max_q * (nh / kvh);
    p.many = rows > 16;
    p.block = p.many ? 128 : BLOCK;
    p.align = p.many ? 128 : GROUP;
    p.tile_rows = !p.many ? 16 : rows > 128 ? 256 : 128;
    p.row_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
    int64_t len = max_len;
    if (window && window + max_q + p.align < len) len = window + max_q + p.align;
    const int64_t most = B * kvh * p.row_tiles * ((len + p.block - 1) / p.block);
    const int64_t want = (int64_t)sms * (p.many ? 1 : fmt == DS41_KV_E4M3 ? 3 : 2);
    p.workers = (int)(most < 1 ? 1 : most < want ? most : want);
    p.part_bytes = (size_t)p.workers * 2 * p.tile_rows * hd * 4;
    p.ml_bytes = (size_t)p.workers * 2 * p.tile_rows * 8;
    p.ends_bytes = (size_t)B * kvh * p.row_tiles * 8;
    return p;
}

int check_sizes(const char* name, int64_t B, int64_t Tq, int64_t max_q, int64_t max_len,
                int64_t window) {
    const int64_t lim = int64_t(1) << 31;
    DS41_REQUIRE(B >= 0 && B < 65536 && Tq >= 0 && Tq < lim && max_q >= 0 && max_q <= 256 &&
                     max_len >= 0 && max_len < lim / 2,
                 DS41_E_RANGE, "%s: B=%lld Tq=%lld max_q=%lld (at most 256) max_len=%lld", name,
                 (long long)B, (long long)Tq, (long long)max_q, (long long)max_len);
    DS41_REQUIRE(window == 0 || window >= max_q, DS41_E_ARG,
                 "%s: window=%lld is below max_q=%lld", name, (long long)window, (long long)max_q);
    return DS41_OK;
}

template <int HD, bool E4M3>
int launch_few(const Args& a, const char* name, cudaStream_t st) {
    constexpr int smem = Cfg<HD, E4M3>::BYTES;
    if (int rc = allow_smem<tree_few_kernel<HD, E4M3>>(smem, name)) return rc;
    return launch_pdl(tree_few_kernel<HD, E4M3>, dim3((unsigned)a.workers), dim3(NT), smem, st,
                      name, a);
}

}  // namespace tree
}  // namespace ds41

using namespace ds41;

extern "C" size_t ds41_tree_attn_workspace_bytes(int64_t B, int64_t Tq, int64_t max_q,
                                                 int64_t max_len, int64_t nh, int64_t kvh,
                                                 int64_t hd, int64_t window, int fmt) {
    const char* name = "ds41_tree_attn_workspace_bytes";
    if (check_heads(name, nh, kvh, hd, 1.0f, window) || check_cache_form(name, fmt, kvh, hd) ||
        tree::check_sizes(name, B, Tq, max_q, max_len, window) || B == 0 || Tq == 0 || max_q == 0)
        return 0;
    return tree::make_plan(B, max_q, max_len, nh, kvh, hd, finite_window(window), fmt,
                           sm_count_once())
        .bytes();
}

extern "C" int ds41_tree_attn_fwd(const ds41_bf16* q, int64_t q_tok, int64_t q_head,
                                  const void* k_cache, const void* v_cache, const float* k_scales,
                                  const float* v_scales, int fmt, int64_t n_pages, int64_t page,
                                  const int32_t* page_table, int64_t max_pages,
                                  const int32_t* lens, const int32_t* cu_q, const int64_t* mask,
                                  int64_t mask_words, int64_t B, int64_t Tq, int64_t max_q,
                                  int64_t max_len, int64_t nh, int64_t kvh, int64_t hd, float scale,
                                  int64_t window, const float* sink, ds41_bf16* o, float* lse,
                                  void* ws, size_t ws_bytes, ds41_stream_t stream) {
    const char* name = "ds41_tree_attn_fwd";
    if (int rc = check_heads(name, nh, kvh, hd, scale, window)) return rc;
    tree::Args a{};
    if (int rc = check_paged(name, k_cache, v_cache, k_scales, v_scales, fmt, n_pages, page, kvh,
                             hd, &a.kv))
        return rc;
    if (int rc = tree::check_sizes(name, B, Tq, max_q, max_len, window)) return rc;
    DS41_REQUIRE(max_pages >= 0 && max_pages < int64_t(1) << 31, DS41_E_RANGE, "%s: max_pages=%lld",
                 name, (long long)max_pages);
    DS41_REQUIRE(!mask || (mask_words >= 1 && mask_words <= 4 && max_q <= 64 * mask_words),
                 DS41_E_ARG, "%s: mask_words=%lld for max_q=%lld", name, (long long)mask_words,
                 (long long)max_q);
    window = finite_window(window);
    if (B == 0 || Tq == 0 || max_q == 0) return DS41_OK;
    DS41_REQUIRE(q && o && cu_q && lens && page_table, DS41_E_ARG,
                 "%s: q, page_table, lens, cu_q and o must be non-null", name);
    DS41_REQUIRE(aligned16(q) && aligned16(o) && aligned_to(cu_q, 4) && aligned_to(lens, 4) &&
                     aligned_to(page_table, 4) && aligned_to(mask, 8) && aligned_to(sink, 4) &&
                     aligned_to(lse, 4),
                 DS41_E_ARG, "%s: q and o must be 16-byte aligned", name);
    DS41_REQUIRE(good_strides(q_tok, q_head, hd), DS41_E_ARG,
                 "%s: strides must be multiples of 8 and at least hd", name);
    const int sms = sm_count_once();
    const tree::Plan pl = tree::make_plan(B, max_q, max_len, nh, kvh, hd, window, fmt, sms);
    DS41_REQUIRE(ws && aligned16(ws) && ws_bytes >= pl.bytes(), DS41_E_WORKSPACE,
                 "%s: needs %zu bytes of workspace, got %zu", name, pl.bytes(), ws ? ws_bytes : 0);
    a.q = q;
    a.q_tok = q_tok;
    a.q_head = q_head;
    a.table = page_table;
    a.max_pages = (int)max_pages;
    a.lens = lens;
    a.max_len = (int)max_len;
    a.mask = mask;
    a.mask_words = (int)mask_words;
    a.cu_q = cu_q;
    a.Tq = Tq;
    a.max_q = (int)max_q;
    a.nh = (int)nh;
    a.kvh = (int)kvh;
    a.hd = (int)hd;
    a.G = (int)(nh / kvh);
    a.scale_log2 = scale * tc::SM_LOG2E;
    a.window = window;
    a.sink = sink;
    a.o = o;
    a.lse = lse;
    a.B = (int)B;
    a.block = pl.block;
    a.align = pl.align < page ? pl.align : (int)page;
    a.tile_rows = pl.tile_rows;
    a.row_tiles = pl.row_tiles;
    a.workers = pl.workers;
    a.part = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(ws) + pl.part_bytes);
    a.ends = reinterpret_cast<int2*>(static_cast<uint8_t*>(ws) + pl.part_bytes + pl.ml_bytes);
    if (int rc = status_word(&a.status)) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    if (pl.many) {
        if (int rc = tree::launch_many(a, name, st)) return rc;
    } else {
        const bool e = fmt == DS41_KV_E4M3;
        if (int rc = e ? (hd <= 64 ? tree::launch_few<64, true>(a, name, st)
                                   : tree::launch_few<128, true>(a, name, st))
                       : (hd <= 64 ? tree::launch_few<64, false>(a, name, st)
                                   : tree::launch_few<128, false>(a, name, st)))
            return rc;
    }
    if (pl.workers == 1) return DS41_OK;  // every unit was whole
    const int64_t rows = max_q * nh;
    const bool few_rows = rows * B <= 8 * (int64_t)sms;
    return launch_pdl(few_rows ? tree::tree_join_kernel<tree::WARPS> : tree::tree_join_kernel<1>,
                      dim3((unsigned)(few_rows ? rows : (rows + tree::WARPS - 1) / tree::WARPS),
                           (unsigned)B),
                      dim3(tree::NT), 0, st, name, a);
}
