// ds41_few.cuh - attention of up to 16 query rows over keys that arrive 16 at a time, by one
// warp: shared by the kernels of few rows per key/value head (trees of drafted tokens,
// picked blocks of a cache).
//
// A warp streams its own groups of 16 keys (a group lies in one page, so its K and its V
// are one contiguous run each) through a private ring of cp.async stages, and takes
// the fragments from shared memory with an order of hd (for Q K^T) and of the output
// columns (for P V) in which each lane's share is contiguous: the same order on both operands
// leaves the product unchanged.  e4m3 codes are widened in registers on the way into the
// products.  The mathematics stands in ds41_tree_attn.cu.
#pragma once

#include "ds41_softmax_tc.cuh"

namespace ds41 {
namespace few {

using tc::bf16x2;
using tc::ex2;

constexpr int GROUP = 16;  // keys of a group

template <int HD, bool E4M3>
struct Cfg {
    static constexpr int RB = HD * (E4M3 ? 1 : 2);          // bytes of a row's slot
    static constexpr int STAGES = RB == 256 ? 3 : 4;
    static constexpr int STAGE = 2 * GROUP * RB + 2 * GROUP * 4;  // K, V, their scales
    static constexpr int RING = STAGES * STAGE;              // of a warp
    static constexpr int CH = RB / 16;                       // 16-byte pieces of a row
    static constexpr int P = HD + 4;                         // floats of a row's result
};

// Where piece ch of row r lies: rows that one quarter-warp reads together fall
// into different banks.
template <int RB>
__device__ __forceinline__ int k_piece(int r, int ch) {
    return RB == 64 ? ch : ch ^ ((r & 1) << 2);
}
template <int RB>
__device__ __forceinline__ int v_piece(int r, int ch) {
    const int c = (r >> 1) & 3;
    return RB == 64    ? ch ^ ((c & 1) << 1)
           : RB == 128 ? ch ^ (c << 1)
                       : ch ^ ((c & 1) | ((c >> 1) << 2));
}

// A lane's part of the copies of a group's K and V (and scales) into a stage: piece ch of the
// rows r_in, r_in + RPI, ...  What of the addresses does not change is worked out once.
template <int HD, bool E4M3>
struct Copier {
    using C = Cfg<HD, E4M3>;
    static constexpr int RPI = 32 / C::CH;
    int r_in, ch, rb, lane_off;
    bool in_row;
    __device__ __forceinline__ Copier(int hd, int lane)
        : r_in(lane / C::CH), ch(lane % C::CH), rb(hd * (E4M3 ? 1 : 2)) {
        in_row = ch * 16 < rb;
        lane_off = r_in * rb + ch * 16;
    }
    // row: the group's first in the cache; rows from `live` on are read as zeros, whatever
    // they hold; ok: the page exists (its scales may be read)
    __device__ __forceinline__ void copy(uint32_t stage, const PagedKv& kv, int64_t row, int live,
                                         bool ok, int lane) const {
        const uint32_t dst = stage + r_in * C::RB;
        const uint8_t* kp = kv.k + row * rb + lane_off;
        const uint8_t* vp = kv.v + row * rb + lane_off;
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
            const float* src = (lane < 4 ? kv.ks : kv.vs) + row + (lane & 3) * 4;
            cp_async16(stage + 2 * GROUP * C::RB + lane * 16, src, ok);
        }
    }
};

// A lane's part of 16 rows (rows g = lane / 4 and g + 8): their queries, and what they have
// gathered.
template <int HD, bool E4M3>
struct Rows {
    using C = Cfg<HD, E4M3>;
    uint32_t qf[HD / 16][4];
    float cr[2];
    float o[HD / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0, 0};
    float lr[2] = {0.0f, 0.0f}, vlim = 0.0f;
    float lim[2] = {tc::SM_RESCALE_LOG2, tc::SM_RESCALE_LOG2};
    float base[2] = {0.0f, 0.0f};  // c m + lr: what an exponent is reduced by

    // Row g + 8 i's queries, hd in the order of the keys' fragments (fp8: lane c owns bytes
    // 16 c .. and 64 + 16 c .. of a row, bf16: 16 c + 64 i ..; four elements a step)
    __device__ __forceinline__ void query(int i, const uint16_t* qp, int hd, int c) {
#pragma unroll
        for (int st = 0; st < HD / 16; st++) {
            const int d = E4M3 ? (c + 4 * (st / 4)) * 16 + 4 * (st % 4)
                               : (c + 4 * (st / 2)) * 8 + 4 * (st % 2);
            const uint2 v = d < hd ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0, 0);
            qf[st][i] = v.x;
            qf[st][i + 2] = v.y;
        }
    }
    // Both rows are there: the scale of their scores; e4m3: the queries as f16.
    __device__ __forceinline__ void start(float scale_log2) {
        cr[0] = cr[1] = scale_log2;
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
    }
    // One group, in the stage at kx.  masked: some key is not seen by some row; sees(i, x):
    // whether row g + 8 i sees key x of the group.
    template <typename Sees>
    __device__ __forceinline__ void group(const uint8_t* kx, bool masked, Sees sees, int g,
                                          int c) {
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
        if (masked) {
#pragma unroll
            for (int n = 0; n < 2; n++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (!sees(e >> 1, n * 8 + 2 * c + (e & 1))) sc[n][e] = -INFINITY;
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
    }
    // The rows' results to out: 16 rows of P floats, the reference (in log2) and the sum
    // behind a row's columns.
    __device__ __forceinline__ void put(float* out, int g, int c) {
        constexpr int P = C::P;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
            l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            float* row = out + (g + 8 * i) * P;
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
    }
};

// The same for up to 8 rows, the products transposed: keys, and the columns of V, are the rows of
// a product, the queries its 8 columns.  No half of a tile is padding then, and scores,
// queries and outputs take half the registers.  A lane has the keys g and g + 8 of a group
// and the queries 2 c and 2 c + 1; the weights change places (movmatrix) on their way to
// being the other product's columns.  Fragments and their orders are those of Rows.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {  // 8 x 8 of 16 bits
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// over the lanes that have the same queries
__device__ __forceinline__ float max_keys(float x) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
template <int HD, bool E4M3>
struct Rows8 {
    using C = Cfg<HD, E4M3>;
    uint32_t qf[HD / 16][2];
    float cr[2];
    float o[HD / 16][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0, 0};
    float lr[2] = {0.0f, 0.0f}, vlim = 0.0f;
    float lim[2] = {tc::SM_RESCALE_LOG2, tc::SM_RESCALE_LOG2};
    float base[2] = {0.0f, 0.0f};

    // row g's queries, in the order of the keys' fragments; their scale
    __device__ __forceinline__ void query(const uint16_t* qp, int hd, float scale_log2, int c) {
#pragma unroll
        for (int st = 0; st < HD / 16; st++) {
            const int d = E4M3 ? (c + 4 * (st / 4)) * 16 + 4 * (st % 4)
                               : (c + 4 * (st / 2)) * 8 + 4 * (st % 2);
            const uint2 v = d < hd ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0, 0);
            qf[st][0] = v.x;
            qf[st][1] = v.y;
        }
        cr[0] = cr[1] = scale_log2;
        if (E4M3) {
            uint32_t m2 = 0;
#pragma unroll
            for (int st = 0; st < HD / 16; st++)
                m2 = __vmaxu2(m2, __vmaxu2(qf[st][0] & 0x7fff7fffu, qf[st][1] & 0x7fff7fffu));
            uint32_t mb = max(m2 & 0xffffu, m2 >> 16);  // four lanes have the row
            mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
            mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
            const int e = query_exponent(mb);
            const float down = exp2f((float)-e);
            const float mine = fmaxf(scale_log2 * exp2f((float)e), tc::SM_C_MIN);
#pragma unroll
            for (int i = 0; i < 2; i++) cr[i] = __shfl_sync(0xffffffffu, mine, (2 * c + i) * 4);
#pragma unroll
            for (int st = 0; st < HD / 16; st++) {
                qf[st][0] = bf16x2_to_f16x2(qf[st][0], down);
                qf[st][1] = bf16x2_to_f16x2(qf[st][1], down);
            }
        }
    }
    // One group, in the stage at kx; the keys from `live` on are not seen.
    __device__ __forceinline__ void group(const uint8_t* kx, int live, int g, int c) {
        const uint8_t* vx = kx + GROUP * C::RB;
        const float* sx = reinterpret_cast<const float*>(kx + 2 * GROUP * C::RB);
        // ---- S^T = K Q^T: keys g (0, 1) and g + 8 (2, 3), queries 2 c (0, 2) and 2 c + 1 ----
        float sc[4] = {}, s2[4] = {};
#pragma unroll
        for (int x = 0; x < C::CH / 4; x++) {
            uint32_t w[2][4];
#pragma unroll
            for (int n = 0; n < 2; n++) {
                const int r = n * 8 + g;
                *reinterpret_cast<uint4*>(w[n]) = *reinterpret_cast<const uint4*>(
                    kx + r * C::RB + k_piece<C::RB>(r, c + 4 * x) * 16);
            }
            if (E4M3) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int q = 4 * x + e;
                    uint32_t lo[2], hi[2];
                    e4m3x4_to_f16(w[0][e], lo[0], hi[0]);
                    e4m3x4_to_f16(w[1][e], lo[1], hi[1]);
                    mma_f16((e & 1) ? s2 : sc, lo[0], lo[1], hi[0], hi[1], qf[q][0], qf[q][1]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int q = 2 * x + e;
                    mma_bf16(e ? s2 : sc, w[0][2 * e], w[1][2 * e], w[0][2 * e + 1],
                             w[1][2 * e + 1], qf[q][0], qf[q][1]);
                }
            }
        }
#pragma unroll
        for (int x = 0; x < 4; x++) sc[x] += s2[x];
        // ---- softmax ----
        float vs[2] = {};
        if (E4M3) {
#pragma unroll
            for (int n = 0; n < 2; n++) {
                const float ks = sx[n * 8 + g];
                vs[n] = sx[16 + n * 8 + g];
                sc[2 * n] *= ks;
                sc[2 * n + 1] *= ks;
            }
        }
        const bool masked = live < GROUP;
        if (masked) {
#pragma unroll
            for (int n = 0; n < 2; n++)
                if (n * 8 + g >= live) sc[2 * n] = sc[2 * n + 1] = -INFINITY;
        }
        const float mx[2] = {fmaxf(sc[0], sc[2]), fmaxf(sc[1], sc[3])};
        // (scales that no key needs may be NaN, which fmaxf skips, or anything: the look
        // at the group that follows is exact)
        float vm = E4M3 ? fmaxf(fmaxf(0.0f, fabsf(vs[0])), fabsf(vs[1])) : 0.0f;
        const bool look = (mx[0] - m[0]) * cr[0] > lim[0] || (mx[1] - m[1]) * cr[1] > lim[1];
        if (__any_sync(0xffffffffu, look || (E4M3 && vm > vlim))) {
            float up = 0.0f;
            if (E4M3) {
                vm = max_keys(vm);
                up = tc::unit_limit(vm, vlim);
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const float t = max_keys(mx[i]);
                float f = 1.0f;
                if (E4M3) {
                    // the largest weight of the keys that the row sees
                    float e = -INFINITY;
#pragma unroll
                    for (int n = 0; n < 2; n++)
                        e = fmaxf(e, fmaf(sc[2 * n + i] - t, cr[i], tc::lg2(fabsf(vs[n]))));
                    f = tc::move_unit(t, max_keys(e), cr[i], m[i], lr[i]);
                    lim[i] = lr[i] + up;
                } else if ((t - m[i]) * cr[i] > tc::SM_RESCALE_LOG2) {
                    f = exp2f((m[i] - t) * cr[i]);
                    m[i] = t;
                }
                l[i] *= f;
#pragma unroll
                for (int d = 0; d < HD / 16; d++) {
                    o[d][i] *= f;
                    o[d][2 + i] *= f;
                }
                base[i] = m[i] == -INFINITY ? 0.0f : fmaf(m[i], cr[i], lr[i]);
            }
        }
        float p[4];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            float less = base[i], at = 0.0f;
            if (fabsf(less) > 0x1p22f) {  // c m is rounded too far: the difference first
                less = lr[i];
                at = m[i];
            }
#pragma unroll
            for (int n = 0; n < 2; n++) {
                const float e = ex2(fmaf(sc[2 * n + i] - at, cr[i], -less));
                l[i] += e;
                p[2 * n + i] = E4M3 ? e * vs[n] : e;
                // a row that is not seen weighs nothing, whatever its scale holds
                if (E4M3 && masked && sc[2 * n + i] == -INFINITY) p[2 * n + i] = 0.0f;
            }
        }
        uint32_t pf[2];
#pragma unroll
        for (int n = 0; n < 2; n++)
            pf[n] = transposed(E4M3 ? tc::f16x2(p[2 * n], p[2 * n + 1])
                                    : bf16x2(p[2 * n], p[2 * n + 1]));
        // ---- O^T += V^T P^T: rows g and g + 8 of tile d are columns g HD/8 + 2 d, + 1 ----
        uint32_t w[4][C::CH / 2];
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const int row = 2 * c + (r & 1) + 8 * (r >> 1);
            if (C::RB == 64) {
                *reinterpret_cast<uint2*>(w[r]) = *reinterpret_cast<const uint2*>(
                    vx + row * C::RB + v_piece<C::RB>(row, g >> 1) * 16 + (g & 1) * 8);
            } else {
#pragma unroll
                for (int x = 0; x < C::RB / 128; x++)
                    *reinterpret_cast<uint4*>(w[r] + 4 * x) = *reinterpret_cast<const uint4*>(
                        vx + row * C::RB + v_piece<C::RB>(row, g * (C::RB / 128) + x) * 16);
            }
        }
#pragma unroll
        for (int d = 0; d < HD / 16; d++) {
            if (E4M3) {
                // bytes 2 d, 2 d + 1 of two rows, side by side
                const uint32_t sel = (d & 1) ? 0x7362u : 0x5140u;
                uint32_t a0, a1, b0, b1;
                e4m3x4_to_f16(__byte_perm(w[0][d / 2], w[1][d / 2], sel), a0, a1);
                e4m3x4_to_f16(__byte_perm(w[2][d / 2], w[3][d / 2], sel), b0, b1);
                mma_f16(o[d], a0, a1, b0, b1, pf[0], pf[1]);
            } else {
                mma_bf16(o[d], __byte_perm(w[0][d], w[1][d], 0x5410u),
                         __byte_perm(w[0][d], w[1][d], 0x7632u),
                         __byte_perm(w[2][d], w[3][d], 0x5410u),
                         __byte_perm(w[2][d], w[3][d], 0x7632u), pf[0], pf[1]);
            }
        }
    }
    // The rows' results to out, as Rows::put, 8 of them.
    __device__ __forceinline__ void put(float* out, int g, int c) {
        constexpr int P = C::P;
#pragma unroll
        for (int i = 0; i < 2; i++) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
            float* row = out + (2 * c + i) * P;
            if (g == 0) {
                row[HD] = m[i] == -INFINITY ? -INFINITY : fmaf(m[i], cr[i], lr[i]);
                row[HD + 1] = l[i];
            }
#pragma unroll
            for (int d = 0; d < HD / 16; d++) {
                row[g * (HD / 8) + 2 * d] = o[d][i];
                row[g * (HD / 8) + 2 * d + 1] = o[d][2 + i];
            }
        }
    }
};

}  // namespace few
}  // namespace ds41
