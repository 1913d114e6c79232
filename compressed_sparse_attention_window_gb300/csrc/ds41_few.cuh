// ds41_few.cuh - attention of 8 or 16 query rows over keys that arrive 16 at a time, by one
// warp.  (Tree attention's kernel of few rows has its stages and their layout from here.)
//
// A warp streams its own groups of 16 keys (a group lies in one page, so its K and its V
// are one contiguous run each) through a private ring of cp.async stages, and takes
// the fragments from shared memory with an order of hd (for Q K^T) and of the output
// columns (for P V) in which each lane's share is contiguous: the same order on both operands
// leaves the product unchanged.  e4m3 codes are widened in registers on the way into the
// products.  The mathematics is that of ds41_tree_attn.cu.
//
// The products are transposed: keys, and the columns of V, are the rows of a product,
// the queries its 8 columns, so that 8 rows leave no half of a tile to padding.  A lane has
// the keys g and g + 8 of a group and the queries 2 c and 2 c + 1 of each 8; the weights
// change places (movmatrix) on their way to being the other product's columns.
//
// Roundings.  The second product takes 16-bit operands: weights are rounded to bf16 beside bf16
// values (off by 2^-8 of themselves; the sum of the weights is taken before), to f16 in a row's
// own unit beside e4m3 ones.  (Outputs to 64 bits: bf16 2.3e-3 at most, with weights in 32 bits
// 1.7e-3, which is the outputs' own rounding; e4m3 1.7e-3, as with weights in 32 bits.)
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
// N times 8 query rows, and what they have gathered.
template <int HD, bool E4M3, int N>
struct Rows {
    using C = Cfg<HD, E4M3>;
    uint32_t qf[N][HD / 16][2];
    float cr[N][2];
    float o[N][HD / 16][4] = {}, m[N][2], l[N][2] = {}, lr[N][2] = {}, vlim = 0.0f, lim[N][2];
    float base[N][2] = {};  // c m + lr: what an exponent is reduced by

    // Row 8 n + g's queries, hd in the order of the keys' fragments (fp8: lane c owns bytes
    // 16 c .. and 64 + 16 c .. of a row, bf16: 16 c + 64 i ..; four elements a step); the
    // scale of their scores; e4m3: the queries as f16.
    __device__ __forceinline__ void query(int n, const uint16_t* qp, int hd, float scale_log2,
                                          int c) {
#pragma unroll
        for (int st = 0; st < HD / 16; st++) {
            const int d = E4M3 ? (c + 4 * (st / 4)) * 16 + 4 * (st % 4)
                               : (c + 4 * (st / 2)) * 8 + 4 * (st % 2);
            const uint2 v = d < hd ? *reinterpret_cast<const uint2*>(qp + d) : make_uint2(0, 0);
            qf[n][st][0] = v.x;
            qf[n][st][1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < 2; i++) {
            m[n][i] = -INFINITY;
            lim[n][i] = tc::SM_RESCALE_LOG2;
            cr[n][i] = scale_log2;
        }
        if (E4M3) {
            uint32_t m2 = 0;
#pragma unroll
            for (int st = 0; st < HD / 16; st++)
                m2 = __vmaxu2(m2,
                              __vmaxu2(qf[n][st][0] & 0x7fff7fffu, qf[n][st][1] & 0x7fff7fffu));
            uint32_t mb = max(m2 & 0xffffu, m2 >> 16);  // four lanes have the row
            mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));
            mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
            const int e = query_exponent(mb);
            const float down = exp2f((float)-e);
            const float mine = fmaxf(scale_log2 * exp2f((float)e), tc::SM_C_MIN);
#pragma unroll
            for (int i = 0; i < 2; i++)
                cr[n][i] = __shfl_sync(0xffffffffu, mine, (2 * c + i) * 4);
#pragma unroll
            for (int st = 0; st < HD / 16; st++) {
                qf[n][st][0] = bf16x2_to_f16x2(qf[n][st][0], down);
                qf[n][st][1] = bf16x2_to_f16x2(qf[n][st][1], down);
            }
        }
    }
    // One group, in the stage at kx; the keys from `live` on are not seen.
    __device__ __forceinline__ void group(const uint8_t* kx, int live, int g, int c) {
        const uint8_t* vx = kx + GROUP * C::RB;
        const float* sx = reinterpret_cast<const float*>(kx + 2 * GROUP * C::RB);
        // ---- S^T = K Q^T: keys g (0, 1) and g + 8 (2, 3), queries 2 c (0, 2) and 2 c + 1;
        // eight queries have two sums of each, so that products do not wait for one another ----
        float sc[N][4] = {}, s2[N][4] = {};
#pragma unroll
        for (int x = 0; x < C::CH / 4; x++) {
            uint32_t w[2][4];
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const int r = k * 8 + g;
                *reinterpret_cast<uint4*>(w[k]) = *reinterpret_cast<const uint4*>(
                    kx + r * C::RB + k_piece<C::RB>(r, c + 4 * x) * 16);
            }
#pragma unroll
            for (int e = 0; e < (E4M3 ? 4 : 2); e++) {
                const int q = (E4M3 ? 4 : 2) * x + e;
                uint32_t lo[2], hi[2];
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    if (E4M3) {
                        e4m3x4_to_f16(w[k][e], lo[k], hi[k]);
                    } else {
                        lo[k] = w[k][2 * e];
                        hi[k] = w[k][2 * e + 1];
                    }
                }
#pragma unroll
                for (int n = 0; n < N; n++) {
                    float* to = N == 1 && (e & 1) ? s2[n] : sc[n];
                    if (E4M3) mma_f16(to, lo[0], lo[1], hi[0], hi[1], qf[n][q][0], qf[n][q][1]);
                    else mma_bf16(to, lo[0], lo[1], hi[0], hi[1], qf[n][q][0], qf[n][q][1]);
                }
            }
        }
        // ---- softmax ----
        float ks[2] = {}, vs[2] = {};
        if (E4M3) {
#pragma unroll
            for (int k = 0; k < 2; k++) {
                ks[k] = sx[k * 8 + g];
                vs[k] = sx[16 + k * 8 + g];
            }
        }
        const bool masked = live < GROUP;
        bool look = false;
#pragma unroll
        for (int n = 0; n < N; n++) {
#pragma unroll
            for (int x = 0; x < 4; x++) {
                if (N == 1) sc[n][x] += s2[n][x];
                if (E4M3) sc[n][x] *= ks[x >> 1];
            }
            if (masked) {
#pragma unroll
                for (int x = 0; x < 4; x++)
                    if ((x >> 1) * 8 + g >= live) sc[n][x] = -INFINITY;
            }
#pragma unroll
            for (int i = 0; i < 2; i++)
                look |= (fmaxf(sc[n][i], sc[n][2 + i]) - m[n][i]) * cr[n][i] > lim[n][i];
        }
        // (scales that no key needs may be NaN, which fmaxf skips, or anything: the look
        // at the group that follows is exact)
        float vm = E4M3 ? fmaxf(fmaxf(0.0f, fabsf(vs[0])), fabsf(vs[1])) : 0.0f;
        if (__any_sync(0xffffffffu, look || (E4M3 && vm > vlim))) {
            float up = 0.0f;
            if (E4M3) {
                vm = max_keys(vm);
                up = tc::unit_limit(vm, vlim);
            }
#pragma unroll
            for (int n = 0; n < N; n++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float t = max_keys(fmaxf(sc[n][i], sc[n][2 + i]));
                    float f = 1.0f;
                    if (E4M3) {
                        // the largest weight of the keys that the row sees
                        float e = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 2; k++)
                            e = fmaxf(e, fmaf(sc[n][2 * k + i] - t, cr[n][i],
                                              tc::lg2(fabsf(vs[k]))));
                        f = tc::move_unit(t, max_keys(e), cr[n][i], m[n][i], lr[n][i]);
                        lim[n][i] = lr[n][i] + up;
                    } else if ((t - m[n][i]) * cr[n][i] > tc::SM_RESCALE_LOG2) {
                        f = exp2f((m[n][i] - t) * cr[n][i]);
                        m[n][i] = t;
                    }
                    l[n][i] *= f;
#pragma unroll
                    for (int d = 0; d < HD / 16; d++) {
                        o[n][d][i] *= f;
                        o[n][d][2 + i] *= f;
                    }
                    base[n][i] =
                        m[n][i] == -INFINITY ? 0.0f : fmaf(m[n][i], cr[n][i], lr[n][i]);
                }
        }
        uint32_t pf[N][2];
#pragma unroll
        for (int n = 0; n < N; n++) {
            float p[4];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                float less = base[n][i], at = 0.0f;
                if (fabsf(less) > 0x1p22f) {  // c m is rounded too far: the difference first
                    less = lr[n][i];
                    at = m[n][i];
                }
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const float e = ex2(fmaf(sc[n][2 * k + i] - at, cr[n][i], -less));
                    l[n][i] += e;
                    p[2 * k + i] = E4M3 ? e * vs[k] : e;
                    // a row that is not seen weighs nothing, whatever its scale holds
                    if (E4M3 && masked && sc[n][2 * k + i] == -INFINITY) p[2 * k + i] = 0.0f;
                }
            }
#pragma unroll
            for (int k = 0; k < 2; k++)
                pf[n][k] = transposed(E4M3 ? tc::f16x2(p[2 * k], p[2 * k + 1])
                                           : bf16x2(p[2 * k], p[2 * k + 1]));
        }
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
            uint32_t a0, a1, b0, b1;
            if (E4M3) {
                // bytes 2 d, 2 d + 1 of two rows, side by side
                const uint32_t sel = (d & 1) ? 0x7362u : 0x5140u;
                e4m3x4_to_f16(__byte_perm(w[0][d / 2], w[1][d / 2], sel), a0, a1);
                e4m3x4_to_f16(__byte_perm(w[2][d / 2], w[3][d / 2], sel), b0, b1);
            } else {
                a0 = __byte_perm(w[0][d], w[1][d], 0x5410u);
                a1 = __byte_perm(w[0][d], w[1][d], 0x7632u);
                b0 = __byte_perm(w[2][d], w[3][d], 0x5410u);
                b1 = __byte_perm(w[2][d], w[3][d], 0x7632u);
            }
#pragma unroll
            for (int n = 0; n < N; n++) {
                if (E4M3) mma_f16(o[n][d], a0, a1, b0, b1, pf[n][0], pf[n][1]);
                else mma_bf16(o[n][d], a0, a1, b0, b1, pf[n][0], pf[n][1]);
            }
        }
    }
    // The rows' results to out: 8 N rows of P floats, the reference (in log2) and the sum
    // behind a row's columns.
    __device__ __forceinline__ void put(float* out, int g, int c) {
        constexpr int P = C::P;
#pragma unroll
        for (int n = 0; n < N; n++)
#pragma unroll
            for (int i = 0; i < 2; i++) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1)
                    l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], x);
                float* row = out + (8 * n + 2 * c + i) * P;
                if (g == 0) {
                    row[HD] = m[n][i] == -INFINITY ? -INFINITY
                                                   : fmaf(m[n][i], cr[n][i], lr[n][i]);
                    row[HD + 1] = l[n][i];
                }
#pragma unroll
                for (int d = 0; d < HD / 16; d++) {
                    row[g * (HD / 8) + 2 * d] = o[n][d][i];
                    row[g * (HD / 8) + 2 * d + 1] = o[n][d][2 + i];
                }
            }
    }
};

}  // namespace few
}  // namespace ds41
