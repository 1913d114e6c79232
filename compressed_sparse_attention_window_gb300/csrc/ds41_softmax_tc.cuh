// ds41_softmax_tc.cuh - one block of 128 keys of a softmax whose scores and
// output live in tensor memory: shared by the tensor-core kernels of the dense
// attention (packed prompts, trees over a paged cache).
#pragma once

#include "ds41_dense.cuh"
#include "ds41_tc.cuh"

namespace ds41 {
namespace tc {

constexpr float SM_LOG2E = 1.4426950408889634f;
constexpr float SM_LN2 = 0.6931471805599453f;
// Plain form (bf16 weights): the reference of a row moves when a block's maximum
// exceeds it by this power of two.
constexpr float SM_RESCALE_LOG2 = 8.0f;
// Scaled form (f16 weights p_j vs_j): a row's unit is chosen so that the largest weight
// is 2^8 of it, and moves when one would pass 2^15 (f16 ends at 2^16); f16's smallest
// step is then 2^-32 of the largest weight at most.  No unit is below 2^-96 of the
// largest p_j, which keeps the sum of the p_j in that unit inside f32.
constexpr float SM_WEIGHT_LOG2 = 8.0f;
constexpr float SM_WEIGHT_MOVE_LOG2 = 15.0f;
constexpr float SM_UNIT_MIN_LOG2 = -96.0f;
constexpr float SM_UNIT_MOVE_LOG2 = 100.0f;
// The scale of a row's scores with its queries' exponent in it is not below this: at 0 a
// masked score of -inf would be NaN.  (Scores that small are 0 beside each other.)
constexpr float SM_C_MIN = 0x1p-126f;

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
// idesc_bf16 with f16 A and B: formats 0 in place of 1.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
    return idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}
// D += A B with A in tensor memory (bf16, two per column, lane = row)
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t acc) {
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
// x, which all lanes of the warp hold alike, in a form that says so: what is derived
// from it (loop bounds, stage numbers, descriptors) may live in uniform registers,
// where the MMAs want their operands.  (Read back from shared memory it would not:
// 16384-token prompt 1595 us, with this 1380 at the time.)
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// One lane of a converged warp, the same one every time.  The warps that issue
// MMAs run their loops as whole warps and elect a lane around each sequence: a
// loop that one lane runs alone cannot keep its descriptors in uniform registers,
// and every MMA then waits for them to be moved there (measured: 144 cycles an
// MMA instead of 64, twice the time of a long prompt).
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(r));
    return r != 0;
}
// A whole warp's bounded wait: all of its lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_f,
                                          unsigned int* status) {
    return __all_sync(0xffffffffu, wait_bar(bar, parity, abort_f, status));
}
// The two words of a descriptor of 64-column blocks of [rows][128 bytes], 128-byte
// swizzled: the upper one is the same for all of them (stride 1024 bytes); the
// lower one holds the address and the leading stride (1 for K-major, the distance
// of two blocks for N-major).
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead) {
    return (saddr >> 4) | ((lead >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
    return ((uint64_t)DESC_HI << 32) | lo;
}
// S = Q K^T for 128 rows and 128 keys, both K-major.  (The empty statement keeps the
// compiler from computing all of the steps' descriptors ahead of the key loop: they
// would not fit the issuing warp's registers.)
template <int D, uint32_t IDESC>
__device__ __forceinline__ void mma_scores(uint32_t d, uint32_t q, uint32_t k) {
    asm volatile("" : "+r"(q), "+r"(k));
#pragma unroll
    for (int x = 0; x < D / 16; x++) {
        constexpr uint32_t BLK = 128 * 128;
        const uint32_t off = ((x >> 2) * BLK + (x & 3) * 32) >> 4;
        tc_mma(d, desc_of(q + off), desc_of(k + off), IDESC, x > 0);
    }
}
// O (+)= P V, P in tensor memory, V [128 keys][D] N-major
template <int D, uint32_t IDESC>
__device__ __forceinline__ void mma_output(uint32_t d, uint32_t p, uint32_t v, bool acc) {
    asm volatile("" : "+r"(p), "+r"(v));
#pragma unroll
    for (int x = 0; x < 8; x++)
        tc_mma_ts(d, p + 8 * x, desc_of(v + ((x * 2048) >> 4)), IDESC, acc || x > 0);
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float u2f(uint32_t x) { return __uint_as_float(x); }

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The state of a row: the reference m (in units of its scores), the sum l of
// 2^(c (S - m) - lr).  For scaled values 2^(c m + lr) is the row's unit: the largest
// p_j vs_j of the keys that the row sees, whatever the scales of the others, is 2^8 of
// it or more (see above).  Both O and l are in that unit, so nothing has to be undone
// at the end.
struct RowState {
    float m = -INFINITY, l = 0.0f, lr = 0.0f;
    __device__ __forceinline__ float reference(float c) const {  // in log2 units
        return m == -INFINITY ? -INFINITY : fmaf(m, c, lr);
    }
};
// What scores may rise above m, in log2 units less lr, before the unit has to be looked at,
// as long as no value scale is above vlim, twice vmax's next power of two.  (For groups of
// a few keys: their largest scales are compared, 48 single tokens 94.9 us; turned into a
// limit for every group 97.2.)
__device__ __forceinline__ float unit_limit(float vmax, float& vlim) {
    const float log2_vlim = (float)((int)(__float_as_uint(vmax) >> 23) - 125);
    vlim = ex2(log2_vlim);
    return fminf(SM_WEIGHT_MOVE_LOG2 - log2_vlim, SM_UNIT_MOVE_LOG2);
}
// The same for one block whose largest scale is vmax.
__device__ __forceinline__ float unit_limit(float vmax) {
    const float log2_vmax = (float)((int)(__float_as_uint(vmax) >> 23) - 126);
    return fminf(SM_WEIGHT_MOVE_LOG2 - log2_vmax, SM_UNIT_MOVE_LOG2);
}
// Moves a row's unit if a block asks for it: top is the largest score that the row sees
// there, e the largest log2 of a weight against top's own p.  Returns the factor for
// what is in the old unit.
__device__ __forceinline__ float move_unit(float top, float e, float c, float& m, float& lr) {
    const float rise = (top - m) * c;  // (-inf - -inf is NaN: no move)
    if (!(rise + e > lr + SM_WEIGHT_MOVE_LOG2 || rise > lr + SM_UNIT_MOVE_LOG2)) return 1.0f;
    const float to_m = fmaxf(m, top);
    const float to =
        fmaxf((top - to_m) * c + fminf(e, 128.0f) - SM_WEIGHT_LOG2, SM_UNIT_MIN_LOG2);
    const float f = ex2((m - to_m) * c + lr - to);
    m = to_m;
    lr = to;
    return f;
}

__device__ __forceinline__ void tc_ld8(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

// 32 scores of a row, scaled by ks, with those that are not seen at -inf.
template <bool SCALED, bool MASKED>
__device__ __forceinline__ void prepare32(uint32_t (&s)[32], const float* ks, uint32_t vis) {
    if (SCALED) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
            const float4 k4 = *reinterpret_cast<const float4*>(ks + e);
            float a, b;
            unf2(mul2(f2(u2f(s[e]), u2f(s[e + 1])), f2(k4.x, k4.y)), a, b);
            s[e] = __float_as_uint(a);
            s[e + 1] = __float_as_uint(b);
            unf2(mul2(f2(u2f(s[e + 2]), u2f(s[e + 3])), f2(k4.z, k4.w)), a, b);
            s[e + 2] = __float_as_uint(a);
            s[e + 3] = __float_as_uint(b);
        }
    }
    if (MASKED) {
#pragma unroll
        for (int e = 0; e < 32; e++)
            if (!((vis >> e) & 1)) s[e] = 0xff800000u;
    }
}
__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
    float a = fmaxf(u2f(s[0]), u2f(s[1])), b = fmaxf(u2f(s[2]), u2f(s[3]));
#pragma unroll
    for (int e = 4; e < 32; e += 4) {
        a = max3(a, u2f(s[e]), u2f(s[e + 1]));
        b = max3(b, u2f(s[e + 2]), u2f(s[e + 3]));
    }
    return fmaxf(a, b);
}
// 32 scores -> 32 weights in pk, two to a register; their sum joins `sum`
template <bool SCALED, bool MASKED>
__device__ __forceinline__ void weights32(const uint32_t (&s)[32], uint32_t (&pk)[16], float c,
                                          float base, const float* vs, uint32_t vis,
                                          uint64_t (&sum)[2]) {
    const uint64_t c2 = f2(c, c), b2 = f2(-base, -base);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
        float p[4];
        unf2(fma2(f2(u2f(s[e]), u2f(s[e + 1])), c2, b2), p[0], p[1]);
        unf2(fma2(f2(u2f(s[e + 2]), u2f(s[e + 3])), c2, b2), p[2], p[3]);
#pragma unroll
        for (int x = 0; x < 4; x++) p[x] = ex2(p[x]);
        sum[0] = add2(sum[0], f2(p[0], p[1]));
        sum[1] = add2(sum[1], f2(p[2], p[3]));
        if (SCALED) {
            const float4 v4 = *reinterpret_cast<const float4*>(vs + e);
            unf2(mul2(f2(p[0], p[1]), f2(v4.x, v4.y)), p[0], p[1]);
            unf2(mul2(f2(p[2], p[3]), f2(v4.z, v4.w)), p[2], p[3]);
            if (MASKED) {
#pragma unroll
                for (int x = 0; x < 4; x++)
                    if (!((vis >> (e + x)) & 1)) p[x] = 0.0f;
            }
        }
        pk[e / 2] = SCALED ? f16x2(p[0], p[1]) : bf16x2(p[0], p[1]);
        pk[e / 2 + 1] = SCALED ? f16x2(p[2], p[3]) : bf16x2(p[2], p[3]);
    }
}
// The reference has moved: the D columns of O at tm_o, computed with the old one, times f.
template <int D>
__device__ __forceinline__ void rescale(uint32_t tm_o, float f) {
    tc_wait_st();
#pragma unroll 1
    for (int x = 0; x < D; x += 16) {
        uint32_t ov[16];
        tc_ld16(tm_o + x, ov);
        tc_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e++) ov[e] = __float_as_uint(u2f(ov[e]) * f);
        tc_st16(tm_o + x, ov);
    }
}

// One thread's row: its 128 scores of the block (columns tm_s .. of its lane)
// become weights, two per column from tm_s on: bf16, or f16 in the scaled form.
//   t_j = c S_j (scaled: c ks_j S_j), p_j = 2^(t_j - reference), l += p_j, the
//   weight p_j (scaled: p_j vs_j; 0 for a key that is not seen, whatever vs_j
//   holds)
// MASKED: keys whose bit of vis is clear are not seen.  A block that every row
// sees whole takes the other instance: as a run-time choice the compiler turned
// the selects into predicated code for every block, twice the instructions.
// Where a maximum exceeds the reference by 2^8 (scaled: where a weight passes the row's
// unit by 2^15), which is so in few blocks, the reference moves and what it has been used
// for is rescaled - the caller has seen the products before this block complete.  All
// lanes of a warp take part; `live` = the row exists.
// Both forms hold the 128 scores in registers.
template <int D, bool MASKED>
__device__ __forceinline__ void softmax_block(uint32_t tm_s, uint32_t tm_o, bool have_o,
                                              const uint32_t (&vis)[4], float c, bool live,
                                              RowState& st) {
    uint32_t s[4][32];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; i++) tc_ld32(tm_s + 32 * i, s[i]);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 4; i++) {
        prepare32<false, MASKED>(s[i], nullptr, vis[i]);
        top = fmaxf(top, max32(s[i]));
    }
    // (-inf - -inf is NaN: no move)
    const bool move = (top - st.m) * c > SM_RESCALE_LOG2 && live;
    if (__any_sync(0xffffffffu, move)) {
        const float f = move ? ex2((st.m - top) * c) : 1.0f;
        if (move) st.m = top;
        st.l *= f;
        if (have_o) rescale<D>(tm_o, f);
    }
    float base = st.m == -INFINITY ? 0.0f : st.m * c;
    if (fabsf(base) > 0x1p22f) {
        // c m itself is rounded by more than a fraction of one power of two: take
        // the differences first
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 32; e++) s[i][e] = __float_as_uint(u2f(s[i][e]) - st.m);
        base = 0.0f;
    }
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t pk[16];
        weights32<false, MASKED>(s[i], pk, c, base, nullptr, vis[i], sum);
        tc_st16(tm_s + 16 * i, pk);
    }
    float x, y;
    unf2(add2(sum[0], sum[1]), x, y);
    st.l += x + y;
    tc_wait_st();
}

// The scaled form (e4m3 caches).  vmax: the largest |vs| of the block's real keys, seen or
// not: a bound alone.
template <int D, bool MASKED>
__device__ __forceinline__ void softmax_block_scaled(uint32_t tm_s, uint32_t tm_o, bool have_o,
                                                     const uint32_t (&vis)[4], float c,
                                                     const float* ks, const float* vs, float vmax,
                                                     bool live, RowState& st) {
    uint32_t s[4][32];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; i++) tc_ld32(tm_s + 32 * i, s[i]);
    tc_wait_ld();
#pragma unroll
    for (int i = 0; i < 4; i++) {
        prepare32<true, MASKED>(s[i], ks + 32 * i, vis[i]);
        top = fmaxf(top, max32(s[i]));
        asm volatile("" ::: "memory");
    }
    const bool look = (top - st.m) * c > st.lr + unit_limit(vmax) && live;
    if (__any_sync(0xffffffffu, look)) {
        // the largest weight of the keys that the row sees (the scores once more: their
        // scaled form is in registers that a loop cannot index; eight at a time, sixteen
        // push some of those into local memory: trees of 16 tokens 89.7 us, with eight 85.9)
        float e = -INFINITY;
#pragma unroll 1
        for (int x = 0; x < 128; x += 8) {
            uint32_t r[8];
            tc_ld8(tm_s + x, r);
            tc_wait_ld();
            const uint32_t w = x < 64 ? (x < 32 ? vis[0] : vis[1]) : (x < 96 ? vis[2] : vis[3]);
#pragma unroll
            for (int y = 0; y < 8; y++) {
                // (the product rounded as top was: a fused one would be off by as much as
                // the unit of large scores)
                const float t = fmaf(__fmul_rn(u2f(r[y]), ks[x + y]) - top, c,
                                     lg2(fabsf(vs[x + y])));
                if (!MASKED || ((w >> ((x & 24) + y)) & 1)) e = fmaxf(e, t);
            }
        }
        const float f = live ? move_unit(top, e, c, st.m, st.lr) : 1.0f;
        st.l *= f;
        if (have_o) rescale<D>(tm_o, f);
    }
    float base = st.m == -INFINITY ? 0.0f : fmaf(st.m, c, st.lr);
    if (fabsf(base) > 0x1p22f) {
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int e = 0; e < 32; e++) s[i][e] = __float_as_uint(u2f(s[i][e]) - st.m);
        base = st.lr;
    }
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        uint32_t pk[16];
        weights32<true, MASKED>(s[i], pk, c, base, vs + 32 * i, vis[i], sum);
        tc_st16(tm_s + 16 * i, pk);
    }
    float x, y;
    unf2(add2(sum[0], sum[1]), x, y);
    st.l += x + y;
    tc_wait_st();
}

// The end of a row: the sink joins the denominator; O times factor is the
// output.  m in log2 units, snk in natural ones; a row that saw nothing (m =
// -inf) has factor 0.
struct RowEnd {
    float factor, lse;
};
__device__ __forceinline__ RowEnd row_end(float m, float l, float snk) {
    snk *= SM_LOG2E;
    const float top = fmaxf(m, snk);
    const float base = top == -INFINITY ? 0.0f : top;
    const float f = exp2f(m - base);
    const float den = l * f + exp2f(snk - base);
    RowEnd r;
    r.factor = den == 0.0f ? 0.0f : f / den;
    r.lse = (base + log2f(den)) * SM_LN2;
    return r;
}

// A warp's 32 rows of O, times inv, as bf16 to o + off (off < 0: not written; a
// lane's off is that of row `lane`).  A lane has one row of tensor memory, but stores
// of 16 bytes to 32 rows each take 32 lines' worth of issue; so the rows go back into
// O's own columns as bf16 and are read in the shape that gives four lanes a row's 64
// bytes (words 4c .. 4c + 3 for lane c, by the order in which they are written): 8
// lines a store.  done(): O's columns are free.  (Seven
// prompts of 415 .. 2000 tokens 162 -> 152 us, one of 16384 tokens 1369 -> 1355 us.)
__device__ __forceinline__ void tc_ld_16x256b(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
        "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}
template <int D, typename Done>
__device__ __forceinline__ void store_rows(uint32_t tm_o, bool any, float inv, uint16_t* o,
                                           int off, int hd, Done done) {
#pragma unroll
    for (int x = 0; x < D; x += 32) {
        uint32_t ov[32] = {}, w[16];
        if (any) {
            tc_ld32(tm_o + x, ov);
            tc_wait_ld();
        }
#pragma unroll
        for (int i = 0; i < 16; i++)
            w[((i >> 1) & 1) * 8 + (i >> 2) * 2 + (i & 1)] =
                bf16x2(u2f(ov[2 * i]) * inv, u2f(ov[2 * i + 1]) * inv);
        tc_st16(tm_o + x / 2, w);  // (these columns have been read)
    }
    tc_wait_st();
    const int lane = threadIdx.x & 31, d0 = (lane & 3) * 8;
#pragma unroll
    for (int half = 0; half < 2; half++) {
        uint32_t r[D / 64][16];
#pragma unroll
        for (int x = 0; x < D / 64; x++)
            tc_ld_16x256b(tm_o + ((uint32_t)(16 * half) << 16) + 32 * x, r[x]);
        tc_wait_ld();
        if (half == 1) done();
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int to = __shfl_sync(0xffffffffu, off, 16 * half + 8 * i + (lane >> 2));
#pragma unroll
            for (int d = 0; d < D; d += 32) {
                const uint32_t* v = r[d / 64] + (d % 64) / 4 + 2 * i;
                if (to >= 0 && d + d0 < hd)
                    *reinterpret_cast<uint4*>(o + to + d + d0) = make_uint4(v[0], v[1], v[4], v[5]);
            }
        }
    }
}

}  // namespace tc
}  // namespace ds41
