// ds41_dense_attn.cu - dense attention with grouped heads: causal attention
// over packed prompts, and attention of drafted tokens over a paged cache.
//
// Mathematics.  One pass over the keys with the running maximum m and the
// running sum l of a softmax, in units of log2: with t_j = scale log2(e)
// <q, k_j>, a tile of keys replaces m by max(m, max t_j), scales l and the
// accumulated output by 2^(m_old - m) and adds 2^(t_j - m) and
// 2^(t_j - m) v_j.  The sink enters once, at the end, as one more term of l.
//
// The rows of a (sequence, key/value head) are all its queries times the
// query heads that share the head, token-major: row r is query r / G of head
// r % G of the group, so a tile of rows shares every key it reads.
#include "ds41_dense.cuh"

namespace ds41 {
namespace {

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

struct DenseArgs {
    const uint16_t* q;
    int64_t q_tok, q_head;
    // packed keys and values
    const uint16_t* k;
    int64_t k_tok, k_head;
    const uint16_t* v;
    int64_t v_tok, v_head;
    const int32_t* cu_k;
    int64_t Tk;
    // paged
    PagedKv kv;
    const int32_t* table;
    const int32_t* lens;
    const int64_t* mask;
    int max_pages, mask_words, max_len;
    // both
    const int32_t* cu_q;
    const float* sink;
    uint16_t* o;
    float* lse;
    int64_t Tq;
    int max_q, nh, kvh, hd, G;
    float scale_log2;
    int64_t window;
    unsigned int* status;
};

// The sequence of a CTA, checked: queries q0 .. q0 + n - 1 and `len` keys.
struct Seq {
    int q0, n, k0, len;
    bool ok;
};

template <bool PAGED>
__device__ __forceinline__ Seq load_seq(const DenseArgs& a, int b) {
    Seq s;
    s.q0 = a.cu_q[b];
    const int64_t n = (int64_t)a.cu_q[b + 1] - s.q0;
    s.ok = s.q0 >= 0 && n >= 0 && n <= a.max_q && s.q0 + n <= a.Tq;
    s.n = (int)n;
    if (PAGED) {
        s.k0 = 0;
        s.len = a.lens[b];
        s.ok = s.ok && s.len >= n && s.len <= a.max_len &&
               s.len <= (int64_t)a.max_pages * a.kv.page;
    } else {
        s.k0 = a.cu_k[b];
        const int64_t len = (int64_t)a.cu_k[b + 1] - s.k0;
        s.ok = s.ok && s.k0 >= 0 && len >= 0 && s.k0 + len <= a.Tk;
        s.len = (int)len;
    }
    return s;
}

// What one row sees: earlier keys lo < j < pre, then those of the drafted
// part.  Packed prompts: pre = last + 1 and no drafted part.
struct RowView {
    int64_t lo;      // keys at or before lo are not seen (before `pre`)
    int pre;         // keys below pre go by lo alone
    int chain_last;  // keys pre .. chain_last are seen (no mask)
    const int64_t* bits;
};

template <bool PAGED>
__device__ __forceinline__ RowView row_view(const DenseArgs& a, const Seq& s, int t) {
    RowView w;
    w.bits = nullptr;
    if (!PAGED) {
        const int p = t + s.len - s.n;
        w.pre = p + 1;
        w.chain_last = p;
        w.lo = a.window ? (int64_t)p - a.window : -1;
        return w;
    }
    w.pre = s.len - s.n;
    int d = t;
    w.chain_last = w.pre + t;
    if (a.mask) {
        w.bits = a.mask + (int64_t)(s.q0 + t) * a.mask_words;
        d = -1;
        for (int i = 0; i * 64 < s.n; i++) {
            uint64_t m = (uint64_t)w.bits[i];
            if (s.n - 64 * i < 64) m &= (1ull << (s.n - 64 * i)) - 1;
            d += __popcll(m);
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

constexpr int ROWS = 64, KEYS = 64, NT = 128;

template <int HD, bool PAGED, bool E4M3>
__global__ void __launch_bounds__(NT) dense_attn_kernel(const DenseArgs a) {
    pdl_wait();
    pdl_trigger();
    __shared__ __align__(16) uint16_t sk[KEYS][HD + 8], sv[KEYS][HD + 8];
    __shared__ float sks[KEYS], svs[KEYS];
    __shared__ uint8_t sok[KEYS];
    const int b = blockIdx.z, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Seq s = load_seq<PAGED>(a, b);
    if (!s.ok) {
        if (threadIdx.x == 0) raise_status(a.status, DS41_E_INDEX);
        return;
    }
    const int64_t rows = (int64_t)s.n * a.G, r0 = (int64_t)blockIdx.x * ROWS;
    if (r0 >= rows) return;
    // the queries, in registers
    RowView view[2];
    bool live[2];
    const uint16_t* qp[2];
    int tok[2], head[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        int64_t r = r0 + warp * 16 + (lane >> 2) + 8 * i;
        live[i] = r < rows;
        if (!live[i]) r = rows - 1;
        tok[i] = (int)(r / a.G);
        head[i] = h * a.G + (int)(r % a.G);
        qp[i] = a.q + (s.q0 + tok[i]) * a.q_tok + head[i] * a.q_head;
        view[i] = row_view<PAGED>(a, s, tok[i]);
    }
    uint32_t qf[HD / 16][4];
#pragma unroll
    for (int kk = 0; kk < HD / 16; kk++) {
        const int c = kk * 16 + (lane & 3) * 2;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            qf[kk][i] = c < a.hd ? *reinterpret_cast<const uint32_t*>(qp[i] + c) : 0;
            qf[kk][i + 2] = c + 8 < a.hd ? *reinterpret_cast<const uint32_t*>(qp[i] + c + 8) : 0;
        }
    }
    float o[HD / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0, 0};
    // the keys that some row of the tile sees
    const int t_first = (int)(r0 / a.G), t_last = (int)((min(rows, r0 + ROWS) - 1) / a.G);
    int64_t k_lo = 0, k_hi = s.len;
    if (!PAGED) {
        k_hi = min((int64_t)s.len, (int64_t)t_last + s.len - s.n + 1);
        if (a.window) k_lo = max((int64_t)0, (int64_t)t_first + s.len - s.n - a.window + 1);
    } else if (a.window) {
        // a drafted token stands at or behind the row before the drafted ones
        k_lo = max((int64_t)0, (int64_t)s.len - s.n - a.window);
    }
    for (int64_t j0 = k_lo / KEYS * KEYS; j0 < k_hi; j0 += KEYS) {
        __syncthreads();
        for (int x = threadIdx.x; x < KEYS * (HD / 8); x += NT) {
            const int row = x / (HD / 8), c = (x % (HD / 8)) * 8;
            const int64_t j = j0 + row;
            uint4 kx = make_uint4(0, 0, 0, 0), vx = kx;
            bool ok = j < s.len;
            float ks = 1.0f, vs = 1.0f;
            if (PAGED) {
                int64_t pg = -1, at = 0;
                if (ok) {
                    pg = a.table[(int64_t)b * a.max_pages + (j >> a.kv.page_shift)];
                    if (pg < 0 || pg >= a.kv.n_pages) {
                        ok = false;
                        raise_status(a.status, DS41_E_INDEX);
                    } else {
                        at = paged_row(a.kv, pg, h, (int)(j & (a.kv.page - 1)));
                    }
                }
                if (ok && c < a.hd) {
                    if (E4M3) {
                        const uint2 kc = *reinterpret_cast<const uint2*>(a.kv.k + at * a.hd + c);
                        const uint2 vc = *reinterpret_cast<const uint2*>(a.kv.v + at * a.hd + c);
                        kx = make_uint4(e4m3_spread(__byte_perm(kc.x, 0, 0x1404)),
                                        e4m3_spread(__byte_perm(kc.x, 0, 0x3424)),
                                        e4m3_spread(__byte_perm(kc.y, 0, 0x1404)),
                                        e4m3_spread(__byte_perm(kc.y, 0, 0x3424)));
                        vx = make_uint4(e4m3_spread(__byte_perm(vc.x, 0, 0x1404)),
                                        e4m3_spread(__byte_perm(vc.x, 0, 0x3424)),
                                        e4m3_spread(__byte_perm(vc.y, 0, 0x1404)),
                                        e4m3_spread(__byte_perm(vc.y, 0, 0x3424)));
                        ks = a.kv.ks[at];
                        vs = a.kv.vs[at];
                    } else {
                        kx = *reinterpret_cast<const uint4*>(a.kv.k + (at * a.hd + c) * 2);
                        vx = *reinterpret_cast<const uint4*>(a.kv.v + (at * a.hd + c) * 2);
                    }
                }
            } else if (ok && c < a.hd) {
                kx = *reinterpret_cast<const uint4*>(a.k + (s.k0 + j) * a.k_tok + h * a.k_head + c);
                vx = *reinterpret_cast<const uint4*>(a.v + (s.k0 + j) * a.v_tok + h * a.v_head + c);
            }
            *reinterpret_cast<uint4*>(&sk[row][c]) = kx;
            *reinterpret_cast<uint4*>(&sv[row][c]) = vx;
            if (c == 0) {
                sks[row] = ks;
                svs[row] = vs;
                sok[row] = ok;
            }
        }
        __syncthreads();
        float sc[KEYS / 8][4];
#pragma unroll
        for (int n = 0; n < KEYS / 8; n++) {
#pragma unroll
            for (int e = 0; e < 4; e++) sc[n][e] = 0.0f;
#pragma unroll
            for (int kk = 0; kk < HD / 16; kk++) {
                const uint16_t* kp = &sk[n * 8 + (lane >> 2)][kk * 16 + (lane & 3) * 2];
                mma_bf16(sc[n], qf[kk][0], qf[kk][1], qf[kk][2], qf[kk][3],
                         *reinterpret_cast<const uint32_t*>(kp),
                         *reinterpret_cast<const uint32_t*>(kp + 8));
            }
        }
        float mx[2] = {m[0], m[1]};
#pragma unroll
        for (int n = 0; n < KEYS / 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int row = n * 8 + (lane & 3) * 2 + (e & 1);
                const bool see = sok[row] && seen(view[e >> 1], (int)(j0 + row), s.len);
                sc[n][e] = see ? sc[n][e] * (a.scale_log2 * sks[row]) : -INFINITY;
                mx[e >> 1] = fmaxf(mx[e >> 1], sc[n][e]);
            }
        float alpha[2], base[2];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
            mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
            base[i] = mx[i] == -INFINITY ? 0.0f : mx[i];  // nothing seen so far
            alpha[i] = exp2f(m[i] - base[i]);
            m[i] = mx[i];
            l[i] *= alpha[i];
        }
#pragma unroll
        for (int n = 0; n < HD / 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[n][e] *= alpha[e >> 1];
#pragma unroll
        for (int n = 0; n < KEYS / 8; n++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const bool gone = sc[n][e] == -INFINITY;
                const float p = exp2f(sc[n][e] - base[e >> 1]);
                l[e >> 1] += p;
                sc[n][e] = gone ? 0.0f : p * svs[n * 8 + (lane & 3) * 2 + (e & 1)];
            }
#pragma unroll
        for (int n = 0; n < KEYS / 16; n++) {
            const uint32_t p0 = pack_bf16x2(sc[2 * n][0], sc[2 * n][1]);
            const uint32_t p1 = pack_bf16x2(sc[2 * n][2], sc[2 * n][3]);
            const uint32_t p2 = pack_bf16x2(sc[2 * n + 1][0], sc[2 * n + 1][1]);
            const uint32_t p3 = pack_bf16x2(sc[2 * n + 1][2], sc[2 * n + 1][3]);
#pragma unroll
            for (int d = 0; d < HD / 8; d += 2) {
                uint32_t v0, v1, v2, v3;
                ldsm_x4_t(smem_u32(&sv[n * 16 + (lane & 15)][d * 8 + (lane >> 4) * 8]), v0, v1, v2,
                          v3);
                mma_bf16(o[d], p0, p1, p2, p3, v0, v1);
                mma_bf16(o[d + 1], p0, p1, p2, p3, v2, v3);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
        l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
        if (!live[i]) continue;
        float f = 1.0f;
        const float snk = a.sink ? a.sink[head[i]] * LOG2E : -INFINITY;
        const float top = fmaxf(m[i], snk);
        const float base = top == -INFINITY ? 0.0f : top;
        f = exp2f(m[i] - base);
        const float den = l[i] * f + exp2f(snk - base);
        const float inv = den == 0.0f ? 0.0f : f / den;
        const int64_t at = (int64_t)(s.q0 + tok[i]) * a.nh + head[i];
        if (a.lse && (lane & 3) == 0) a.lse[at] = (base + log2f(den)) * LN2;
#pragma unroll
        for (int d = 0; d < HD / 8; d++) {
            const int c = d * 8 + (lane & 3) * 2;
            if (c < a.hd)
                *reinterpret_cast<uint32_t*>(a.o + at * a.hd + c) =
                    pack_bf16x2(o[d][2 * i] * inv, o[d][2 * i + 1] * inv);
        }
    }
}

}  // namespace
}  // namespace ds41

using namespace ds41;

extern "C" size_t ds41_tree_attn_workspace_bytes(int64_t, int64_t, int64_t, int64_t, int64_t,
                                                 int64_t, int64_t, int) {
    return 0;
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
    DenseArgs a{};
    if (int rc = check_paged(name, k_cache, v_cache, k_scales, v_scales, fmt, n_pages, page, kvh,
                             hd, &a.kv))
        return rc;
    const int64_t lim = int64_t(1) << 31;
    DS41_REQUIRE(B >= 0 && B < 65536 && Tq >= 0 && Tq < lim && max_q >= 0 && max_q <= 256 &&
                     max_len >= 0 && max_len < lim && max_pages >= 0 && max_pages < lim,
                 DS41_E_RANGE, "%s: B=%lld Tq=%lld max_q=%lld (at most 256) max_len=%lld", name,
                 (long long)B, (long long)Tq, (long long)max_q, (long long)max_len);
    DS41_REQUIRE(!mask || (mask_words >= 1 && mask_words <= 4 && max_q <= 64 * mask_words),
                 DS41_E_ARG, "%s: mask_words=%lld for max_q=%lld", name, (long long)mask_words,
                 (long long)max_q);
    DS41_REQUIRE(window == 0 || window >= max_q, DS41_E_ARG,
                 "%s: window=%lld is below max_q=%lld", name, (long long)window, (long long)max_q);
    if (B == 0 || Tq == 0 || max_q == 0) return DS41_OK;
    DS41_REQUIRE(q && o && cu_q && lens && page_table, DS41_E_ARG,
                 "%s: q, page_table, lens, cu_q and o must be non-null", name);
    DS41_REQUIRE(aligned16(q) && aligned16(o) && aligned_to(cu_q, 4) && aligned_to(lens, 4) &&
                     aligned_to(page_table, 4) && aligned_to(mask, 8) && aligned_to(sink, 4) &&
                     aligned_to(lse, 4),
                 DS41_E_ARG, "%s: q and o must be 16-byte aligned", name);
    DS41_REQUIRE(good_strides(q_tok, q_head, hd), DS41_E_ARG,
                 "%s: strides must be multiples of 8 and at least hd", name);
    a.q = q; a.q_tok = q_tok; a.q_head = q_head;
    a.table = page_table; a.max_pages = (int)max_pages; a.lens = lens; a.max_len = (int)max_len;
    a.mask = mask; a.mask_words = (int)mask_words;
    a.cu_q = cu_q; a.Tq = Tq;
    a.max_q = (int)max_q; a.nh = (int)nh; a.kvh = (int)kvh; a.hd = (int)hd; a.G = (int)(nh / kvh);
    a.scale_log2 = scale * LOG2E; a.window = window; a.sink = sink; a.o = o; a.lse = lse;
    if (int rc = status_word(&a.status)) return rc;
    const int64_t tiles = (max_q * a.G + ROWS - 1) / ROWS;
    auto kern = fmt == DS41_KV_E4M3
                    ? (hd <= 64 ? dense_attn_kernel<64, true, true> : dense_attn_kernel<128, true, true>)
                    : (hd <= 64 ? dense_attn_kernel<64, true, false>
                                : dense_attn_kernel<128, true, false>);
    return launch_pdl(kern, dim3((unsigned)tiles, (unsigned)kvh, (unsigned)B), dim3(NT), 0,
                      (cudaStream_t)stream, name, a);
}
