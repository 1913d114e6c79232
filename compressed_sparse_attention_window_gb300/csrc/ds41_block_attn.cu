// ds41_block_attn.cu - attention over the blocks that were picked for each token and
// key/value head: over the pages of a cache, and over packed prompts.
//
// Mathematics.  One pass with a running reference m and sum l per row:
//   s_j = scale <q, k_j>,  p_j = e^(s_j - m),  l += p_j,  o += p_j v_j
// over the rows j <= p of the listed blocks, the sink joining l at the end.
#include "ds41_softmax_tc.cuh"

namespace ds41 {
namespace ba {

struct Args {
    const uint16_t* q;
    int64_t q_tok, q_head;
    PagedKv kv;              // pages
    const uint16_t* x[2];    // or packed k, v
    int64_t tok[2], head[2];
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu_q;
    const int32_t* cu_k;
    const int32_t* idx;
    const float* sink;
    uint16_t* o;
    float* lse;
    int64_t Tq, Tk, max_pages;
    int B, max_q, max_k, nh, kvh, hd, G, topk, block, block_shift;
    float scale;
    unsigned int* status;
};

struct Seq {
    int q0, n, k0, len;
    bool ok;
};
template <bool PAGED>
__device__ __forceinline__ Seq load_seq(const Args& a, int b) {
    Seq s;
    s.q0 = a.cu_q[b];
    const int64_t n = (int64_t)a.cu_q[b + 1] - s.q0;
    s.n = (int)n;
    s.k0 = PAGED ? 0 : a.cu_k[b];
    const int64_t len = PAGED ? a.lens[b] : (int64_t)a.cu_k[b + 1] - s.k0;
    s.len = (int)len;
    s.ok = s.q0 >= 0 && n >= 0 && n <= a.max_q && s.q0 + n <= a.Tq && len >= n &&
           (PAGED ? len <= a.max_pages * a.block
                  : s.k0 >= 0 && len <= a.max_k && s.k0 + len <= a.Tk);
    return s;
}

constexpr int WARPS = 4;

// A CTA for a token and a key/value head, a warp for every fourth of its query heads;
// four elements of a row a lane.
template <bool PAGED, bool E4M3>
__global__ void __launch_bounds__(WARPS * 32) block_attn_kernel(const Args a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x == 0 && blockIdx.y == 0)
        for (int b = threadIdx.x; b < a.B; b += WARPS * 32)
            if (!load_seq<PAGED>(a, b).ok) raise_status(a.status, DS41_E_INDEX);
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y;
    int b = 0, end = a.B;  // the last b with cu_q[b] <= t
    while (end - b > 1) {
        const int mid = (b + end) >> 1;
        if (a.cu_q[mid] <= t) b = mid;
        else end = mid;
    }
    const Seq s = load_seq<PAGED>(a, b);
    if (!s.ok || t < s.q0 || t >= s.q0 + s.n) return;
    const int p = s.len - s.n + (int)(t - s.q0);
    const int32_t* list = a.idx + (t * a.kvh + h) * a.topk;
    const bool mine = lane * 4 < a.hd;
    for (int y = warp; y < a.G; y += WARPS) {
        const int head = h * a.G + y;
        float q[4] = {0, 0, 0, 0}, o[4] = {0, 0, 0, 0}, m = -INFINITY, l = 0.0f;
        auto four = [&](const uint16_t* at, float (&v)[4]) {
            const uint2 w = *reinterpret_cast<const uint2*>(at);
            v[0] = __uint_as_float(w.x << 16);
            v[1] = __uint_as_float(w.x & 0xffff0000u);
            v[2] = __uint_as_float(w.y << 16);
            v[3] = __uint_as_float(w.y & 0xffff0000u);
        };
        if (mine) four(a.q + t * a.q_tok + head * a.q_head + lane * 4, q);
        int before = -1;
        for (int i = 0; i < a.topk; i++) {
            const int x = list[i];
            if (x == -1) break;
            if (x <= before || x > p >> a.block_shift) {
                if (lane == 0) raise_status(a.status, DS41_E_INDEX);
                break;
            }
            before = x;
            int64_t row = 0;
            if (PAGED) {
                const int pg = a.table[(int64_t)b * a.max_pages + x];
                if (pg < 0 || pg >= a.kv.n_pages) {
                    if (lane == 0) raise_status(a.status, DS41_E_INDEX);
                    continue;
                }
                row = paged_row(a.kv, pg, h, 0);
            }
            const int rows = min(a.block, p - (x << a.block_shift) + 1);
            for (int r = 0; r < rows; r++) {
                float kv[2][4] = {};
                if (mine) {
#pragma unroll
                    for (int z = 0; z < 2; z++) {
                        if (!PAGED) {
                            four(a.x[z] + (s.k0 + ((int64_t)x << a.block_shift) + r) * a.tok[z] +
                                     h * a.head[z] + lane * 4, kv[z]);
                        } else if (!E4M3) {
                            four(reinterpret_cast<const uint16_t*>(z ? a.kv.v : a.kv.k) +
                                     (row + r) * a.hd + lane * 4, kv[z]);
                        } else {
                            const uint32_t w = *reinterpret_cast<const uint32_t*>(
                                (z ? a.kv.v : a.kv.k) + (row + r) * a.hd + lane * 4);
                            const float f = (z ? a.kv.vs : a.kv.ks)[row + r];
#pragma unroll
                            for (int e = 0; e < 4; e++)
                                kv[z][e] = e4m3_to_f32(w >> (8 * e)) * f;
                        }
                    }
                }
                float sc = q[0] * kv[0][0] + q[1] * kv[0][1] + q[2] * kv[0][2] + q[3] * kv[0][3];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    sc += __shfl_xor_sync(0xffffffffu, sc, off);
                sc *= a.scale;
                const float to = fmaxf(m, sc), f = m == -INFINITY ? 0.0f : expf(m - to);
                const float w = to == -INFINITY ? 0.0f : expf(sc - to);
                l = l * f + w;
#pragma unroll
                for (int e = 0; e < 4; e++) o[e] = o[e] * f + w * kv[1][e];
                m = to;
            }
        }
        const tc::RowEnd end_of =
            tc::row_end(m * tc::SM_LOG2E, l, a.sink ? a.sink[head] : -INFINITY);
        const int64_t at = t * a.nh + head;
        if (a.lse && lane == 0) a.lse[at] = end_of.lse;
        if (mine)
            *reinterpret_cast<uint2*>(a.o + at * a.hd + lane * 4) =
                make_uint2(tc::bf16x2(o[0] * end_of.factor, o[1] * end_of.factor),
                           tc::bf16x2(o[2] * end_of.factor, o[3] * end_of.factor));
    }
}

int check_lists(const char* name, const int32_t* idx, int64_t topk, int64_t block) {
    DS41_REQUIRE(block >= 16 && block <= 256 && (block & (block - 1)) == 0, DS41_E_ARG,
                 "%s: blocks of %lld rows (a power of two of 16 .. 256)", name, (long long)block);
    DS41_REQUIRE(topk >= 1 && topk <= 1024, DS41_E_ARG, "%s: topk=%lld (1 .. 1024)", name,
                 (long long)topk);
    return DS41_OK;
}

}  // namespace ba
}  // namespace ds41

using namespace ds41;

extern "C" size_t ds41_block_attn_workspace_bytes(int64_t Tq, int64_t topk, int64_t page,
                                                  int64_t nh, int64_t kvh, int64_t hd, int fmt) {
    return 0;
}

extern "C" int ds41_block_attn_fwd(const ds41_bf16* q, int64_t q_tok, int64_t q_head,
                                   const void* k_cache, const void* v_cache,
                                   const float* k_scales, const float* v_scales, int fmt,
                                   int64_t n_pages, int64_t page, const int32_t* page_table,
                                   int64_t max_pages, const int32_t* lens, const int32_t* cu_q,
                                   const int32_t* idx, int64_t topk, int64_t B, int64_t Tq,
                                   int64_t max_q, int64_t nh, int64_t kvh, int64_t hd, float scale,
                                   const float* sink, ds41_bf16* o, float* lse, void* ws,
                                   size_t ws_bytes, ds41_stream_t stream) {
    const char* name = "ds41_block_attn_fwd";
    if (int rc = check_heads(name, nh, kvh, hd, scale, 0)) return rc;
    ba::Args a{};
    if (int rc = check_paged(name, k_cache, v_cache, k_scales, v_scales, fmt, n_pages, page, kvh,
                             hd, &a.kv))
        return rc;
    if (int rc = ba::check_lists(name, idx, topk, page)) return rc;
    const int64_t lim = int64_t(1) << 31;
    DS41_REQUIRE(B >= 0 && B < 65536 && Tq >= 0 && Tq < lim && max_q >= 0 && max_q < lim &&
                     max_pages >= 0 && max_pages < lim,
                 DS41_E_RANGE, "%s: B=%lld Tq=%lld max_q=%lld max_pages=%lld", name, (long long)B,
                 (long long)Tq, (long long)max_q, (long long)max_pages);
    if (B == 0 || Tq == 0 || max_q == 0) return DS41_OK;
    DS41_REQUIRE(q && o && cu_q && lens && page_table && idx, DS41_E_ARG,
                 "%s: q, page_table, lens, cu_q, idx and o must be non-null", name);
    DS41_REQUIRE(aligned16(q) && aligned16(o) && aligned_to(cu_q, 4) && aligned_to(lens, 4) &&
                     aligned_to(page_table, 4) && aligned_to(idx, 4) && aligned_to(sink, 4) &&
                     aligned_to(lse, 4),
                 DS41_E_ARG, "%s: q and o must be 16-byte aligned", name);
    DS41_REQUIRE(good_strides(q_tok, q_head, hd), DS41_E_ARG,
                 "%s: strides must be multiples of 8 and at least hd", name);
    a.q = q;
    a.q_tok = q_tok;
    a.q_head = q_head;
    a.table = page_table;
    a.max_pages = max_pages;
    a.lens = lens;
    a.cu_q = cu_q;
    a.idx = idx;
    a.sink = sink;
    a.o = o;
    a.lse = lse;
    a.Tq = Tq;
    a.B = (int)B;
    a.max_q = (int)max_q;
    a.nh = (int)nh;
    a.kvh = (int)kvh;
    a.hd = (int)hd;
    a.G = (int)(nh / kvh);
    a.topk = (int)topk;
    a.block = (int)page;
    a.block_shift = a.kv.page_shift;
    a.scale = scale;
    if (int rc = status_word(&a.status)) return rc;
    return launch_pdl(fmt == DS41_KV_E4M3 ? ba::block_attn_kernel<true, true>
                                          : ba::block_attn_kernel<true, false>,
                      dim3((unsigned)Tq, (unsigned)kvh), dim3(ba::WARPS * 32), 0,
                      (cudaStream_t)stream, name, a);
}

extern "C" size_t ds41_block_prompt_attn_workspace_bytes(int64_t B, int64_t Tq, int64_t max_q,
                                                         int64_t max_k, int64_t topk,
                                                         int64_t block, int64_t nh, int64_t kvh) {
    return 0;
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
    if (int rc = ba::check_lists(name, idx, topk, block)) return rc;
    const int64_t lim = int64_t(1) << 31;
    DS41_REQUIRE(B >= 0 && B < 65536 && Tq >= 0 && Tq < lim && Tk >= 0 && Tk < lim && max_q >= 0 &&
                     max_q < lim && max_k >= 0 && max_k <= 32768 * block && kvh < 65536,
                 DS41_E_RANGE,
                 "%s: B=%lld Tq=%lld Tk=%lld max_q=%lld max_k=%lld (at most 32768 blocks)", name,
                 (long long)B, (long long)Tq, (long long)Tk, (long long)max_q, (long long)max_k);
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
    ba::Args a{};
    a.q = q;
    a.q_tok = q_tok;
    a.q_head = q_head;
    a.x[0] = k;
    a.x[1] = v;
    a.tok[0] = k_tok;
    a.tok[1] = v_tok;
    a.head[0] = k_head;
    a.head[1] = v_head;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.idx = idx;
    a.sink = sink;
    a.o = o;
    a.lse = lse;
    a.Tq = Tq;
    a.Tk = Tk;
    a.B = (int)B;
    a.max_q = (int)max_q;
    a.max_k = (int)max_k;
    a.nh = (int)nh;
    a.kvh = (int)kvh;
    a.hd = (int)hd;
    a.G = (int)(nh / kvh);
    a.topk = (int)topk;
    a.block = (int)block;
    while ((1 << a.block_shift) < block) a.block_shift++;
    a.scale = scale;
    if (int rc = status_word(&a.status)) return rc;
    return launch_pdl(ba::block_attn_kernel<false, false>, dim3((unsigned)Tq, (unsigned)kvh),
                      dim3(ba::WARPS * 32), 0, (cudaStream_t)stream, name, a);
}
