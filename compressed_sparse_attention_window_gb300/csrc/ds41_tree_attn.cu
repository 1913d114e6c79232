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

using few::GROUP;

constexpr int WARPS = 4;
constexpr int NT = WARPS * 32;
constexpr int BLOCK = WARPS * GROUP;  // keys of a block: a group for every warp

// shared memory: the warps' rings, then their results
template <int HD, bool E4M3>
constexpr int few_bytes() {
    using C = few::Cfg<HD, E4M3>;
    return WARPS * (C::RING > 16 * C::P * 4 ? C::RING : 16 * C::P * 4);
}

template <int HD, bool E4M3>
__global__ void __launch_bounds__(NT, E4M3 ? 3 : 2) tree_few_kernel(const Args a) {
    pdl_wait();
    using C = few::Cfg<HD, E4M3>;
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

        uint8_t* ring = smem + warp * C::RING;
        const int n_groups = (k1 - k0 + GROUP - 1) / GROUP;
        const int mine = (n_groups - warp + WARPS - 1) / WARPS;  // groups warp, warp + 4, ...
        const int32_t* table = a.table + (int64_t)pc.b * a.max_pages;
        unsigned bad = 0;  // stages whose page does not exist

        const few::Copier<HD, E4M3> copier(a.hd, lane);
        const int head_rows = h * a.kv.page;
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
                copier.copy(ring_u + st * C::STAGE, a.kv, row, ok ? min(GROUP, k1 - j) : 0, ok,
                            lane);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < C::STAGES - 1; i++) fetch(i);

        // the queries: rows g and g + 8 of the tile
        RowView view[2];
        few::Rows<HD, E4M3> mem;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int r = min(g + 8 * i, rows - 1);
            const int t = r / a.G;
            view[i] = row_view(a, s, t);
            mem.query(i, a.q + (s.q0 + t) * a.q_tok + (h * a.G + r % a.G) * a.q_head, a.hd, c);
        }
        mem.start(a.scale_log2);
        // keys below `easy` are seen by both rows (and none lies at or before lo)
        const int easy = min(view[0].pre, view[1].pre);
        const int64_t lo = view[0].lo > view[1].lo ? view[0].lo : view[1].lo;

        for (int i = 0; i < mine; i++) {
            fetch(i + C::STAGES - 1);
            cp_async_wait<C::STAGES - 1>();
            __syncwarp();
            const int st = i % C::STAGES, j = k0 + (i * WARPS + warp) * GROUP;
            const bool none = (bad >> st) & 1;
            mem.group(
                ring + st * C::STAGE, none || j + GROUP > easy || j <= lo,
                [&](int i2, int x) { return !none && seen(view[i2], j + x, s.len); }, g, c);
            __syncwarp();  // the stage is read before it is filled again
        }
        cp_async_wait<0>();
        __syncthreads();
        // ---- the warps' results: through shared memory, 16 rows ----
        constexpr int P = C::P;
        float* out = reinterpret_cast<float*>(smem);
        mem.put(out + warp * 16 * P, g, c);
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
    constexpr int smem = few_bytes<HD, E4M3>();
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
