// ds41_block_attn.cu - attention of few tokens over the blocks that were picked for each of
// them and each key/value head, on the pages of a cache.
//
// Mathematics.  As tree attention of few rows (ds41_tree_attn.cu, ds41_few.cuh): one pass
// over the rows j <= p of the listed pages, with a lazily moved reference per row.  The
// rows of a tile are the query heads of one token that share a key/value head (lists
// differ from token to token), 8 for groups of at most 8 heads, else 16.
//
// What bounds it.  Each listed row is read once a token: HBM when there are tokens
// enough.  A token's list is cut into as many runs as fill the GPU, at most eight, the
// CTAs of a cluster, which join their results through each other's shared memory: no
// second launch and no scratch.  The chain before the first row arrives (which sequence, its
// length, the list, the table) is walked by all threads at once.  (16 tokens of 64 heads of
// 128 over 8, 64 blocks of 64 e4m3 rows each: 29.7 us, 4.7 TB/s, of which the chain before
// and the joining behind are about a quarter; as rows of 16, half of them padding, 31.8.)
#include <type_traits>

#include "ds41_few.cuh"

namespace ds41 {
namespace ba {

using few::GROUP;

struct Args {
    const uint16_t* q;
    int64_t q_tok, q_head;
    PagedKv kv;
    const int32_t* table;
    const int32_t* lens;
    const int32_t* cu_q;
    const int32_t* idx;
    const float* sink;
    uint16_t* o;
    float* lse;
    int64_t Tq, max_pages;
    int B, max_q, nh, kvh, hd, G, topk, block, block_shift;
    float scale;
    int tiles;  // of a group's query heads
    int runs;   // of a list
    unsigned int* status;
};

struct Seq {
    int q0, n, len;
    bool ok;
};
__device__ __forceinline__ Seq load_seq(const Args& a, int b) {
    Seq s;
    s.q0 = a.cu_q[b];
    const int64_t n = (int64_t)a.cu_q[b + 1] - s.q0;
    s.n = (int)n;
    s.len = a.lens[b];
    s.ok = s.q0 >= 0 && n >= 0 && n <= a.max_q && s.q0 + n <= a.Tq && s.len >= n &&
           s.len <= a.max_pages * a.block;
    return s;
}

constexpr int WARPS = 4;
constexpr int NT = WARPS * 32;
constexpr int MAX_LIST = 1024;
constexpr int MAX_RUNS = 8;  // CTAs of a cluster

// RT: rows of a tile, 8 or 16
template <int HD, bool E4M3, int RT>
struct Shape {
    using C = few::Cfg<HD, E4M3>;
    // CTAs of an SM: what the registers and the rings leave room for (three of 16 rows, which
    // spill some registers: 16 tokens of 128 heads over 8, e4m3, 35.1 us, two 32.7)
    static constexpr int CTAS = C::RB < 256 && RT == 8 ? 4 : 2;
    static constexpr int STAGES = CTAS == 4 && C::RB == 128 ? 3 : C::STAGES;
    static constexpr int RING = STAGES * C::STAGE;  // of a warp
    static constexpr int OUT = RT * C::P * 4;
    static constexpr int BYTES = WARPS * (RING > OUT ? RING : OUT);
    static_assert(CTAS * (BYTES + 6144) <= 232448, "shared memory of an SM");
};

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                     : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];\n"
                 : "=f"(v.x), "=f"(v.y)
                 : "r"(at)
                 : "memory");
    return v;
}

template <int HD, bool E4M3, int RT>
__global__ void __launch_bounds__(NT, Shape<HD, E4M3, RT>::CTAS) tokens_kernel(const Args a) {
    pdl_wait();
    using C = few::Cfg<HD, E4M3>;
    using S = Shape<HD, E4M3, RT>;
    constexpr int P = C::P;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int list[MAX_LIST];  // pages, -1: outside the cache
    __shared__ int found[2][WARPS];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    const int run = blockIdx.x % a.runs, item = blockIdx.x / a.runs;
    const int unit = item / a.tiles, h = unit % a.kvh, t = unit / a.kvh;
    const int y0 = (item - unit * a.tiles) * RT, rows = min(RT, a.G - y0);
    if (blockIdx.x == 0)
        for (int b = tid; b < a.B; b += NT)
            if (!load_seq(a, b).ok) raise_status(a.status, DS41_E_INDEX);
    // the sequence that has the token (among prefix sums that fall, too: those of a sequence
    // that is skipped do not hide another's)
    int b = -1;
    for (int x = tid; x < a.B; x += NT) {
        const int from = a.cu_q[x], to = a.cu_q[x + 1];
        if (from >= 0 && from <= t && t < to && to <= a.Tq && to - from <= a.max_q) b = x;
    }
    const int32_t* src = a.idx + ((int64_t)t * a.kvh + h) * a.topk;
    int mine[MAX_LIST / NT], before[MAX_LIST / NT];
#pragma unroll
    for (int k = 0; k < MAX_LIST / NT; k++) {
        const int i = k * NT + tid;
        mine[k] = i < a.topk ? src[i] : -1;
        before[k] = i > 0 && i < a.topk ? src[i - 1] : -1;
        if ((k + 1) * NT >= a.topk) break;
    }
    b = __reduce_max_sync(0xffffffffu, b);
    if (lane == 0) found[0][warp] = b;
    __syncthreads();
    b = max(max(found[0][0], found[0][1]), max(found[0][2], found[0][3]));
    if (b < 0) return;  // (the same for the whole cluster)
    const Seq s = load_seq(a, b);
    if (!s.ok) return;
    const int p = s.len - s.n + (t - s.q0), cur = p >> a.block_shift;
    // the list ends at the first entry that does not rise or lies past the token (an entry
    // behind the end may be anything: one below 0 can rise above another)
    const int32_t* table = a.table + (int64_t)b * a.max_pages;
    int end = a.topk;
#pragma unroll
    for (int k = 0; k < MAX_LIST / NT; k++) {
        const int i = k * NT + tid;
        if (i < a.topk) {
            if (mine[k] < 0 || mine[k] <= before[k] || mine[k] > cur) {
                end = min(end, i);
            } else {
                const int pg = table[mine[k]];
                list[i] = pg >= 0 && pg < a.kv.n_pages ? pg : -1;
            }
        }
        if ((k + 1) * NT >= a.topk) break;
    }
    const int least = __reduce_min_sync(0xffffffffu, end);
    if (lane == 0) found[1][warp] = least;
    __syncthreads();
    const int count = min(min(found[1][0], found[1][1]), min(found[1][2], found[1][3]));
#pragma unroll
    for (int k = 0; k < MAX_LIST / NT; k++) {
        const int i = k * NT + tid;
        if (i < a.topk && ((i == count && mine[k] != -1) || (i < count && list[i] < 0)))
            raise_status(a.status, DS41_E_INDEX);
        if ((k + 1) * NT >= a.topk) break;
    }
    // rows of the list: its last block may be the token's own
    int keys = 0;
    if (count > 0)
        keys = (count - 1) * a.block + min(a.block, p - (src[count - 1] << a.block_shift) + 1);
    const int groups = (keys + GROUP - 1) / GROUP;
    const int first = (int)((int64_t)groups * run / a.runs);
    const int own = (int)((int64_t)groups * (run + 1) / a.runs) - first;
    const int n_mine = (own - warp + WARPS - 1) / WARPS;  // groups first + warp, + 4, ...

    uint8_t* ring = smem + warp * S::RING;
    const uint32_t ring_u = smem_u32(ring);
    const few::Copier<HD, E4M3> copier(a.hd, lane);
    const int per = a.block_shift - 4;  // log2 of a page's groups
    unsigned bad = 0;                   // stages whose page does not exist
    auto fetch = [&](int i) {
        if (i < n_mine) {
            const int st = i % S::STAGES, x = first + i * WARPS + warp;
            const int pg = list[x >> per];
            const bool ok = pg >= 0;
            bad = ok ? bad & ~(1u << st) : bad | (1u << st);
            const int64_t row = ok ? ((int64_t)pg * a.kvh + h) * a.block +
                                         ((x & ((1 << per) - 1)) * GROUP)
                                   : 0;
            copier.copy(ring_u + st * C::STAGE, a.kv, row, ok ? min(GROUP, keys - x * GROUP) : 0,
                        ok, lane);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S::STAGES - 1; i++) fetch(i);

    few::Rows<HD, E4M3, RT / 8> mem;
    const uint16_t* q = a.q + t * a.q_tok + ((int64_t)h * a.G + y0) * a.q_head;
#pragma unroll
    for (int n = 0; n < RT / 8; n++)
        mem.query(n, q + min(8 * n + g, rows - 1) * a.q_head, a.hd, a.scale * tc::SM_LOG2E, c);
    for (int i = 0; i < n_mine; i++) {
        fetch(i + S::STAGES - 1);
        cp_async_wait<S::STAGES - 1>();
        __syncwarp();
        const int st = i % S::STAGES, live = keys - (first + i * WARPS + warp) * GROUP;
        const bool none = (bad >> st) & 1;
        mem.group(ring + st * C::STAGE, none ? 0 : live, g, c);
        __syncwarp();  // the stage is read before it is filled again
    }
    cp_async_wait<0>();
    __syncthreads();
    // ---- the warps' results joined into warp 0's place ----
    float* out = reinterpret_cast<float*>(smem);
    mem.put(out + warp * RT * P, g, c);
    __syncthreads();
    constexpr int PER = NT / RT;  // threads of a row
    const int r = tid / PER, part = tid % PER;
    float mm = -INFINITY, f[WARPS], ll = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; w++) mm = fmaxf(mm, out[(w * RT + r) * P + HD]);
    const float ref = mm == -INFINITY ? 0.0f : mm;
#pragma unroll
    for (int w = 0; w < WARPS; w++) {
        f[w] = exp2f(out[(w * RT + r) * P + HD] - ref);
        ll += f[w] * out[(w * RT + r) * P + HD + 1];
    }
    __syncwarp();  // (a row's threads are in one warp)
    for (int x = part * 4; x < a.hd; x += PER * 4) {
        float4 v = make_float4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < WARPS; w++) {
            const float4 ow = *reinterpret_cast<const float4*>(&out[(w * RT + r) * P + x]);
            v.x += f[w] * ow.x;
            v.y += f[w] * ow.y;
            v.z += f[w] * ow.z;
            v.w += f[w] * ow.w;
        }
        *reinterpret_cast<float4*>(&out[r * P + x]) = v;
    }
    if (part == 0) {
        out[r * P + HD] = mm;
        out[r * P + HD + 1] = ll;
    }
    // ---- the runs' results: each CTA writes its share of the pieces of four columns ----
    if (a.runs > 1) cluster_sync();
    else __syncthreads();
    const int cols = a.hd / 4;
    for (int x = run * NT + tid; x < rows * cols; x += a.runs * NT) {
        const int y = x / cols, d = (x - y * cols) * 4;
        float m = -INFINITY, l = 0.0f;
        float4 v = make_float4(0, 0, 0, 0);
        if (a.runs == 1) {
            m = out[y * P + HD];
            l = out[y * P + HD + 1];
            v = *reinterpret_cast<const float4*>(&out[y * P + d]);
        } else {
            float2 ml[MAX_RUNS];
            float4 o[MAX_RUNS];
#pragma unroll
            for (int k = 0; k < MAX_RUNS; k++)
                if (k < a.runs) {
                    ml[k] = ld_cluster2(cluster_addr(&out[y * P + HD], k));
                    o[k] = ld_cluster4(cluster_addr(&out[y * P + d], k));
                }
#pragma unroll
            for (int k = 0; k < MAX_RUNS; k++)
                if (k < a.runs) m = fmaxf(m, ml[k].x);
            const float base = m == -INFINITY ? 0.0f : m;
#pragma unroll
            for (int k = 0; k < MAX_RUNS; k++)
                if (k < a.runs) {
                    const float e = exp2f(ml[k].x - base);
                    l += e * ml[k].y;
                    v.x += e * o[k].x;
                    v.y += e * o[k].y;
                    v.z += e * o[k].z;
                    v.w += e * o[k].w;
                }
        }
        const int head = h * a.G + y0 + y;
        const tc::RowEnd fin = tc::row_end(m, l, a.sink ? a.sink[head] : -INFINITY);
        const int64_t at = (int64_t)t * a.nh + head;
        if (a.lse && d == 0) a.lse[at] = fin.lse;
        *reinterpret_cast<uint2*>(a.o + at * a.hd + d) =
            make_uint2(tc::bf16x2(v.x * fin.factor, v.y * fin.factor),
                       tc::bf16x2(v.z * fin.factor, v.w * fin.factor));
    }
    pdl_trigger();
    if (a.runs > 1) cluster_sync();  // nobody leaves while its results are read
}

template <int HD, bool E4M3, int RT>
int launch_tokens(Args& a, int64_t page, const char* name, cudaStream_t st) {
    using S = Shape<HD, E4M3, RT>;
    constexpr int smem = S::BYTES;
    a.tiles = (a.G + RT - 1) / RT;
    // runs of a list: as many as the GPU holds CTAs for, of two groups a warp at least
    const int64_t items = a.Tq * a.kvh * a.tiles;
    const int64_t fit = (int64_t)sm_count_once() * S::CTAS / items;
    const int64_t most = a.topk * page / (2 * WARPS * GROUP);
    const int64_t runs = fit < most ? fit : most;
    a.runs = (int)(runs < 1 ? 1 : runs < MAX_RUNS ? runs : MAX_RUNS);
    DS41_REQUIRE(items * a.runs < int64_t(1) << 31, DS41_E_RANGE, "%s: Tq=%lld kvh=%d", name,
                 (long long)a.Tq, a.kvh);
    const unsigned ctas = (unsigned)(items * a.runs);
    if (int rc = status_word(&a.status)) return rc;
    if (int rc = allow_smem<tokens_kernel<HD, E4M3, RT>>(smem, name)) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)a.runs;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.runs > 1 ? 2 : 1;
    if (int rc = cuda_check(cudaLaunchKernelEx(&cfg, tokens_kernel<HD, E4M3, RT>, a), name)) return rc;
    return launch_check(name);
}

}  // namespace ba
}  // namespace ds41

using namespace ds41;
using few::GROUP;

extern "C" int ds41_block_attn_fwd(const ds41_bf16* q, int64_t q_tok, int64_t q_head,
                                   const void* k_cache, const void* v_cache,
                                   const float* k_scales, const float* v_scales, int fmt,
                                   int64_t n_pages, int64_t page, const int32_t* page_table,
                                   int64_t max_pages, const int32_t* lens, const int32_t* cu_q,
                                   const int32_t* idx, int64_t topk, int64_t B, int64_t Tq,
                                   int64_t max_q, int64_t nh, int64_t kvh, int64_t hd, float scale,
                                   const float* sink, ds41_bf16* o, float* lse,
                                   ds41_stream_t stream) {
    const char* name = "ds41_block_attn_fwd";
    if (int rc = check_heads(name, nh, kvh, hd, scale, 0)) return rc;
    ba::Args a{};
    if (int rc = check_paged(name, k_cache, v_cache, k_scales, v_scales, fmt, n_pages, page, kvh,
                             hd, &a.kv))
        return rc;
    DS41_REQUIRE(topk >= 1 && topk <= ba::MAX_LIST, DS41_E_ARG, "%s: topk=%lld (1 .. %d)", name,
                 (long long)topk, ba::MAX_LIST);
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
    cudaStream_t st = (cudaStream_t)stream;
    const auto launch = [&](auto hd_, auto e4m3) {
        constexpr int HD = decltype(hd_)::value;
        constexpr bool E4M3 = decltype(e4m3)::value;
        return a.G <= 8 ? ba::launch_tokens<HD, E4M3, 8>(a, page, name, st)
                        : ba::launch_tokens<HD, E4M3, 16>(a, page, name, st);
    };
    using W64 = std::integral_constant<int, 64>;
    using W128 = std::integral_constant<int, 128>;
    if (fmt == DS41_KV_E4M3)
        return hd <= 64 ? launch(W64{}, std::true_type{}) : launch(W128{}, std::true_type{});
    return hd <= 64 ? launch(W64{}, std::false_type{}) : launch(W128{}, std::false_type{});
}
