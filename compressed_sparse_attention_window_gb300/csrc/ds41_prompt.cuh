// ds41_prompt.cuh - what the tensor-core kernels over packed prompts share (all keys, picked
// blocks): tile shapes and shared memory, how a CTA takes over another's item, tensor maps.
#pragma once

#include "ds41_dense.cuh"
#include "ds41_softmax_tc.cuh"

namespace ds41 {
namespace pa {

using namespace tc;

constexpr int KB = 128;         // keys per block
constexpr int ROWS = 128;       // rows per tile
constexpr int THREADS = 384;

template <int D>
struct Cfg {
    static constexpr int NB = D / 64;                   // 64-column blocks of a row
    static constexpr uint32_t BLK = 128 * 128;          // [128 rows][64 columns] bf16
    static constexpr uint32_t TILE = NB * BLK;          // a query tile, or a K or V block
    static constexpr int STAGES = D == 128 ? 5 : 9;
    static constexpr int QB = D == 128 ? 1 : 2;         // items whose queries are held
    static constexpr uint32_t Q_OFF = 0;                // two query tiles each
    static constexpr uint32_t KV_OFF = QB * 2 * TILE;
    static constexpr uint32_t BAR_OFF = KV_OFF + STAGES * TILE;
    static constexpr uint32_t SMEM = BAR_OFF + 640 + 1024;
    static_assert(SMEM <= 232448, "shared memory budget");
};

// tensor memory columns: S_0 S_1 O_0 O_1
constexpr uint32_t TM_S = 0, TM_O = 256;

// the lowest n bits (none for n <= 0, all for n >= 32)
__device__ __forceinline__ uint32_t low_bits(int n) {
    return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// A CTA that is through with an item takes over one whose CTA has not started yet:
// the grid has a CTA for every item, and the launch queue is the list of what is
// left, longest first, so the SMs end together (items dealt out beforehand left
// one of them 7% more blocks than the average of a 16384-token prompt).
__device__ __forceinline__ void take_over(uint32_t response, uint64_t* bar) {
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    mbar_arrive_expect_tx(bar, 16);
    asm volatile(
        "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
        "[%0], [%1];\n" ::"r"(response),
        "r"(smem_u32(bar))
        : "memory");
}
// the answer: the CTA's index, or -1: all have started
__device__ __forceinline__ int taken_over(uint32_t response) {
    uint32_t got, x;
    asm volatile(
        "{\n.reg .pred p;\n.reg .b128 r;\nld.shared.b128 r, [%2];\n"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
        "selp.u32 %0, 1, 0, p;\nmov.u32 %1, 0;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n}\n"
        : "=r"(got), "=r"(x)
        : "r"(response)
        : "memory");
    return got ? (int)x : -1;
}

// Host: heads of a tile (the whole group, or its largest divisor that fits), and tiles' head
// groups per key/value head.
inline int heads_of_tile(int64_t group, int* subs) {
    int G = (int)group;
    *subs = 1;
    if (G > ROWS) {
        int d = ROWS;
        while (G % d) d--;
        *subs = G / d;
        G = d;
    }
    return G;
}

// [tokens][heads][hd] with strides in elements; a box of 64 columns x box_h
// heads x box_t tokens, 128-byte swizzle, zeros outside.
inline int make_map_heads(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* m, const void* ptr,
                   int64_t tokens, int64_t heads, int64_t hd, int64_t tok, int64_t head, int box_h,
                   int box_t) {
    cuuint64_t dims[3] = {(cuuint64_t)hd, (cuuint64_t)heads, (cuuint64_t)tokens};
    cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)tok * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)box_h, (cuuint32_t)box_t};
    cuuint32_t estr[3] = {1u, 1u, 1u};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                     box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail(DS41_E_CUDA, "cuTensorMapEncodeTiled (heads) failed (%d)", (int)r);
    return DS41_OK;
}

}  // namespace pa
}  // namespace ds41
