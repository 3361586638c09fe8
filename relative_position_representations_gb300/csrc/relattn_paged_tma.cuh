// Tensor maps over the pages of the cache, for the paged attention kernels that load by TMA.
#pragma once

#include "relattn_paged.cuh"
#include "relattn_tc_launch.cuh"

namespace relattn {
namespace paged {

// k_pages or v_pages as [num_pages][Hkv][page_size][d], box of 64 columns x `box` keys with
// 128-byte swizzle. A box at page num_pages lies outside the tensor and reads as zeros.
inline bool make_page_map(CUtensorMap *m, const void *ptr, const PagedArgs &a, int box) {
    tc::EncodeTiledFn enc = tc::encode_fn();
    if (!enc) return false;
    const cuuint64_t dim[4] = {(cuuint64_t)a.d, (cuuint64_t)a.page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
    const cuuint64_t stride[3] = {(cuuint64_t)a.d * 2, (cuuint64_t)a.page_size * a.d * 2, (cuuint64_t)a.page_stride * 2};
    const cuuint32_t bx[4] = {64, (cuuint32_t)box, 1, 1}, es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(ptr), dim, stride, bx, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q as [tokens][H][d], box of 64 columns x g heads x T tokens: the rows of a tile, token by token
inline bool make_query_map(CUtensorMap *m, const PagedArgs &a, int g, int T) {
    tc::EncodeTiledFn enc = tc::encode_fn();
    if (!enc) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)a.d, (cuuint64_t)a.H, (cuuint64_t)a.tokens};
    const cuuint64_t stride[2] = {(cuuint64_t)a.d * 2, (cuuint64_t)a.q_stride * 2};
    const cuuint32_t bx[3] = {64, (cuuint32_t)g, (cuuint32_t)T}, es[3] = {1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(a.q), dim, stride, bx, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16, d = 64 or 128, boxes of whole 8-row swizzle atoms, rows and strides that TMA can address
inline bool pages_by_tma(const PagedArgs &a) {
    return a.bf16 && (a.d == 64 || a.d == 128) && a.page_size >= 8 && a.page_stride < (1LL << 38) &&
           a.q_stride < (1LL << 38) && a.ths < (1LL << 38) && wide_rows(a);
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *tm, uint32_t bar, int c0, int c1, int c2,
                                            int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

}  // namespace paged
}  // namespace relattn
