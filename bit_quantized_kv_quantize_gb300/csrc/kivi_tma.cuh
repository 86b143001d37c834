// kivi_tma.cuh -- TMA tile copies of fp16 [rows][D] arrays into chunk-major
// core-matrix tiles: the tensor maps (host) and the copy (device).
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kivi_mma.cuh"

namespace {

// one TMA tile copy (rows row0.. of the tensor map's array, all D columns)
// into dst, completing `bytes` on bar (one thread)
__device__ __forceinline__ void tma_tile(void *dst, const CUtensorMap *tm, int row0, uint64_t *bar,
                                         unsigned bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
                 : "memory");
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(tm), "r"(0), "r"(row0), "r"(0), "r"(smem_u32(bar))
        : "memory");
}

// The encoder of TMA tensor maps, from the driver (through the runtime, no
// link to the driver library); null if unavailable.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
                cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// Tensor map over an fp16 [rows][D] array giving chunk-major core-matrix
// tiles of box_rows rows (16-byte chunk c of row r at
// byte c box_rows 16 + r 16): dimensions (8, rows, D / 8), strides
// (2 D bytes, 16 bytes), box (8, box_rows, D / 8).
cudaError_t make_tile_map(CUtensorMap *tm, const __half *base, long long rows, int D, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dim[3] = {8, (cuuint64_t)rows, (cuuint64_t)(D / 8)};
    const cuuint64_t str[2] = {(cuuint64_t)D * 2, 16};
    const cuuint32_t box[3] = {8, (cuuint32_t)box_rows, (cuuint32_t)(D / 8)};
    const cuuint32_t es[3] = {1, 1, 1};
    const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half *>(base), dim, str, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tensor map over an fp16 [rows][cols] array giving tiles of box_rows rows x 64
// columns in the 128-byte swizzle.
cudaError_t make_sw_map(CUtensorMap *tm, const __half *base, long long rows, int cols, int box_rows) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t dim[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t str[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)box_rows};
    const cuuint32_t es[2] = {1, 1};
    const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half *>(base), dim, str, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// one such tile, from row row0 and column col0 (a multiple of 8) on
__device__ __forceinline__ void tma_sw(void *dst, const CUtensorMap *tm, int col0, int row0, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(tm), "r"(col0), "r"(row0), "r"(smem_u32(bar))
        : "memory");
}

// Tensor map over queries [heads / hg][hg][n][D] whose boxes are 128 rows
// (token r, head e of a group), e fastest, in chunk-major order: dimensions
// (8, hg, n, D / 8, heads / hg), box (8, hg, 128 / hg, D / 8, 1).
cudaError_t make_group_rows_map(CUtensorMap *tm, const __half *base, long long groups, int hg, int n, int D) {
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    const cuuint64_t row = (cuuint64_t)D * 2;
    const cuuint64_t dim[5] = {8, (cuuint64_t)hg, (cuuint64_t)n, (cuuint64_t)(D / 8), (cuuint64_t)groups};
    const cuuint64_t str[4] = {row * n, row, 16, row * n * hg};
    const cuuint32_t box[5] = {8, (cuuint32_t)hg, (cuuint32_t)(128 / hg), (cuuint32_t)(D / 8), 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 5, const_cast<__half *>(base), dim, str, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace
