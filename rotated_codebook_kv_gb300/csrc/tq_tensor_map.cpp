// tq_tensor_map.cpp -- host-side encoding of the tensor maps through which the bf16 and
// 8-bit page pools are read.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

#include "tq_internal.h"

namespace tq {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder(cudaError_t *err)
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static cudaError_t e = cudaSuccess;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q);
        if (e == cudaSuccess && q != cudaDriverEntryPointSuccess) e = cudaErrorSymbolNotFound;
        fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    *err = e;
    return fn;
}

}  // namespace

bool encode_pool_map(CUtensorMap *tm, const void *pool, bool bf16, int cols, int64_t rows, int box_cols, int box_rows,
                     cudaError_t *err)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder(err);
    if (!enc) return false;
    const cuuint64_t gdim[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t gstride[1] = {static_cast<cuuint64_t>(cols) * (bf16 ? 2 : 1)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(tm, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                           const_cast<void *>(pool), gdim, gstride, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        *err = cudaErrorInvalidValue;
        return false;
    }
    return true;
}

bool encode_row_blocks_map(CUtensorMap *tm, const void *rows, int cols, int64_t num_rows, int box_rows, int box_blocks, cudaError_t *err)
{
    PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder(err);
    if (!enc) return false;
    const cuuint64_t gdim[3] = {64, static_cast<cuuint64_t>(num_rows), static_cast<cuuint64_t>(cols / 64)};
    const cuuint64_t gstride[2] = {static_cast<cuuint64_t>(cols) * 2, 128};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(box_blocks)};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(rows), gdim, gstride, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        *err = cudaErrorInvalidValue;
        return false;
    }
    return true;
}

}  // namespace tq
