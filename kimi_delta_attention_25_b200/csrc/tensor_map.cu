// tensor_map.cu -- tensor maps of bf16 rows with strides, for the latent attention's copies.
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

#include "kda_internal.cuh"

namespace kda {
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, []() {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    return fn;
}

bool bf16_map(CUtensorMap *m, const void *base, uint32_t rank, const cuuint64_t *dims, const cuuint64_t *strides,
              uint32_t box_cols, uint32_t box_rows)
{
    const PFN_cuTensorMapEncodeTiled_v12000 fn = encoder();
    if (!fn) return false;
    const cuuint32_t box[3] = {box_cols, box_rows, 1u}, estr[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool bf16_rows_map(CUtensorMap *m, const void *base, long long cols, long long rows, long long row_stride,
                   uint32_t box_cols, uint32_t box_rows)
{
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows}, strides[1] = {(cuuint64_t)row_stride * 2};
    return bf16_map(m, base, 2, dims, strides, box_cols, box_rows);
}

bool bf16_heads_map(CUtensorMap *m, const void *base, long long cols, long long heads, long long rows,
                    long long head_stride, long long row_stride, uint32_t box_cols, uint32_t box_rows)
{
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)heads};
    const cuuint64_t strides[2] = {(cuuint64_t)row_stride * 2, (cuuint64_t)head_stride * 2};
    return bf16_map(m, base, 3, dims, strides, box_cols, box_rows);
}

}  // namespace kda
