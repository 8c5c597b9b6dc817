// tensor_map.cu -- TMA tensor maps of the streaming attention calls.
#include <cuda.h>
#include <cuda_runtime.h>

#include <mutex>

#include "stream.h"

namespace svga {

typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

void *encode_tiled_entry()
{
    static void *fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = f;
    });
    return fn;
}

static CUtensorMapDataType map_type(svga_dtype dt)
{
    return dt == SVGA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

bool make_view_map(void *map, const svga_view &v, int batch, int heads, int tokens, int d,
                   svga_dtype dt, int box_rows, int *mul_h, int *mul_b)
{
    EncodeTiled enc = reinterpret_cast<EncodeTiled>(encode_tiled_entry());
    if (!enc) return false;
    *mul_h = heads > 1 && v.stride_head != 0;
    *mul_b = batch > 1 && v.stride_batch != 0;
    // a dimension of one entry never uses its stride: any valid one will do
    const cuuint64_t row = (cuuint64_t)d * 2;
    const bool tok = tokens > 1 && v.stride_token != 0;
    const cuuint64_t dims[5] = {64, (cuuint64_t)tokens, (cuuint64_t)(d / 64),
                                (cuuint64_t)(*mul_h ? heads : 1), (cuuint64_t)(*mul_b ? batch : 1)};
    const cuuint64_t strides[4] = {tok ? (cuuint64_t)v.stride_token * 2 : row, 128,
                                   *mul_h ? (cuuint64_t)v.stride_head * 2 : row,
                                   *mul_b ? (cuuint64_t)v.stride_batch * 2 : row};
    const cuuint32_t box[5] = {64, (cuuint32_t)box_rows, (cuuint32_t)(d / 64), 1, 1};
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return enc(static_cast<CUtensorMap *>(map), map_type(dt), 5, v.data, dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_rows_map(void *map, const void *base, long long rows, int d, svga_dtype dt, int box_rows)
{
    EncodeTiled enc = reinterpret_cast<EncodeTiled>(encode_tiled_entry());
    if (!enc) return false;
    const cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)(d / 64)};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, 128};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_rows, (cuuint32_t)(d / 64)};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(static_cast<CUtensorMap *>(map), map_type(dt), 3, const_cast<void *>(base), dims,
               strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace svga
