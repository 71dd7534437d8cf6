// TMA descriptor encoding through the driver entry point (resolved at run
// time, so the library needs no link against libcuda).
#include "gemm_host.h"
#include "host_util.h"

namespace moe {
namespace {

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (fn == nullptr) {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(f);
  }
  return fn;
}

// 16-bit values are moved as such, whatever they stand for; fp32 is named so
// that it can be added to.
int make_tmap16(CUtensorMap* tm, const void* base, uint32_t rank, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box,
                CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_UINT16,
                CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return MOE_ERR_CUDA;
  }
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(tm, type, rank, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace

int make_tmap_rows16(CUtensorMap* tm, const void* base, uint64_t width, uint64_t rows, uint64_t ld,
                     uint32_t box_rows) {
  const cuuint64_t dims[2] = {width, rows};
  const cuuint64_t strides[1] = {ld * 2};
  const cuuint32_t box[2] = {64u, box_rows};
  return make_tmap16(tm, base, 2, dims, strides, box);
}

int make_tmap_weights16(CUtensorMap* tm, const void* base, uint64_t Kd, uint64_t N, uint64_t E,
                        uint32_t box_n) {
  const cuuint64_t dims[3] = {Kd, N, E};
  const cuuint64_t strides[2] = {Kd * 2, N * Kd * 2};
  const cuuint32_t box[3] = {64u, box_n, 1u};
  return make_tmap16(tm, base, 3, dims, strides, box);
}

int make_tmap_result(CUtensorMap* tm, void* base, bool f32, uint64_t width, uint64_t rows, uint64_t E,
                     uint64_t ld) {
  const uint64_t size = f32 ? 4 : 2;
  const cuuint64_t dims[3] = {width, rows, E};
  const cuuint64_t strides[2] = {ld * size, rows * ld * size};
  const cuuint32_t box[3] = {f32 ? 16u : 32u, 32u, 1u};
  return make_tmap16(tm, base, 3, dims, strides, box,
                     f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16,
                     CU_TENSOR_MAP_SWIZZLE_64B);
}

int make_tmap_codes4(CUtensorMap* tm, const void* base, uint64_t row_bytes, uint64_t rows,
                     uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return MOE_ERR_CUDA;
  }
  const cuuint64_t dims[2] = {row_bytes, rows};
  const cuuint64_t strides[1] = {row_bytes};
  const cuuint32_t box[2] = {64u, box_rows};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

int make_tmap_k128(CUtensorMap* tm, const void* base, uint64_t inner, uint64_t outer,
                   uint64_t stride, uint32_t box_outer) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) {
    set_error("cuTensorMapEncodeTiled is not available from the driver");
    return MOE_ERR_CUDA;
  }
  const cuuint64_t dims[2] = {inner, outer};
  const cuuint64_t strides[1] = {stride};
  const cuuint32_t box[2] = {128u, box_outer};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    set_error("cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace moe
