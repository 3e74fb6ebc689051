// Tensor maps of the attention's arrays and of the dense layer's matrices.
#include <atomic>

#include "attn.cuh"
#include "layers.cuh"

namespace ob {
namespace {

// The driver's encoder, through the runtime: the library links no libcuda.
using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                            const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encoder(Encode* out) {
  static std::atomic<Encode> known{nullptr};  // two threads may both ask the first time
  *out = known.load(std::memory_order_acquire);
  if (*out) return cudaSuccess;
  void* f = nullptr;
  cudaDriverEntryPointQueryResult found;
  const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                         cudaEnableDefault, &found);
  if (e != cudaSuccess) return e;
  if (found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
  *out = reinterpret_cast<Encode>(f);
  known.store(*out, std::memory_order_release);
  return cudaSuccess;
}

// What call() returns; where this thread has no context yet (its first call, of autograd's
// threads for one), once more with the current device's.
template <typename F>
cudaError_t encoded(F call) {
  CUresult r = call();
  int dev = 0;
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess &&
      cudaSetDevice(dev) == cudaSuccess)
    r = call();
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

CUtensorMapDataType map_type(int type) {
  return type == OB_TYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

}  // namespace

cudaError_t attn_tensor_map(CUtensorMap* map, const Heads& t, int type, int D, int L, int H, int B,
                            int rows) {
  Encode encode = nullptr;
  const cudaError_t e = encoder(&encode);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)L, (cuuint64_t)H, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)t.l * 2, (cuuint64_t)t.h * 2, (cuuint64_t)t.b * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, step[4] = {1, 1, 1, 1};
  return encoded([&] {
    return encode(map, map_type(type), 4, t.data, dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

cudaError_t matrix_tensor_map(CUtensorMap* map, const Mat& m, int type, int64_t rows, int64_t cols,
                              int box_cols, int box_rows) {
  Encode encode = nullptr;
  const cudaError_t e = encoder(&encode);
  if (e != cudaSuccess) return e;
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)m.ld * 2};
  const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows}, step[2] = {1, 1};
  return encoded([&] {
    return encode(map, map_type(type), 2, m.data, dims, strides, box, step,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  });
}

}  // namespace ob
