// tensor_map.cuh -- the tensor maps of all kernels: a cache or page pool
// [rows][8][64], fp32 or bf16, as the 2-D tensor (head * 64 + d, row).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "common.cuh"

namespace attn {

// The driver's tensor-map encoder, looked up once (a function-local static is
// initialised once even when the first calls come from several threads).
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  return fn;
}

// A box is 128 bytes (one swizzle row: 32 fp32 or 64 bf16 dims of a head) of
// box_rows rows. Returns an ATTN_* code.
inline int encode_rows_map(const void* base, bool bf16, long long rows, int box_rows, CUtensorMapSwizzle swizzle,
                           CUtensorMap* map) {
  const auto enc = tensor_map_encoder();
  if (!enc) return ATTN_ETMA;
  const cuuint32_t ones[2] = {1, 1};
  const cuuint64_t dims[2] = {(cuuint64_t)kHKV * kD, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)kHKV * kD * (bf16 ? 2 : 4)};
  const cuuint32_t box[2] = {bf16 ? 64u : 32u, (cuuint32_t)box_rows};
  const auto encode = [&] {
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
               const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  int dev = 0;
  // A thread whose first CUDA call this is has no context yet; a runtime call
  // would bind one, the driver's encoder does not.
  if (r == CUDA_ERROR_INVALID_CONTEXT && cudaGetDevice(&dev) == cudaSuccess && cudaSetDevice(dev) == cudaSuccess)
    r = encode();
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ETMA;
}

}  // namespace attn
