// Element access and block reductions shared by the token operators (embedding.cu, rmsnorm.cu,
// policy_loss.cu). Device code only.
#pragma once

#include <cuda_bf16.h>

#include "internal.h"

namespace dmuon {
namespace row {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Token id `i` of an int32 or int64 list.
__device__ __forceinline__ int64_t load_id(const void* ids, int id_bytes, int64_t i) {
  return id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<int64_t>(static_cast<const int*>(ids)[i]);
}

// Sum over the block, in an order fixed by the block size alone; every thread gets it. `red` holds 32
// floats. Called by all threads.
__device__ __forceinline__ float block_sum(float v, float* red) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();  // the previous use of red is over
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nwarps = (blockDim.x + 31) >> 5;
  v = (threadIdx.x & 31) < nwarps ? red[threadIdx.x & 31] : 0.f;
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace row
}  // namespace dmuon
