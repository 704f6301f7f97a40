// Residual addition with RMS norm, h = x + r, y = h * rho * gain with rho = (mean(h^2) + eps)^(-1/2), and
// its backward pass.
//
// The norm is formed from h before h is rounded to its stored type; sums are fp32. With an 8-bit output
// each group of consecutive columns (or the whole row) has scale = max |y| / 448 (1 for a group of zeros)
// and q = e4m3(y / scale).
//
// Backward, for the stored h: with d = dy * gain,
//   dx = dh + rho d - h rho^3 / dim * sum(d h),   dgain = sum over rows of dy h rho.
#include <cuda_fp8.h>

#include "row_ops.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;
constexpr float kFp8Max = 448.f;  // largest finite e4m3
constexpr float kMinScale = 1.17549435e-38f;

__device__ __forceinline__ float scale_of(unsigned top_bits) {
  const float top = __uint_as_float(top_bits);
  return top == 0.f ? 1.f : (top < kFp8Max * kMinScale ? kMinScale : top / kFp8Max);
}

// Largest |y| of the block as the bits of a non-negative float; a NaN is larger than every number.
__device__ __forceinline__ unsigned block_top(unsigned v, unsigned* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0u);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) add_rmsnorm_kernel(const RmsNormLaunch p) {
  __shared__ float red[32];
  __shared__ unsigned redu[32];
  const int64_t i = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + i * p.ldx;
  const T* r = p.residual ? static_cast<const T*>(p.residual) + i * p.ldr : nullptr;
  T* h = p.h ? static_cast<T*>(p.h) + i * p.ldh : nullptr;
  float sq = 0.f;
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) {
    const float v = row::to_f(x[c]) + (r ? row::to_f(r[c]) : 0.f);
    sq = fmaf(v, v, sq);
  }
  sq = row::block_sum(sq, red);
  const float rho = rsqrtf(sq / static_cast<float>(p.dim) + p.eps);
  auto value = [&](int64_t c) {
    const float v = row::to_f(x[c]) + (r ? row::to_f(r[c]) : 0.f);
    return v * rho * (p.gain ? p.gain[c] : 1.f);
  };
  if (!p.scales) {
    T* y = static_cast<T*>(p.y) + i * p.ldy;
    for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) {
      const float v = row::to_f(x[c]) + (r ? row::to_f(r[c]) : 0.f);
      const float yv = v * rho * (p.gain ? p.gain[c] : 1.f);
      if (h) h[c] = row::from_f<T>(v);
      y[c] = row::from_f<T>(yv);
    }
    return;
  }
  uint8_t* q = static_cast<uint8_t*>(p.y) + i * p.ldy;
  const int64_t group = p.group ? p.group : p.dim;
  const int64_t parts = (p.dim + group - 1) / group;
  for (int64_t k = 0; k < parts; ++k) {
    const int64_t begin = k * group, end = min(begin + group, p.dim);
    unsigned top = 0;
    for (int64_t c = begin + threadIdx.x; c < end; c += kThreads) top = max(top, __float_as_uint(fabsf(value(c))));
    const float scale = scale_of(block_top(top, redu));
    const float inv = 1.f / scale;
    if (threadIdx.x == 0) p.scales[i * parts + k] = scale;
    for (int64_t c = begin + threadIdx.x; c < end; c += kThreads) {
      const float v = row::to_f(x[c]) + (r ? row::to_f(r[c]) : 0.f);
      q[c] = __nv_cvt_float_to_fp8(value(c) * inv, __NV_SATFINITE, __NV_E4M3);
      if (h) h[c] = row::from_f<T>(v);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) add_rmsnorm_grad_kernel(const RmsNormGradLaunch p) {
  __shared__ float red[32];
  const int64_t i = blockIdx.x;
  const T* dy = static_cast<const T*>(p.dy) + i * p.lddy;
  const T* h = static_cast<const T*>(p.h) + i * p.ldh;
  const T* dh = p.dh ? static_cast<const T*>(p.dh) + i * p.lddh : nullptr;
  float sq = 0.f, along = 0.f;
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) {
    const float v = row::to_f(h[c]);
    sq = fmaf(v, v, sq);
    along = fmaf(row::to_f(dy[c]) * (p.gain ? p.gain[c] : 1.f), v, along);
  }
  sq = row::block_sum(sq, red);
  along = row::block_sum(along, red);
  const float rho = rsqrtf(sq / static_cast<float>(p.dim) + p.eps);
  const float back = along / static_cast<float>(p.dim) * rho * rho * rho;
  if (!p.dx) {
    if (threadIdx.x == 0) p.rho[i] = rho;
    return;
  }
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) {
    const float d = row::to_f(dy[c]) * (p.gain ? p.gain[c] : 1.f);
    static_cast<T*>(p.dx)[i * p.lddx + c] = row::from_f<T>(rho * d - back * row::to_f(h[c]) + (dh ? row::to_f(dh[c]) : 0.f));
  }
}

// One thread per column, rows in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) rmsnorm_dgain_kernel(const RmsNormGradLaunch p) {
  const int64_t c = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (c >= p.dim) return;
  const T* dy = static_cast<const T*>(p.dy) + c;
  const T* h = static_cast<const T*>(p.h) + c;
  float acc = 0.f;
  for (int64_t i = 0; i < p.n; ++i) acc = fmaf(row::to_f(dy[i * p.lddy]) * p.rho[i], row::to_f(h[i * p.ldh]), acc);
  p.dgain[c] = p.accumulate ? p.dgain[c] + acc : acc;
}

}  // namespace

cudaError_t launch_add_rmsnorm(const RmsNormLaunch& p, cudaStream_t stream) {
  if (p.dtype == 0)
    add_rmsnorm_kernel<float><<<static_cast<unsigned>(p.n), kThreads, 0, stream>>>(p);
  else
    add_rmsnorm_kernel<__nv_bfloat16><<<static_cast<unsigned>(p.n), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

int64_t rmsnorm_grad_workspace(int64_t n, int64_t dim) {
  (void)dim;
  return n * static_cast<int64_t>(sizeof(float));
}

cudaError_t launch_add_rmsnorm_grad(const RmsNormGradLaunch& p, cudaStream_t stream) {
  const unsigned rows = static_cast<unsigned>(p.n), cols = static_cast<unsigned>((p.dim + kThreads - 1) / kThreads);
  if (p.dgain) {  // before dx, which may be written over dy
    RmsNormGradLaunch only_rho = p;
    only_rho.dx = nullptr;
    if (p.dtype == 0) {
      add_rmsnorm_grad_kernel<float><<<rows, kThreads, 0, stream>>>(only_rho);
      rmsnorm_dgain_kernel<float><<<cols, kThreads, 0, stream>>>(p);
    } else {
      add_rmsnorm_grad_kernel<__nv_bfloat16><<<rows, kThreads, 0, stream>>>(only_rho);
      rmsnorm_dgain_kernel<__nv_bfloat16><<<cols, kThreads, 0, stream>>>(p);
    }
  }
  if (p.dtype == 0)
    add_rmsnorm_grad_kernel<float><<<rows, kThreads, 0, stream>>>(p);
  else
    add_rmsnorm_grad_kernel<__nv_bfloat16><<<rows, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dmuon
