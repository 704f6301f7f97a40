// Embedding lookup with scaling, out[i, :] = scale * table[id_i, :], and its gradient,
// grad[v, :] = scale * sum over the tokens i with id_i = v of grad_out[i, :], added in the order of i.
#include "row_ops.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;

template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const EmbeddingLaunch p) {
  const int64_t i = blockIdx.x;
  const int64_t id = row::load_id(p.ids, p.id_bytes, i);
  const bool ok = id >= 0 && id < p.rows;
  if (!ok && threadIdx.x == 0) atomicOr(p.status, kDevIndex);
  const TI* src = static_cast<const TI*>(p.table) + (ok ? id : 0) * p.ld_table;
  TO* dst = static_cast<TO*>(p.out) + i * p.ld_out;
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads)
    dst[c] = row::from_f<TO>(ok ? p.scale * row::to_f(src[c]) : 0.f);
}

// One CTA per table row: it goes over all ids and adds the rows of its tokens, in their order.
template <typename TG>
__global__ void __launch_bounds__(kThreads) embedding_grad_kernel(const EmbeddingGradLaunch p) {
  __shared__ int list[kThreads];
  __shared__ int warp_count[kThreads / 32];
  const int64_t v = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const TG* g = static_cast<const TG*>(p.grad_out);
  float* dst = p.grad + v * p.ld_grad;
  for (int64_t c0 = 0; c0 < p.dim; c0 += kThreads) {
    const int64_t c = c0 + threadIdx.x;
    float acc = 0.f;
    for (int64_t i0 = 0; i0 < p.n; i0 += kThreads) {
      const int64_t i = i0 + threadIdx.x;
      const int64_t id = i < p.n ? row::load_id(p.ids, p.id_bytes, i) : -1;
      if (i < p.n && v == 0 && c0 == 0 && (id < 0 || id >= p.rows)) atomicOr(p.status, kDevIndex);
      const bool mine = i < p.n && id == v && v != p.padding_idx;
      const unsigned votes = __ballot_sync(0xffffffffu, mine);
      if (lane == 0) warp_count[warp] = __popc(votes);
      __syncthreads();
      int at = __popc(votes & ((1u << lane) - 1)), total = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) at += warp_count[w];
        total += warp_count[w];
      }
      if (mine) list[at] = threadIdx.x;
      __syncthreads();
      if (c < p.dim)
        for (int k = 0; k < total; ++k) acc += row::to_f(g[(i0 + list[k]) * p.ld_grad_out + c]);
      __syncthreads();
    }
    if (c < p.dim) dst[c] = p.accumulate ? fmaf(p.scale, acc, dst[c]) : p.scale * acc;
  }
}

}  // namespace

cudaError_t launch_embedding(const EmbeddingLaunch& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.n);
  if (p.table_dtype == 0 && p.out_dtype == 0)
    embedding_kernel<float, float><<<grid, kThreads, 0, stream>>>(p);
  else if (p.table_dtype == 0)
    embedding_kernel<float, __nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
  else if (p.out_dtype == 0)
    embedding_kernel<__nv_bfloat16, float><<<grid, kThreads, 0, stream>>>(p);
  else
    embedding_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_embedding_grad(const EmbeddingGradLaunch& p, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.rows);
  if (p.grad_dtype == 0)
    embedding_grad_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  else
    embedding_grad_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dmuon
