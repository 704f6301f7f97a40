// Attention over whole prompts, sequences packed one behind the other, query heads in groups that share a key head; and
// its backward pass.
//
// Per sequence and query head, over the keys j of the same sequence (j <= i if causal): x_ij = scale q_i . k_j,
// p = softmax of a row of x, o_i = sum p_ij v_j, lse_i = log sum exp x_ij. Backward, with D_i = do_i . o_i:
//   dv_j = sum p_ij do_i,  ds_ij = p_ij (do_i . v_j - D_i),  dq_i = scale sum ds_ij k_j,  dk_j = scale sum ds_ij q_i,
// the last two of a key head over all of its query heads.
//
// One warp per row of the result, its elements spread over the lanes.
#include <algorithm>

#include "row_ops.h"
#include "tc_ptx.h"

namespace dmuon {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Sequence of a token: [begin, end), empty where the token lies in none.
__device__ __forceinline__ void sequence_of(const AttentionLaunch& p, int64_t token, int64_t* begin, int64_t* end) {
  if (!p.offsets) {
    const int64_t len = p.n / p.sequences;
    *begin = token / len * len;
    *end = *begin + len;
    return;
  }
  int64_t lo = 0, hi = p.sequences;  // the last offset that is not behind the token
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (row::load_id(p.offsets, p.id_bytes, mid) <= token) lo = mid;
    else hi = mid - 1;
  }
  const int64_t b = row::load_id(p.offsets, p.id_bytes, lo);
  const int64_t e = lo < p.sequences ? row::load_id(p.offsets, p.id_bytes, lo + 1) : 0;
  *begin = b < 0 ? 0 : b;
  *end = token < b ? token : e > p.n ? p.n : e;
}

struct Row4 {
  float v[4];
};

__device__ __forceinline__ Row4 load4(const bf16* x, int dim) {
  Row4 r;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (threadIdx.x & 31) + 32 * k;
    r.v[k] = c < dim ? row::to_f(x[c]) : 0.f;
  }
  return r;
}

__device__ __forceinline__ void store4(bf16* x, int dim, const Row4& r) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int c = (threadIdx.x & 31) + 32 * k;
    if (c < dim) x[c] = row::from_f<bf16>(r.v[k]);
  }
}

__device__ __forceinline__ float dot(const Row4& a, const Row4& b) {
  float s = a.v[0] * b.v[0] + a.v[1] * b.v[1] + a.v[2] * b.v[2] + a.v[3] * b.v[3];
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ const bf16* at(const HeadArray& a, int64_t token, int64_t head) {
  return static_cast<const bf16*>(a.data) + token * a.token + head * a.head;
}
__device__ __forceinline__ bf16* out_at(const HeadArray& a, int64_t token, int64_t head) {
  return static_cast<bf16*>(const_cast<void*>(a.data)) + token * a.token + head * a.head;
}

__global__ void __launch_bounds__(kThreads) attention_kernel(const __grid_constant__ AttentionLaunch p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= p.n * p.heads) return;
  const int64_t token = unit / p.heads, head = unit % p.heads, kv = head / (p.heads / p.kv_heads);
  int64_t begin, end;
  sequence_of(p, token, &begin, &end);
  if (token >= end) {
    if (p.zero_outside) {
      store4(out_at(p.out, token, head), p.dim, Row4{});
      if ((threadIdx.x & 31) == 0) p.lse[head * p.n + token] = 0.f;
    }
    return;
  }
  const Row4 q = load4(at(p.q, token, head), p.dim);
  float m = -INFINITY, s = 0.f;
  Row4 o{};
  const int64_t last = p.causal ? token + 1 : end;
  for (int64_t j = begin; j < last; ++j) {
    const float x = dot(q, load4(at(p.k, j, kv), p.dim)) * p.scale, top = fmaxf(m, x);
    const float base = top == -INFINITY ? 0.f : top, f = expf(m - base), e = expf(x - base);
    const Row4 v = load4(at(p.v, j, kv), p.dim);
    s = fmaf(s, f, e);
#pragma unroll
    for (int k = 0; k < 4; ++k) o.v[k] = fmaf(o.v[k], f, e * v.v[k]);
    m = top;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) o.v[k] /= s;
  store4(out_at(p.out, token, head), p.dim, o);
  if ((threadIdx.x & 31) == 0) p.lse[head * p.n + token] = m + logf(s);
}

// D of every row.
__global__ void __launch_bounds__(kThreads) attention_delta_kernel(const __grid_constant__ AttentionLaunch p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= p.n * p.heads) return;
  const int64_t token = unit / p.heads, head = unit % p.heads;
  const float d = dot(load4(at(p.out, token, head), p.dim), load4(at(p.dout, token, head), p.dim));
  if ((threadIdx.x & 31) == 0) p.delta[head * p.n + token] = d;
}

__global__ void __launch_bounds__(kThreads) attention_dq_kernel(const __grid_constant__ AttentionLaunch p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= p.n * p.heads) return;
  const int64_t token = unit / p.heads, head = unit % p.heads, kv = head / (p.heads / p.kv_heads);
  int64_t begin, end;
  sequence_of(p, token, &begin, &end);
  if (token >= end) {
    if (p.zero_outside) store4(out_at(p.dq, token, head), p.dim, Row4{});
    return;
  }
  const Row4 q = load4(at(p.q, token, head), p.dim), g = load4(at(p.dout, token, head), p.dim);
  const float lse = p.lse[head * p.n + token], delta = p.delta[head * p.n + token];
  Row4 d{};
  const int64_t last = p.causal ? token + 1 : end;
  for (int64_t j = begin; j < last; ++j) {
    const Row4 k = load4(at(p.k, j, kv), p.dim);
    const float e = expf(dot(q, k) * p.scale - lse);
    const float ds = e * (dot(g, load4(at(p.v, j, kv), p.dim)) - delta) * p.scale;
#pragma unroll
    for (int c = 0; c < 4; ++c) d.v[c] = fmaf(ds, k.v[c], d.v[c]);
  }
  store4(out_at(p.dq, token, head), p.dim, d);
}

__global__ void __launch_bounds__(kThreads) attention_dkv_kernel(const __grid_constant__ AttentionLaunch p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (unit >= p.n * p.kv_heads) return;
  const int64_t token = unit / p.kv_heads, kv = unit % p.kv_heads, group = p.heads / p.kv_heads;
  int64_t begin, end;
  sequence_of(p, token, &begin, &end);
  if (token >= end) {
    if (p.zero_outside) {
      store4(out_at(p.dk, token, kv), p.dim, Row4{});
      store4(out_at(p.dv, token, kv), p.dim, Row4{});
    }
    return;
  }
  const Row4 k = load4(at(p.k, token, kv), p.dim), v = load4(at(p.v, token, kv), p.dim);
  Row4 dk{}, dv{};
  for (int64_t head = kv * group; head < (kv + 1) * group; ++head)
    for (int64_t i = p.causal ? token : begin; i < end; ++i) {
      const Row4 q = load4(at(p.q, i, head), p.dim), g = load4(at(p.dout, i, head), p.dim);
      const float e = expf(dot(q, k) * p.scale - p.lse[head * p.n + i]);
      const float ds = e * (dot(g, v) - p.delta[head * p.n + i]) * p.scale;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        dv.v[c] = fmaf(e, g.v[c], dv.v[c]);
        dk.v[c] = fmaf(ds, q.v[c], dk.v[c]);
      }
    }
  store4(out_at(p.dk, token, kv), p.dim, dk);
  store4(out_at(p.dv, token, kv), p.dim, dv);
}

unsigned ctas_for(int64_t units) { return static_cast<unsigned>((units + kWarps - 1) / kWarps); }

}  // namespace

int64_t attention_workspace(AttentionLaunch& p, char* ws) {
  if (ws) p.delta = reinterpret_cast<float*>(ws);
  return static_cast<int64_t>(sizeof(float)) * p.n * p.heads;
}

cudaError_t launch_attention(AttentionLaunch& p, int sms, cudaStream_t stream) {
  return row::launch(attention_kernel, dim3(ctas_for(p.n * p.heads)), kThreads, 0, stream, p);
}

cudaError_t launch_attention_grad(AttentionLaunch& p, int sms, cudaStream_t stream) {
  cudaError_t e = row::launch(attention_delta_kernel, dim3(ctas_for(p.n * p.heads)), kThreads, 0, stream, p);
  if (e == cudaSuccess) e = row::launch(attention_dq_kernel, dim3(ctas_for(p.n * p.heads)), kThreads, 0, stream, p);
  if (e == cudaSuccess) e = row::launch(attention_dkv_kernel, dim3(ctas_for(p.n * p.kv_heads)), kThreads, 0, stream, p);
  return e;
}

}  // namespace dmuon
