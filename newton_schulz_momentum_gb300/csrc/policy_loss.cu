// Clipped policy loss with a KL term, from logits, with its gradient; and token log-probabilities.
//
// Per row t with logits x, token a, temperature T: z = x / T, lp = z_a - log sum exp z, ratio
// r = exp(lp - old), d = ref - lp,
//   l = -min(r A, clip(r, 1 - lo, 1 + hi) A) + k (exp(d) - d - 1),   loss = sum of w l over the rows,
//   c = d(loss)/d(lp) = w (-A r [r A <= clip(r) A] + k (1 - exp(d))),
//   d(loss)/dx = c / T (onehot(a) - softmax(z)).
// A row of weight 0 or with a negative token is not read: its terms and gradient are 0.
#include "row_ops.h"

namespace dmuon {
namespace {

constexpr int kThreads = 512;
constexpr float kLog2e = 1.4426950408889634f;

// The largest logit m and s = sum of 2^((x - m) k), k = log2(e) / T. The difference is formed before the
// product: it is exact for the largest logit, and small where the terms are large. Against a maximum of
// -infinity (masked logits so far) terms are taken from 0, so that -infinity adds 0 and not NaN.
struct MaxSum {
  float m, s;
};

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float k) {
  const float m = fmaxf(a.m, b.m), base = finite_or_zero(m);
  return {m, a.s * exp2f((a.m - base) * k) + b.s * exp2f((b.m - base) * k)};
}

struct RowTerms {
  float loss, coef;
};

__device__ __forceinline__ RowTerms row_terms(const PolicyLaunch& p, int64_t i, float logp) {
  const float w = p.weights[i], adv = p.advantages[i];
  const float r = expf(logp - p.old_logp[i]);
  const float whole = r * adv, cut = fminf(fmaxf(r, 1.f - p.clip_low), 1.f + p.clip_high) * adv;
  float each = -fminf(whole, cut);
  if (isnan(whole)) each = whole;
  float c = whole <= cut || isnan(whole) ? -whole : 0.f;
  if (p.ref_logp) {
    const float d = p.ref_logp[i] - logp, e = expm1f(d);
    each = fmaf(p.kl_coef, e - d, each);
    c = fmaf(-p.kl_coef, e, c);
  }
  return {each * w, c * w};
}

template <typename T>
__global__ void __launch_bounds__(kThreads) policy_row_kernel(const PolicyLaunch p) {
  __shared__ MaxSum part[kThreads / 32];
  const int64_t i = blockIdx.x;
  const int64_t a = row::load_id(p.targets, p.id_bytes, i);
  const T* x = static_cast<const T*>(p.logits) + i * p.ld;
  T* dx = p.dlogits ? static_cast<T*>(p.dlogits) + i * p.ldd : nullptr;
  bool live = a >= 0 && (!p.weights || p.weights[i] != 0.f);
  if (live && a >= p.vocab) {
    if (threadIdx.x == 0) atomicOr(p.status, kDevIndex);
    live = false;
  }
  if (!live) {
    if (threadIdx.x == 0) {
      if (p.logp) p.logp[i] = 0.f;
      if (p.row_loss) p.row_loss[i] = 0.f;
    }
    if (dx)
      for (int64_t c = threadIdx.x; c < p.vocab; c += kThreads) dx[c] = row::from_f<T>(0.f);
    return;
  }
  const float k = kLog2e / p.temperature;
  MaxSum t{-INFINITY, 0.f};
  for (int64_t c = threadIdx.x; c < p.vocab; c += kThreads) t = join(t, {row::to_f(x[c]), 1.f}, k);
  for (int o = 16; o > 0; o >>= 1)
    t = join(t, {__shfl_xor_sync(0xffffffffu, t.m, o), __shfl_xor_sync(0xffffffffu, t.s, o)}, k);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = t;
  const float xa = row::to_f(x[a]);  // read before any thread writes a gradient over it
  __syncthreads();
  t = part[0];
  for (int w = 1; w < kThreads / 32; ++w) t = join(t, part[w], k);
  const float logp = (xa - t.m) / p.temperature - logf(t.s);  // exactly 0 for the only token left
  float coef = 0.f;
  if (p.weights) {
    const RowTerms rt = row_terms(p, i, logp);
    coef = rt.coef;
    if (threadIdx.x == 0) p.row_loss[i] = rt.loss;
  }
  if (threadIdx.x == 0 && p.logp) p.logp[i] = logp;
  if (!dx) return;
  const float scale = coef / p.temperature, per = -scale / t.s;
  for (int64_t c = threadIdx.x; c < p.vocab; c += kThreads) {
    const float e = per * exp2f((row::to_f(x[c]) - finite_or_zero(t.m)) * k);
    dx[c] = row::from_f<T>(c == a ? e + scale : e);
  }
}

__global__ void __launch_bounds__(kThreads) policy_sum_kernel(const PolicyLaunch p) {
  __shared__ float red[32];
  float acc = 0.f;
  for (int64_t i = threadIdx.x; i < p.n; i += kThreads) acc += p.row_loss[i];
  acc = row::block_sum(acc, red);
  if (threadIdx.x == 0) *p.loss = acc;
}

}  // namespace

cudaError_t launch_policy(const PolicyLaunch& p, cudaStream_t stream) {
  if (p.n > 0) {
    if (p.dtype == 0)
      policy_row_kernel<float><<<static_cast<unsigned>(p.n), kThreads, 0, stream>>>(p);
    else
      policy_row_kernel<__nv_bfloat16><<<static_cast<unsigned>(p.n), kThreads, 0, stream>>>(p);
  }
  if (p.loss) policy_sum_kernel<<<1, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dmuon
