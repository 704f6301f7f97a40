// Log-probabilities of given tokens with the entropy and the most likely alternatives of their distributions, from
// logits; and the gradient of the first two.
//
// Per row with logits x, token a, temperature T, z = x / T, m = max x: s = sum of exp((x - m) / T),
//   lp_j = z_j - m / T - log s,   H = -sum of p lp = log s - sum of ((x - m) / T) exp((x - m) / T) / s,
// and the `top` largest logits with their columns, the lowest column first among equals. Backward, for g = dL/dlp_a and
// h = dL/dH:  dL/dx_j = 1 / T (g (1[j = a] - p_j) - h p_j (lp_j + H)).
//
// A row is read once for all of it. The threads of a CTA (of a cluster's CTAs where there are few rows) each keep the
// largest logit of their own granules and, with k = log2(e) / T and c = m k as rounded, s = sum of 2^(x k - c) and
// u = sum of (x k - c) 2^(x k - c), rescaled where the largest logit grows; they join them at the end, where what the
// rounding of c left is taken out again (m k - c, which fma gives exactly). Logits of -infinity, and those below
// `low` = -2^126 (T times that below T = 1.44), are taken as `low`, so that no product is infinity times 0.
//
// The alternatives come from a bound: the threads form 64 groups (32 in a CTA of one warp), at least `top` of which hold
// an element as large as the top-th largest of the groups' maxima, so only elements that reach it can be alternatives: a
// few more than `top` of them as a rule, in as many threads, whose granules alone are read again. Where equal logits make
// them more than the list holds, the row is walked once more in order, the list cut down to its `top` best whenever it
// is full.
//
// What bounds them is memory. Measured, bf16: 8192 rows of 128256, of which 85 in 100 count, with 5 alternatives 317 us, 5.6
// TB/s (0.84 of a copy's rate; the way from a row's last loads to its results takes 4 to 5 us of 27); 8 rows with 20
// alternatives 7 us in clusters of eight. Backward, 4096 rows: 296 us, 0.98 of a copy's rate.
#include <algorithm>

#include "row_ops.h"
#include "tc_ptx.h"

namespace dmuon {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kMaxTop = kMaxAlternatives;
constexpr float kLowest = -1e30f;  // in place of smaller exponents y: 2^y is 0 and so is y 2^y

// 2^x, within 2 units of the last place; below 2^-126 it is 0.
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

// Order of the alternatives: by logit, then the lower column. Zeros of both signs are equal.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t column) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return static_cast<uint64_t>(b & 0x80000000u ? ~b : b | 0x80000000u) << 32 | (0xffffffffu - column);
}
__device__ __forceinline__ float key_logit(uint64_t key) {
  const uint32_t b = static_cast<uint32_t>(key >> 32);
  return __uint_as_float(b & 0x80000000u ? b & 0x7fffffffu : ~b);
}
__device__ __forceinline__ uint32_t key_column(uint64_t key) { return 0xffffffffu - static_cast<uint32_t>(key); }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
        "l"(reinterpret_cast<const unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 c;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(c))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return c;
}

// The larger of two, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// A granule's elements, those below `low` as `low`. (A power of two: bf16 holds it.)
template <typename T>
__device__ __forceinline__ void raise(uint4& raw, float low) {
  uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      w[k] = __float_as_uint(max_nan(__uint_as_float(w[k]), low));
    } else {
      const __nv_bfloat162 v = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&w[k]), __float2bfloat162_rn(low));
      w[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
  }
  raw = make_uint4(w[0], w[1], w[2], w[3]);
}

// m: largest logit; c: what x k is taken from; s = sum of 2^y, u = sum of y 2^y with y = x k - c.
struct Sums {
  float m, c, s, u;
};

__device__ __forceinline__ void rescale(Sums& t, float m, float c) {
  const float by = fmaxf(t.c - c, kLowest), f = pow2(by);  // times s it stays finite
  t.u = f * fmaf(by, t.s, t.u);
  t.s *= f;
  t.m = m, t.c = c;
}

__device__ __forceinline__ Sums join(Sums a, Sums b) {
  const float m = fmaxf(a.m, b.m), c = fmaxf(a.c, b.c);  // c goes with m
  rescale(a, m, c);
  rescale(b, m, c);
  return {m, c, a.s + b.s, a.u + b.u};
}

__device__ __forceinline__ Sums join_warp(Sums t) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    t = join(t, {__shfl_xor_sync(0xffffffffu, t.m, o), __shfl_xor_sync(0xffffffffu, t.c, o),
                 __shfl_xor_sync(0xffffffffu, t.s, o), __shfl_xor_sync(0xffffffffu, t.u, o)});
  return t;
}

template <typename T>
__device__ __forceinline__ float largest(const uint4& raw) {
  if constexpr (sizeof(T) == 4) {
    return fmaxf(fmaxf(__uint_as_float(raw.x), __uint_as_float(raw.y)),
                 fmaxf(__uint_as_float(raw.z), __uint_as_float(raw.w)));
  } else {
    auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 t = __hmax2(__hmax2(two(raw.x), two(raw.y)), __hmax2(two(raw.z), two(raw.w)));
    return fmaxf(__low2float(t), __high2float(t));
  }
}

// Where a row lies: `head` elements before the first 16-byte address, `full` granules, `tail` elements.
template <typename T>
struct RowCut {
  static constexpr int E = 16 / sizeof(T);
  int head, tail;
  int64_t full;
  __device__ __forceinline__ RowCut(const T* x, int64_t n) {
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    head = static_cast<int>(n < ((E - off) & (E - 1)) ? n : (E - off) & (E - 1));
    full = (n - head) / E;
    tail = static_cast<int>(n - head - full * E);
  }
  // Column of the row's e-th element outside of granules.
  __device__ __forceinline__ int64_t edge(int e) const { return e < head ? e : head + full * E + (e - head); }
};

template <int W>
struct StatsShared {
  static constexpr int kList = W == 1 ? 256 : 1024;  // at least kMaxTop and an element of each thread
  Sums sums[W];
  float group_max[64];
  float bound;
  int hot_count, list_count;
  uint16_t hot[W * 32];
  uint64_t list[kList];
  uint64_t best[kMaxTop];  // the CTA's alternatives, best first; 0 where there are none
  uint64_t of_cluster[8 * kMaxTop];
  Sums total;
};

// The `top` best of the list's first `count` keys, which differ from one another, into best. All threads.
template <int W>
__device__ __forceinline__ void best_of(StatsShared<W>& sh, const uint64_t* list, int count, int top) {
  for (int i = threadIdx.x; i < top; i += W * 32) sh.best[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < count; i += W * 32) {
    const uint64_t key = list[i];
    int rank = 0;
    for (int j = 0; j < count; ++j) rank += list[j] > key;
    if (rank < top) sh.best[rank] = key;
  }
  __syncthreads();
}

template <int W>
__device__ __forceinline__ void push(StatsShared<W>& sh, float v, int64_t column) {
  const int at = atomicAdd(&sh.list_count, 1);
  if (at < StatsShared<W>::kList) sh.list[at] = key_of(v, static_cast<uint32_t>(column));
}

// Alternatives of this CTA's elements into sh.best. `mine` is the thread's largest logit; its granules are those of
// thread `thread` of `threads`, from granule `thread` on.
template <typename T, int W>
__device__ void find_top(StatsShared<W>& sh, const T* x, const RowCut<T>& cut, float mine, float low, int top, int rank,
                         int ctas) {
  constexpr int E = 16 / sizeof(T), kCta = W * 32, kGroups = W == 1 ? 32 : 64, kPerGroup = kCta / kGroups;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t threads = static_cast<int64_t>(kCta) * ctas;
  const int edges = cut.head + cut.tail;
  const uint4* granules = reinterpret_cast<const uint4*>(x + cut.head);
  float m = mine;
#pragma unroll
  for (int o = kPerGroup >> 1; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (threadIdx.x % kPerGroup == 0) sh.group_max[threadIdx.x / kPerGroup] = m;
  if (threadIdx.x == 0) sh.hot_count = sh.list_count = 0;
  __syncthreads();
  if (threadIdx.x < kGroups) {
    const float v = sh.group_max[threadIdx.x];
    int larger = 0, before = 0;
    for (int j = 0; j < kGroups; ++j) {
      const float o = sh.group_max[j];
      larger += o > v;
      before += o == v && j < static_cast<int>(threadIdx.x);
    }
    if (larger + before == top - 1) sh.bound = v;
  }
  __syncthreads();
  const float bound = sh.bound;
  if (mine >= bound) sh.hot[atomicAdd(&sh.hot_count, 1)] = static_cast<uint16_t>(threadIdx.x);
  __syncthreads();
  const int hot = sh.hot_count;
  // A warp reads a hot thread's granules again, a lane each.
  for (int q = warp; q < hot; q += W) {
    const int64_t thread = static_cast<int64_t>(rank) * kCta + sh.hot[q];
    if (lane == 0 && thread < edges) {
      const float v = max_nan(row::to_f(x[cut.edge(static_cast<int>(thread))]), low);
      if (v >= bound) push(sh, v, cut.edge(static_cast<int>(thread)));
    }
    for (int64_t i = thread + lane * threads; i < cut.full; i += 32 * threads) {
      float v[E];
      uint4 raw = granules[i];
      raise<T>(raw, low);
      if (!(largest<T>(raw) >= bound)) continue;
      row::unpack16<T>(v, raw);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (v[e] >= bound) push(sh, v[e], cut.head + i * E + e);
    }
  }
  __syncthreads();
  if (sh.list_count <= StatsShared<W>::kList) {
    best_of(sh, sh.list, sh.list_count, top);
    return;
  }
  // Many equal logits: every element of this CTA in the order of its columns, one per thread and step. Keys above
  // the last cut's top-th join the list; a step adds at most one per thread.
  __syncthreads();
  if (threadIdx.x == 0) sh.list_count = 0;
  uint64_t least = 0;
  const int64_t columns = cut.head + cut.full * E + cut.tail;
  __syncthreads();
  for (int64_t c0 = static_cast<int64_t>(rank) * kCta; c0 < columns; c0 += threads) {
    const int64_t c = c0 + threadIdx.x;
    if (c < columns) {
      const float v = max_nan(row::to_f(x[c]), low);
      const uint64_t key = key_of(v, static_cast<uint32_t>(c));
      if (v == v && key > least) push(sh, v, c);
    }
    __syncthreads();
    const int count = sh.list_count;
    if (count > StatsShared<W>::kList - kCta || c0 + threads >= columns) {
      best_of(sh, sh.list, count, top);
      least = sh.best[top - 1];
      if (static_cast<int>(threadIdx.x) < top && sh.best[threadIdx.x]) sh.list[threadIdx.x] = sh.best[threadIdx.x];
      if (threadIdx.x == 0) {
        int kept = 0;
        while (kept < top && sh.best[kept]) ++kept;
        sh.list_count = kept;
      }
      __syncthreads();
    }
  }
}

__device__ __forceinline__ uint32_t load_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// One row per cluster of p.cluster CTAs of W warps.
template <typename T, int W>
__global__ void __launch_bounds__(W * 32) token_stats_kernel(const __grid_constant__ StatsLaunch p) {
  constexpr int E = 16 / sizeof(T), kCta = W * 32, kBatch = 4;
  __shared__ StatsShared<W> sh;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int ctas = p.cluster, rank = ctas > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
  const int64_t i = blockIdx.x / ctas;
  int64_t a = -1;
  bool live = true;
  if (p.targets) {
    a = row::load_id(p.targets, p.id_bytes, i);
    live = a >= 0 && a < p.vocab;
    if (a >= p.vocab && threadIdx.x == 0 && rank == 0) atomicOr(p.status, kDevIndex);
  }
  if (!live) {  // the same for all of the cluster
    if (rank != 0) return;
    for (int t = threadIdx.x; t < p.top; t += kCta) p.top_logp[i * p.top + t] = 0.f, p.top_ids[i * p.top + t] = -1;
    if (threadIdx.x == 0) {
      p.logp[i] = 0.f;  // there are targets
      p.entropy[i] = 0.f;
      p.norm[2 * i] = p.norm[2 * i + 1] = 0.f;
    }
    return;
  }
  const T* x = static_cast<const T*>(p.logits) + i * p.ld;
  const RowCut<T> cut(x, p.vocab);
  const float k = p.log2e_over_t, low = p.low;
  const int64_t threads = static_cast<int64_t>(kCta) * ctas, thread = static_cast<int64_t>(rank) * kCta + threadIdx.x;
  const uint4* granules = reinterpret_cast<const uint4*>(x + cut.head);
  Sums t{low, low * k, 0.f, 0.f};
  auto grow = [&](float m) {
    if (m > t.m) rescale(t, m, m * k);
  };
  if (thread < cut.head + cut.tail) {
    const float v = max_nan(row::to_f(x[cut.edge(static_cast<int>(thread))]), low);
    grow(v);
    const float y = fmaf(v, k, -t.c), e = pow2(y);
    t.s += e;
    t.u = fmaf(y, e, t.u);
  }
  for (int64_t g = thread; g < cut.full; g += kBatch * threads) {
    uint4 raw[kBatch];
    // Behind the row's end the batch repeats its first granule; only its maximum is taken from there.
#pragma unroll
    for (int b = 0; b < kBatch; ++b) raw[b] = granules[g + b * threads < cut.full ? g + b * threads : g];
    float m = low;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      raise<T>(raw[b], low);
      m = fmaxf(m, largest<T>(raw[b]));
    }
    grow(m);
    const float2 k2 = make_float2(k, k), c2 = make_float2(-t.c, -t.c);
    float2 s2 = make_float2(0.f, 0.f), u2 = s2;
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (g + b * threads >= cut.full) break;
      float v[E];
      row::unpack16<T>(v, raw[b]);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 y = fma2(make_float2(v[e], v[e + 1]), k2, c2);
        const float2 q = make_float2(pow2(y.x), pow2(y.y));
        s2 = add2(s2, q);
        u2 = fma2(y, q, u2);
      }
    }
    t.s += s2.x + s2.y;
    t.u += u2.x + u2.y;
  }
  const float mine = t.m;
  t = join_warp(t);
  if ((threadIdx.x & 31) == 0) sh.sums[threadIdx.x >> 5] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    t = sh.sums[0];
    for (int w = 1; w < W; ++w) t = join(t, sh.sums[w]);
    sh.total = t;
  }
  if (p.top > 0) find_top<T, W>(sh, x, cut, mine, low, p.top, rank, ctas);
  else __syncthreads();
  const uint64_t* best = sh.best;
  if (ctas > 1) {
    ptx::cluster_sync_all();
    if (rank == 0) {
      // The CTAs' sums in their order; their alternatives side by side.
      for (int e = threadIdx.x; e < ctas * p.top; e += kCta) {
        const uint32_t from = ptx::map_shared(ptx::smem_u32(&sh.best[e % p.top]), e / p.top);
        sh.of_cluster[e] = static_cast<uint64_t>(load_cluster(from + 4)) << 32 | load_cluster(from);
      }
      if (threadIdx.x == 0) {
        Sums all = sh.total;
        for (int c = 1; c < ctas; ++c) {
          const uint32_t from = ptx::map_shared(ptx::smem_u32(&sh.total), c);
          all = join(all, {__uint_as_float(load_cluster(from)), __uint_as_float(load_cluster(from + 4)),
                           __uint_as_float(load_cluster(from + 8)), __uint_as_float(load_cluster(from + 12))});
        }
        sh.total = all;
      }
      __syncthreads();
    }
    ptx::cluster_sync_all();  // the other CTAs' shared memory has been read
    if (rank != 0) return;
    if (p.top > 0) best_of(sh, sh.of_cluster, ctas * p.top, p.top);
  }
  t = sh.total;
  // From c to m itself, and the logarithm of s. A row of nothing but -infinity has no distribution: NaN.
  const bool none = t.m == low;
  const float back = fmaf(t.m, k, -t.c), f = pow2(-back);
  const float sum = t.s * f, along = f * fmaf(-back, t.s, t.u), log_s = none ? NAN : logf(sum);
  auto logp_of = [&](float v) {
    const float d = v - t.m;
    return v <= low ? -INFINITY - log_s : fmaf(d, p.inv_temperature, fmaf(d, p.inv_temperature_low, -log_s));
  };
  if (threadIdx.x == 0) {
    if (p.targets) p.logp[i] = logp_of(row::to_f(x[a]));
    p.entropy[i] = fmaf(-kLn2 / sum, along, log_s);
    p.norm[2 * i] = none ? -INFINITY : t.m;
    p.norm[2 * i + 1] = sum;
  }
  for (int q = threadIdx.x; q < p.top; q += kCta) {
    const uint64_t key = best[q];
    p.top_logp[i * p.top + q] = key ? logp_of(key_logit(key)) : NAN;
    p.top_ids[i * p.top + q] = key ? static_cast<int64_t>(key_column(key)) : -1;
  }
}

// ---------------------------------------------------------------------------- gradient

constexpr int kGradBatch = 4;

// Each CTA takes kThreads * kGradBatch granules of a row (or a part of it element by element, where logits and
// gradient start at different offsets from 16 bytes).
template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads) token_stats_grad_kernel(const __grid_constant__ StatsGradLaunch p) {
  constexpr int E = 16 / sizeof(T);
  constexpr int64_t kPart = static_cast<int64_t>(kThreads) * kGradBatch;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t i = blockIdx.x / p.parts, part = blockIdx.x - i * p.parts;
  const T* x = static_cast<const T*>(p.logits) + i * p.ld;
  T* dx = static_cast<T*>(p.dlogits) + i * p.ldd;
  int64_t a = -1;
  bool live = true;
  if (p.targets) {
    a = row::load_id(p.targets, p.id_bytes, i);
    live = a >= 0 && a < p.vocab;
    if (a >= p.vocab && threadIdx.x == 0 && part == 0) atomicOr(p.status, kDevIndex);
  }
  // With t = log2 p: dx = p (c0 + c1 t), plus the token's own term.
  float m = 0.f, log2_s = 0.f, inv_s = 0.f, c0 = 0.f, c1 = 0.f, own = 0.f;
  if (live) {
    m = p.norm[2 * i];
    const float s = p.norm[2 * i + 1], g = p.dlogp ? p.dlogp[i] : 0.f, h = p.dentropy ? p.dentropy[i] : 0.f;
    log2_s = log2f(s);
    inv_s = m == -INFINITY ? NAN : 1.f / s;
    own = g * p.inv_temperature;
    c0 = -(h != 0.f ? fmaf(h, p.entropy[i], g) : g) * p.inv_temperature;
    c1 = -h * kLn2 * p.inv_temperature;
  }
  const float base = finite_or_zero(m), k = p.log2e_over_t;
  auto value = [&](float v) {
    const float y = (v - base) * k, e = pow2(y) * inv_s;
    return e * fmaf(c1, fmaxf(y, kLowest) - log2_s, c0);
  };
  if ((reinterpret_cast<uintptr_t>(x) - reinterpret_cast<uintptr_t>(dx)) % 16 != 0) {
    const int64_t end = min(p.vocab, (part + 1) * kPart * E);
    for (int64_t c = part * kPart * E + threadIdx.x; c < end; c += kThreads) {
      float v = 0.f;
      if (live) v = value(row::to_f(x[c])) + (c == a ? own : 0.f);
      dx[c] = row::from_f<T>(v);
    }
    return;
  }
  const RowCut<T> cut(x, p.vocab);
  if (part == 0 && static_cast<int>(threadIdx.x) < cut.head + cut.tail) {
    const int64_t c = cut.edge(threadIdx.x);
    float v = 0.f;
    if (live) v = value(row::to_f(x[c])) + (c == a ? own : 0.f);
    dx[c] = row::from_f<T>(v);
  }
  const uint4* in = reinterpret_cast<const uint4*>(x + cut.head);
  uint4* out = reinterpret_cast<uint4*>(dx + cut.head);
  const int64_t g0 = part * kPart + threadIdx.x, ga = a >= cut.head ? (a - cut.head) / E : -1;
  uint4 raw[kGradBatch];
#pragma unroll
  for (int b = 0; b < kGradBatch; ++b) {
    const int64_t g = g0 + b * kThreads;
    if (live && g < cut.full) raw[b] = __ldcs(in + g);
  }
#pragma unroll
  for (int b = 0; b < kGradBatch; ++b) {
    const int64_t g = g0 + b * kThreads;
    if (g >= cut.full) break;
    float v[E];
    if (live) {
      row::unpack16<T>(v, raw[b]);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = value(v[e]);
      if (g == ga) {
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (cut.head + g * E + e == a) v[e] += own;
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.f;
    }
    __stcs(out + g, row::pack16(v));
  }
}

template <typename T, int W>
cudaError_t launch_stats(StatsLaunch& p, cudaStream_t stream) {
  return row::launch(token_stats_kernel<T, W>, dim3(static_cast<unsigned>(p.n * p.cluster)), W * 32, 0, stream, p, p.cluster);
}

template <typename T>
cudaError_t launch_type(StatsLaunch& p, int sms, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  const int64_t granules = (p.vocab + E - 1) / E;
  p.cluster = 1;
  // An SM holds 4 CTAs of 8 warps, 8 of 4, 32 of one. The widest that has all rows at once; of more rows, by a row's
  // length: a CTA's joins and barriers weigh more the shorter it is. bf16, us of 1, 4 and 8 warps: 608 rows of 3000 7.6,
  // 7.2, 6.0, of 16000 21, 12.7, 8.8; 1216 of 1000 6.7, 7.7, 9.8, of 8000 14.1, 11.1, 12.7; 4864 of 1000 11, 22, 34, of
  // 8000 22, 31, 42, of 16000 43, 43, 55, of 32000 86, 66, 78, of 64000 204, 120, 122, of 128256 415, 240, 223. (Two warps
  // were never best by more than a few percent.)
  if (p.n > 4 * sms) {
    if (granules <= 256 || (granules <= 1024 && p.n > 8 * sms)) return launch_stats<T, 1>(p, stream);
    if (granules <= 4096) return launch_stats<T, 4>(p, stream);
  }
  // Few long rows: several CTAs each, one to an SM, or two CTAs each where that makes two to an SM. bf16, us of clusters of
  // 1, 2, 4 and 8: 8 rows of 32000 5.7, 6.4, 6.2, 6.4, of 64000 7.9, 7.6, 6.8, 6.5, of 128256 12.6, 9.8, 7.9, 7.1; 38 rows
  // of 128256 12.6, 11.4, 9.6, 10.1; 152 of 128256 19.7, 15.3, 20.5, 25.
  if (granules >= 6144)
    while (p.cluster < 8 && p.n * p.cluster * 2 <= (p.cluster == 1 ? 2 : 1) * sms) p.cluster *= 2;
  return launch_stats<T, 8>(p, stream);
}

template <typename T, int kThreads>
cudaError_t launch_grad(StatsGradLaunch& p, cudaStream_t stream) {
  constexpr int64_t per = static_cast<int64_t>(kThreads) * kGradBatch * (16 / sizeof(T));
  p.parts = (p.vocab + per - 1) / per;
  // One dimension of the grid holds 2^31 - 1 CTAs: more rows than that allows go in several launches.
  const int64_t rows = std::max<int64_t>(1, ((int64_t(1) << 31) - 1) / p.parts);
  StatsGradLaunch q = p;
  for (int64_t r = 0; r < p.n; r += rows) {
    q.logits = static_cast<const T*>(p.logits) + r * p.ld;
    q.dlogits = static_cast<T*>(p.dlogits) + r * p.ldd;
    q.targets = p.targets ? static_cast<const char*>(p.targets) + r * p.id_bytes : nullptr;
    q.norm = p.norm + 2 * r;
    q.entropy = p.entropy ? p.entropy + r : nullptr;
    q.dlogp = p.dlogp ? p.dlogp + r : nullptr;
    q.dentropy = p.dentropy ? p.dentropy + r : nullptr;
    const int64_t ctas = std::min(rows, p.n - r) * p.parts;
    const cudaError_t e =
        row::launch(token_stats_grad_kernel<T, kThreads>, dim3(static_cast<unsigned>(ctas)), kThreads, 0, stream, q);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <typename T>
cudaError_t launch_grad_type(StatsGradLaunch& p, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  const int64_t granules = (p.vocab + E - 1) / E;
  // A CTA of a short row has little to do, so that more of them are needed for the same bytes under way. bf16, us of 32,
  // 64, 128 and 256 threads: 9728 rows of 1000 10.3, 11.7, 14.8, 24.7, of 3000 29.8, 22.4, 21.4, 31.3, of 32000 313, 179,
  // 180, 183; fp32, 152 rows of 50257 15.7, 10.0, 9.2, 9.6.
  if (granules <= 256) return launch_grad<T, 64>(p, stream);
  return launch_grad<T, 128>(p, stream);
}

}  // namespace

cudaError_t launch_token_stats(StatsLaunch& p, int sms, cudaStream_t stream) {
  return p.dtype == 0 ? launch_type<float>(p, sms, stream) : launch_type<__nv_bfloat16>(p, sms, stream);
}

cudaError_t launch_token_stats_grad(StatsGradLaunch& p, cudaStream_t stream) {
  return p.dtype == 0 ? launch_grad_type<float>(p, stream) : launch_grad_type<__nv_bfloat16>(p, stream);
}

}  // namespace dmuon
