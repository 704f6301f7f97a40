// Clipped policy loss with a KL term, from logits, with its gradient; and token log-probabilities.
//
// Per row t with logits x, token a, temperature T: z = x / T, lp = z_a - log sum exp z, ratio
// r = exp(lp - old), d = ref - lp,
//   l = -min(r A, clip(r, 1 - lo, 1 + hi) A) + k (exp(d) - d - 1),   loss = sum of w l over the rows,
//   c = d(loss)/d(lp) = w (-A r [r A <= clip(r) A] + k (1 - exp(d))),
//   d(loss)/dx = c / T (onehot(a) - softmax(z)).
// A row of weight 0 or with a negative token is not read: its terms and gradient are 0.
//
// c needs the whole row's sum before the first element of the gradient, and a row of a large vocabulary is more
// than an SM holds (128256 bf16: 257 KB), so the row is split over the CTAs of a cluster. It waits in their shared
// memory while they join their sums, and is read and written once: 4 bytes a bf16 element, 8 an fp32 one. A row of
// up to 18 KB is one warp's; beyond the cluster's memory a row is read twice.
//
// Bounds: fp32 by memory (8388 x 32001: 333 us, 6.0 TB/s), bf16 by the instructions of two exponentials and four
// conversions per two bytes beside it (8192 x 128256: 731 us, 5.3 TB/s; 2092 x 128256 without a gradient 139 us,
// 3.9 TB/s). Short rows by the row itself: about 500 instructions of each warp that has a share in it
// (500000 x 500 bf16: 500 us, 2.0 TB/s). A few rows by latency: 8 x 128256 bf16 10 us on the device, 16 to 18 with
// the host's steps.
//
// Memory is read and written in 16-byte granules at aligned addresses, wherever a row starts; the sum runs over
// groups of as many elements counted from the row's first one. So its order goes by the vocabulary alone: a row
// gives the same bits whatever the other rows are, and wherever it and its gradient lie.
#include <algorithm>
#include <type_traits>

#include "row_ops.h"
#include "tc_ptx.h"

namespace dmuon {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The exponentials are the hardware's, of base 2. Beside the rounding of their own, exp(y) = 2^(y log2 e) is off by
// about |y| 2^-24 of itself from the product's: the more, the less a logit's probability counts, or the further two
// policies are apart. With expf and expm1f for a row's ratio and KL term and logf for its sum, 134150 x 2001 bf16 took
// 282 us in place of 267 and 8192 x 128256 764 in place of 750, for gradients as near as these.

// 2^x, within 2 units of the last place; below 2^-126 it is 0.
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log(x) of a sum of terms up to 1. The hardware's log2 is off by up to 2^-22 of itself, and by 2^-23 to one side in
// the mean, which a loss would add up over its rows; one Newton step, y + (x exp(-y) - 1), leaves what 2^-y is off,
// 2^-24 in the mean. log(1) is 0. (Log-probabilities of 1025 x 50257 bf16: off by 5e-8 in the mean and 2.6e-7 in the root
// mean square, 1.0e-7 and 2.9e-7 without the step, at a temperature of 1.3 6e-8 and 1.9e-7, before that one's inverse
// came in two parts; logf: 754 us for 8192 x 128256 in place of 727.)
__device__ __forceinline__ float log_of(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return fmaf(y, kLn2, fmaf(x, pow2(-y), -1.f));
}

// The largest logit m and s = sum of 2^((x - m) k), k = log2(e) / T. The difference is formed before the
// product: it is exact for the largest logit, and small where the terms are large. Against a maximum of
// -infinity (masked logits so far) terms are taken from 0, so that -infinity adds 0 and not NaN.
struct alignas(8) MaxSum {
  float m, s;
};

__device__ __forceinline__ float finite_or_zero(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float k) {
  const float m = fmaxf(a.m, b.m), base = finite_or_zero(m);
  return {m, a.s * pow2((a.m - base) * k) + b.s * pow2((b.m - base) * k)};
}

// Over a warp: the maximum as one integer reduction (of bits that order as the floats do), then the sums.
__device__ __forceinline__ float warp_max(float m) {
  const uint32_t bits = __float_as_uint(m);
  const uint32_t top = __reduce_max_sync(0xffffffffu, bits & 0x80000000u ? ~bits : bits | 0x80000000u);
  return __uint_as_float(top & 0x80000000u ? top & 0x7fffffffu : ~top);
}

__device__ __forceinline__ float warp_sum(float s) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

__device__ __forceinline__ MaxSum join_warp(MaxSum t, float k) {
  const float m = warp_max(t.m);
  return {m, warp_sum(t.s * pow2((t.m - finite_or_zero(m)) * k))};
}

// Of n sums in shared memory, by a warp.
__device__ __forceinline__ MaxSum join_list(const MaxSum* list, int n, float k) {
  const int lane = threadIdx.x & 31;
  float m = -INFINITY, s = 0.f;
  for (int w = lane; w < n; w += 32) m = fmaxf(m, list[w].m);
  m = warp_max(m);
  const float base = finite_or_zero(m);
  for (int w = lane; w < n; w += 32) s = fmaf(list[w].s, pow2((list[w].m - base) * k), s);
  return {m, warp_sum(s)};
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 c;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(c))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return c;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 c;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(c))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return c;
}

// The largest element of granules; of bf16, two at a time. (NaN is left to the sum.)
template <typename T>
struct Largest;

template <>
struct Largest<float> {
  float m = -INFINITY;
  __device__ __forceinline__ void add(const uint4& raw) {
    m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(raw.x), __uint_as_float(raw.y)),
                       fmaxf(__uint_as_float(raw.z), __uint_as_float(raw.w))));
  }
  __device__ __forceinline__ float get() const { return m; }
};

template <>
struct Largest<__nv_bfloat16> {
  uint32_t m = 0xff80ff80u;
  static __device__ __forceinline__ __nv_bfloat162 two(uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); }
  __device__ __forceinline__ void add(const uint4& raw) {
    const __nv_bfloat162 t = __hmax2(__hmax2(two(raw.x), two(raw.y)), __hmax2(two(raw.z), two(raw.w)));
    const __nv_bfloat162 n = __hmax2(two(m), t);
    m = *reinterpret_cast<const uint32_t*>(&n);
  }
  __device__ __forceinline__ float get() const {
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};

// A granule of -infinity.
template <typename T>
__device__ __forceinline__ uint4 lowest() {
  const uint32_t w = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
  return make_uint4(w, w, w, w);
}

// The sum of 2^((x - base) k) over granules.
struct Terms {
  float2 less, kk, acc;

  __device__ __forceinline__ Terms(float base, float k)
      : less(make_float2(-base, -base)), kk(make_float2(k, k)), acc(make_float2(0.f, 0.f)) {}

  template <typename T>
  __device__ __forceinline__ void add(const uint4& raw) {
    constexpr int E = 16 / sizeof(T);
    float v[E];
    row::unpack16<T>(v, raw);
#pragma unroll
    for (int j = 0; j < E; j += 2) add_pair(v[j], v[j + 1]);
  }
  __device__ __forceinline__ void add_pair(float x, float y) {
    const float2 z = mul2(add2(make_float2(x, y), less), kk);
    acc = add2(acc, make_float2(pow2(z.x), pow2(z.y)));
  }
  __device__ __forceinline__ float get() const { return acc.x + acc.y; }
};

// The 16 bytes that start WORDS words, and with HALF two more bytes, into a and b.
template <int WORDS, bool HALF>
__device__ __forceinline__ uint4 shifted(const uint4& a, const uint4& b) {
  const uint32_t w[9] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, 0};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = HALF ? __funnelshift_r(w[i + WORDS], w[i + WORDS + 1], 16) : w[i + WORDS];
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The elements of a granule from `left` on become -infinity.
template <typename T>
__device__ __forceinline__ uint4 cut_behind(const uint4& raw, int left) {
  uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int j = 0; j < 16 / static_cast<int>(sizeof(T)); ++j) {
    if (j < left) continue;
    if constexpr (sizeof(T) == 4)
      w[j] = 0xff800000u;
    else
      w[j / 2] = j % 2 ? (w[j / 2] & 0xffffu) | 0xff800000u : (w[j / 2] & 0xffff0000u) | 0xff80u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a row needs beside its logits; a < 0: the row is not read.
struct RowMeta {
  int a;
  float w, old, ref, adv;
};

__device__ __forceinline__ RowMeta row_meta(const PolicyLaunch& p, int64_t i) {
  RowMeta r{-1, 0.f, 0.f, 0.f, 0.f};
  if (i >= p.n) return r;
  const int64_t a = row::load_id(p.targets, p.id_bytes, i);
  if (p.weights) {
    r.w = __ldg(p.weights + i);
    r.old = __ldg(p.old_logp + i);
    r.adv = __ldg(p.advantages + i);
    if (p.ref_logp) r.ref = __ldg(p.ref_logp + i);
    if (r.w == 0.f) return r;
  }
  if (a >= p.vocab) atomicOr(p.status, kDevIndex);
  r.a = a < 0 || a >= p.vocab ? -1 : static_cast<int>(a);
  return r;
}

// exp(d) - 1: near 0 by its series up to d^7 / 7!, 1e-8 off at 1/4.
__device__ __forceinline__ float exp_less_1(float d) {
  float r = 1.f / 5040.f;
  r = fmaf(r, d, 1.f / 720.f);
  r = fmaf(r, d, 1.f / 120.f);
  r = fmaf(r, d, 1.f / 24.f);
  r = fmaf(r, d, 1.f / 6.f);
  r = fmaf(r, d, 0.5f);
  r = fmaf(r * d, d, d);
  return fabsf(d) < 0.25f ? r : pow2(d * kLog2e) - 1.f;
}

// Writes the row's log-probability (one thread), adds its term to `loss` and gives its gradient's scale c / T.
__device__ __forceinline__ float row_end(const PolicyLaunch& p, int64_t i, const RowMeta& r, float xa, MaxSum t,
                                         bool writes, float& loss) {
  // The token's distance from the maximum is exact in many cases, and the logarithm of a sum of 1 is 0. A distance of
  // -infinity stays one.
  const float from_top = xa - t.m, low = from_top > -INFINITY ? from_top * p.inv_temperature_low : 0.f;
  const float logp = fmaf(from_top, p.inv_temperature, low - log_of(t.s));
  float each = 0.f, c = 0.f;
  if (p.weights) {
    const float ratio = pow2((logp - r.old) * kLog2e);
    const float whole = ratio * r.adv, cut = fminf(fmaxf(ratio, 1.f - p.clip_low), 1.f + p.clip_high) * r.adv;
    // Not "whole <= cut": a NaN stays one.
    each = whole > cut ? -cut : -whole;
    c = whole > cut ? 0.f : -whole;
    if (p.ref_logp) {
      const float d = r.ref - logp, e = exp_less_1(d);
      each = fmaf(p.kl_coef, e - d, each);
      c = fmaf(-p.kl_coef, e, c);
    }
  }
  if (writes && p.logp) p.logp[i] = logp;
  loss = fmaf(each, r.w, loss);
  return c * r.w * p.inv_temperature;
}

// Leaves a term of the loss; who leaves the last one adds them all, in an order that their number fixes. The counter
// lies in front of the stream's or graph's scratch, and its last increment sets it back to 0. Called by one whole warp
// per term. (A launch of its own for the sum: 4 more microseconds for a call of 8 rows.)
__device__ __forceinline__ void leave_term(const PolicyLaunch& p, int64_t at, float loss) {
  const int lane = threadIdx.x & 31;
  unsigned before = 0;
  if (lane == 0) {
    p.loss_terms[at] = loss;
    __threadfence();
    before = atomicInc(p.terms_done, static_cast<unsigned>(p.terms) - 1);
  }
  if (__shfl_sync(0xffffffffu, before, 0) + 1 < static_cast<unsigned>(p.terms)) return;
  __threadfence();
  float acc = 0.f;
  int64_t i = lane;
  for (; i + 7 * 32 < p.terms; i += 8 * 32) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __ldcg(p.loss_terms + i + 32 * k);
#pragma unroll
    for (int k = 0; k < 8; ++k) acc += v[k];
  }
  for (; i < p.terms; i += 32) acc += __ldcg(p.loss_terms + i);
  acc = warp_sum(acc);
  if (lane == 0) *p.loss = acc;
}

__device__ __forceinline__ void row_skipped(const PolicyLaunch& p, int64_t i) {
  if (p.logp) p.logp[i] = 0.f;
}

// The gradient of a granule's logits: scale (onehot - 2^((x - base) k) / s), with per = -scale / s.
template <int E>
__device__ __forceinline__ void gradient(float (&v)[E], float base, float k, float per) {
  const float2 less = make_float2(-base, -base), kk = make_float2(k, k), pp = make_float2(per, per);
#pragma unroll
  for (int j = 0; j < E; j += 2) {
    const float2 z = mul2(add2(make_float2(v[j], v[j + 1]), less), kk);
    const float2 g = mul2(make_float2(pow2(z.x), pow2(z.y)), pp);
    v[j] = g.x, v[j + 1] = g.y;
  }
}

// Where a row lies: `head` elements before the first 16-byte address, `full` whole granules, `tail` elements.
struct Cut {
  int head, full, tail;
};

template <typename T>
__device__ __forceinline__ Cut cut_row(const T* x, int vocab) {
  constexpr int E = 16 / sizeof(T);
  const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  Cut c;
  c.head = min((E - off) & (E - 1), vocab);
  c.full = (vocab - c.head) / E;
  c.tail = vocab - c.head - c.full * E;
  return c;
}

// ---------------------------------------------------------------------------- rows in shared memory

constexpr int kRingSlots = 3;     // of a warp: one being loaded, one worked on, one being written
constexpr int kBatch = 4;         // granules of a lane at a time
constexpr int kSlotBytes = 4608;  // of a warp that shares a row: two CTAs' slots fill an SM's shared memory
constexpr int kWarpGroups = kSlotBytes / 16 - 2;  // beside the rest of the first granule, and the one read past the last
constexpr int kMaxCluster = 16;
// Rows whose sums are on their way or being read, of those that are read at all. A warp sends its sum of the
// n-th when it has joined the (n - 2)-th: then every warp has sent that one, and before it has read the
// (n - 4)-th, whose place the n-th takes.
constexpr int kJoins = 4;

// Who takes a row: one warp, as long as four warps' slots fit an SM (33554 x 8000 bf16: 243 us, shared by a cluster
// 417; 32772 x 8191: 278 and 757); a cluster of a portable size, of CTAs of 128 threads, four per SM (33554 x 8000
// fp32: 316 us, with 256 threads 437; 13421 x 20000 bf16 225 and 281), or of 256, two per SM (8192 x 128256 bf16: 912
// us when one CTA of 512 took 1135, and four of 128 952); or, for rows beyond eight of those, a cluster of CTAs
// twice as large (1024 x 262144 bf16: 221 us, 4.9 TB/s).
enum RingMode { kSolo, kSmall, kShared, kWide };

template <int MODE>
struct Ring {
  static constexpr int kThreads = MODE == kSolo || MODE == kSmall ? 128 : MODE == kShared ? 256 : 512;
  static constexpr int kPerSm = 512 / kThreads;
  static constexpr int kWarps = kThreads / 32;
  static constexpr int kSmem = kWarps * kRingSlots * kSlotBytes + 128;
  static constexpr int kCluster = MODE == kSolo ? 1 : MODE == kWide ? kMaxCluster : 8;  // CTAs per row at most
};
constexpr int kSoloSlotBytes = 18432;  // the most for which four warps' slots fit an SM

// Writes v into a CTA of the cluster and counts its bytes at that CTA's barrier (shared::cluster addresses).
__device__ __forceinline__ void send(uint32_t addr, MaxSum v, uint32_t barrier) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr), "f"(v.m),
               "f"(v.s), "r"(barrier)
               : "memory");
}

__device__ __forceinline__ void send(uint32_t addr, float v, uint32_t barrier) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];" ::"r"(addr), "f"(v), "r"(barrier)
               : "memory");
}

// What a row needs beside its logits, one word per lane, so that one load per warp brings all of it and nothing
// waits for it until its row is near: lanes 0 and 1 the token's low and high word, then weight, old
// log-probability, advantage and reference.
struct LaneMeta {
  const char* at = nullptr;
  int64_t stride = 4;

  __device__ __forceinline__ LaneMeta(const PolicyLaunch& p, int lane) {
    if (lane < 2 && 4 * lane < p.id_bytes) {
      at = static_cast<const char*>(p.targets) + 4 * lane;
      stride = p.id_bytes;
    } else if (lane >= 2 && lane < 6) {
      const float* from = lane == 2 ? p.weights : lane == 3 ? p.old_logp : lane == 4 ? p.advantages : p.ref_logp;
      at = reinterpret_cast<const char*>(from);
    }
  }
  __device__ __forceinline__ uint32_t load(int64_t i, int64_t n) const {
    return at && i < n ? __ldg(reinterpret_cast<const uint32_t*>(at + i * stride)) : 0u;
  }
};

// The row's token, or -1: the row is not read.
__device__ __forceinline__ int token_of(const PolicyLaunch& p, uint32_t word, int64_t i) {
  const uint32_t lo = __shfl_sync(0xffffffffu, word, 0);
  const int hi = p.id_bytes == 8 ? static_cast<int>(__shfl_sync(0xffffffffu, word, 1)) : static_cast<int>(lo) >> 31;
  const float w = __uint_as_float(__shfl_sync(0xffffffffu, word, 2));
  if (i >= p.n || hi < 0 || (p.weights && w == 0.f)) return -1;
  if (hi > 0 || lo >= static_cast<uint32_t>(p.vocab)) {
    if ((threadIdx.x & 31) == 0) atomicOr(p.status, kDevIndex);
    return -1;
  }
  return static_cast<int>(lo);
}

// A cluster takes every gridDim.x / C-th row, and each of its warps an equal share of it (kSolo: every warp rows
// of its own). The warps work by themselves: bulk copies bring a share's whole granules into the warp's slots and
// take their gradients, formed in place, out; up to E - 1 elements on either side of them go through registers.
// Where they meet is the row's sum: every warp sends its own to every CTA of the cluster (and who has the target, its
// logit), forms its sum of the next row, and goes on when all have arrived. (With barriers over the cluster and the CTA in their place, 38% of the
// warps' time went into those and the fences they imply.)
// EDGES: shares that are not whole granules.
template <typename T, int MODE, bool EDGES>
__global__ void __launch_bounds__(Ring<MODE>::kThreads, Ring<MODE>::kPerSm) policy_ring_kernel(const PolicyLaunch p) {
  using R = Ring<MODE>;
  constexpr int E = 16 / sizeof(T);
  constexpr bool SOLO = MODE == kSolo;
  extern __shared__ uint8_t dyn[];
  __shared__ MaxSum joined[kJoins][R::kCluster * R::kWarps];
  __shared__ float joined_token[kJoins];
  __shared__ uint64_t joined_full[kJoins];
  __shared__ uint64_t slot_full[R::kWarps][kRingSlots];
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* slots = dyn + (128 - (ptx::smem_u32(dyn) & 127)) % 128 + warp * kRingSlots * p.slot_bytes;
  uint64_t* full = slot_full[warp];
  const int C = p.cluster, unit = SOLO ? 0 : static_cast<int>(ptx::cluster_ctarank()) * R::kWarps + warp;
  const int64_t step = SOLO ? gridDim.x * R::kWarps : gridDim.x / C;
  const int64_t first = SOLO ? blockIdx.x * R::kWarps + warp : blockIdx.x / C;
  const int vocab = static_cast<int>(p.vocab);
  const int units = SOLO ? 1 : C * R::kWarps, groups_each = (vocab + units * E - 1) / (units * E);
  const int from = min(unit * groups_each * E, vocab), length = min(groups_each * E, vocab - from);
  const T* logits = static_cast<const T*>(p.logits) + from;
  const float k = p.log2e_over_t;
  if (threadIdx.x == 0) {
    for (int w = 0; w < R::kWarps; ++w)
      for (int s = 0; s < kRingSlots; ++s) ptx::mbar_init(&slot_full[w][s], 1);
    for (int s = 0; s < kJoins; ++s) ptx::mbar_init(&joined_full[s], 1);
    abort_word = 0;
    ptx::fence_barrier_init();
  }
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  __syncthreads();
  if (!SOLO) ptx::cluster_sync_all();  // every CTA has set up its barriers before another writes into it

  uint64_t policy = 0;
  if (lane == 0) policy = ptx::l2_policy_evict_first();
  auto cut = [&](int64_t i) { return EDGES ? cut_row(logits + i * p.ld, length) : Cut{0, length / E, 0}; };
  auto load = [&](int64_t i, int a, int s) {  // lane 0: this warp's share of row i into slot s
    if (a < 0) return;
    const Cut c = cut(i);
    ptx::mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(c.full) * 16u);
    if (c.full > 0)
      ptx::bulk_load_hint(ptx::smem_u32(slots + s * p.slot_bytes + (c.head ? 16 : 0)), logits + i * p.ld + c.head,
                          static_cast<uint32_t>(c.full) * 16u, &full[s], policy);
  };
  // The element outside the granules that this lane holds, or -1.
  auto edge_of = [&](const Cut& c) {
    if (!EDGES) return -1;
    if (lane < c.head) return lane;
    if (lane >= 16 && lane - 16 < c.tail) return c.head + c.full * E + lane - 16;
    return -1;
  };
  // The edge's logit, as it lies in memory.
  auto fetch = [&](T& xe, int64_t i, int a) {
    if (a < 0) return;
    const int e = EDGES ? edge_of(cut(i)) : -1;
    if (e >= 0) xe = logits[i * p.ld + e];
  };
  uint32_t parity = 0;  // bit s: of the next phase of slot s to wait for
  uint32_t sent = 0, read = 0;  // rows whose sums this warp has sent, has joined
  MaxSum ready{};  // kSolo: the sum of the row last summed, and its token's logit
  float ready_token = 0.f;
  // This warp's sum of row i, in slot s, to every CTA of the cluster; and the logit of the row's token a by the warp
  // whose share holds it. (Not read from memory by each: the gradient may go over the logits, and the others may write
  // theirs once they have this warp's sum. From its own slot a warp reads it before it sends anything.)
  auto sum_row = [&](int64_t i, int s, int a, T xe) {
    const Cut c = cut(i);
    uint4* line = reinterpret_cast<uint4*>(slots + s * p.slot_bytes);
    const uint4* data = line + (c.head ? 1 : 0);
    const int edge = edge_of(c), bytes = c.head ? 16 - c.head * static_cast<int>(sizeof(T)) : 0;
    // A wait that runs out is recorded; the launch goes on to its end on whatever has come, so that no warp of
    // the cluster is left waiting.
    ptx::wait_fast(&full[s], (parity >> s) & 1u, abort_flag, p.status);
    parity ^= 1u << s;
    if (EDGES && (c.head || c.tail)) {
      if (edge >= 0) reinterpret_cast<T*>(line)[bytes / static_cast<int>(sizeof(T)) + edge] = xe;
      __syncwarp();
    }
    // Granules in batches of kBatch per lane, loaded together: a lane has under ten of them, and one at a time
    // each would wait for its load and its chain of operations.
    const uint4 none = lowest<T>();
    Largest<T> top;
    for (int q0 = lane; q0 < c.full; q0 += 32 * kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) raw[b] = q0 + 32 * b < c.full ? data[q0 + 32 * b] : none;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) top.add(raw[b]);
    }
    MaxSum sum;
    sum.m = warp_max(EDGES && edge >= 0 ? fmaxf(top.get(), row::to_f(xe)) : top.get());
    Terms terms(finite_or_zero(sum.m), k);
    if constexpr (sizeof(T) == 4) {
      // Single elements, at any offset: the memory traffic of fp32 leaves time for their loads.
      const float* x = reinterpret_cast<const float*>(line) + bytes / 4;
      for (int e0 = lane; e0 < length; e0 += 32 * 4 * kBatch) {
        float v[4 * kBatch];
#pragma unroll
        for (int b = 0; b < 4 * kBatch; ++b) v[b] = e0 + 32 * b < length ? x[e0 + 32 * b] : -INFINITY;
#pragma unroll
        for (int b = 0; b < 4 * kBatch; b += 2) terms.add_pair(v[b], v[b + 1]);
      }
    } else {
      // Whole groups first, then the last one where it is not; one copy of the loop for each offset from 16 bytes.
      const int whole = length / E;
      auto pass = [&](auto words, auto half) {
        constexpr int W = decltype(words)::value;
        constexpr bool H = decltype(half)::value;
        for (int q0 = lane; q0 < whole; q0 += 32 * kBatch) {
          uint4 raw[kBatch];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int q = q0 + 32 * b;
            raw[b] = none;
            if (q < whole) raw[b] = W == 0 && !H ? line[q] : shifted<W, H>(line[q], line[q + 1]);
          }
#pragma unroll
          for (int b = 0; b < kBatch; ++b) terms.template add<T>(raw[b]);
        }
        if (EDGES && whole * E < length && lane == 31)
          terms.template add<T>(cut_behind<T>(shifted<W, H>(line[whole], line[whole + 1]), length - whole * E));
      };
      if constexpr (!EDGES) {
        pass(std::integral_constant<int, 0>(), std::false_type());
      } else {
        switch (bytes >> 1) {
          case 0: pass(std::integral_constant<int, 0>(), std::false_type()); break;
          case 1: pass(std::integral_constant<int, 0>(), std::true_type()); break;
          case 2: pass(std::integral_constant<int, 1>(), std::false_type()); break;
          case 3: pass(std::integral_constant<int, 1>(), std::true_type()); break;
          case 4: pass(std::integral_constant<int, 2>(), std::false_type()); break;
          case 5: pass(std::integral_constant<int, 2>(), std::true_type()); break;
          case 6: pass(std::integral_constant<int, 3>(), std::false_type()); break;
          default: pass(std::integral_constant<int, 3>(), std::true_type()); break;
        }
      }
    }
    sum.s = warp_sum(terms.get());
    const bool here = a >= from && a < from + length;
    const T* share = reinterpret_cast<const T*>(line) + bytes / static_cast<int>(sizeof(T));
    const float token = here ? row::to_f(share[a - from]) : 0.f;
    if (SOLO) {
      ready = sum;
      ready_token = token;
      return;
    }
    const int j = sent++ % kJoins;
    if (threadIdx.x == 0)
      ptx::mbar_arrive_expect_tx(&joined_full[j], static_cast<uint32_t>(units * sizeof(MaxSum) + sizeof(float)));
    if (lane < C) {
      const uint32_t barrier = ptx::map_shared(ptx::smem_u32(&joined_full[j]), lane);
      if (here) send(ptx::map_shared(ptx::smem_u32(&joined_token[j]), lane), token, barrier);
      send(ptx::map_shared(ptx::smem_u32(&joined[j][unit]), lane), sum, barrier);
    }
  };

  const LaneMeta meta(p, lane);
  uint32_t word = meta.load(first, p.n), word1 = meta.load(first + step, p.n), word2 = meta.load(first + 2 * step, p.n);
  int a = token_of(p, word, first), a1 = token_of(p, word1, first + step);
  T xe{}, xe1{};
  fetch(xe, first, a);
  fetch(xe1, first + step, a1);
  if (lane == 0) {
    load(first, a, 0);
    load(first + step, a1, 1);
  }
  float loss = 0.f;
  if (a >= 0) sum_row(first, 0, a, xe);
  int s = 0;
  for (int64_t i = first; i < p.n; i += step) {
    const uint32_t word3 = meta.load(i + 3 * step, p.n);
    const int s1 = s == 2 ? 0 : s + 1, s2 = s == 0 ? 2 : s - 1;
    MaxSum sum = ready;
    float token_logit = ready_token;
    if (a1 >= 0) sum_row(i + step, s1, a1, xe1);
    // The slot of the row before takes the row after next, once its gradient has left it.
    const int a2 = token_of(p, word2, i + 2 * step);
    T xe2{};
    fetch(xe2, i + 2 * step, a2);
    if (lane == 0) {
      ptx::bulk_wait_read0();
      ptx::fence_async_smem();
      load(i + 2 * step, a2, s2);
    }
    const Cut c = cut(i);
    // The share lies in the slot as it does around 16-byte addresses; `data` are its whole granules.
    uint4* data = reinterpret_cast<uint4*>(slots + s * p.slot_bytes) + (c.head ? 1 : 0);
    const int edge = edge_of(c);
    T* dx = p.dlogits ? static_cast<T*>(p.dlogits) + i * p.ldd + from : nullptr;
    if (a >= 0) {
      if (!SOLO) {
        const int j = read % kJoins;
        ptx::wait_fast(&joined_full[j], (read++ / kJoins) & 1u, abort_flag, p.status);
        sum = join_list(joined[j], units, k);
        token_logit = __shfl_sync(0xffffffffu, joined_token[j], 0);  // so that it has been read before the next send
      }
      RowMeta now;
      now.w = __uint_as_float(__shfl_sync(0xffffffffu, word, 2));
      now.old = __uint_as_float(__shfl_sync(0xffffffffu, word, 3));
      now.adv = __uint_as_float(__shfl_sync(0xffffffffu, word, 4));
      now.ref = __uint_as_float(__shfl_sync(0xffffffffu, word, 5));
      const float scale = row_end(p, i, now, token_logit, sum, unit == 0 && lane == 0, loss);
      if (dx) {
        const float base = finite_or_zero(sum.m), per = -scale * __frcp_rn(sum.s);
        const int inside = a - from - c.head;  // the token's place in this share, if it has one
        const int token_q = inside >= 0 ? inside / E : -1, token_j = inside & (E - 1);
        for (int q0 = lane; q0 < c.full; q0 += 32 * kBatch) {
          uint4 raw[kBatch];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) raw[b] = q0 + 32 * b < c.full ? data[q0 + 32 * b] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int q = q0 + 32 * b;
            float v[E];
            row::unpack16<T>(v, raw[b]);
            gradient(v, base, k, per);
            if (q == token_q)
#pragma unroll
              for (int e = 0; e < E; ++e)
                if (e == token_j) v[e] += scale;
            if (q < c.full) data[q] = row::pack16(v);
          }
        }
        if (edge >= 0) {
          const float g = per * pow2((row::to_f(xe) - base) * k);
          dx[edge] = row::from_f<T>(from + edge == a ? g + scale : g);
        }
      }
    } else {
      if (unit == 0 && lane == 0) row_skipped(p, i);
      if (dx) {
        for (int q = lane; q < c.full; q += 32) data[q] = make_uint4(0, 0, 0, 0);
        if (edge >= 0) dx[edge] = row::from_f<T>(0.f);
      }
    }
    if (dx && p.same_cut) ptx::fence_async_smem();
    __syncwarp();  // every lane is done with the slot
    if (dx && p.same_cut) {
      if (lane == 0) {
        if (c.full > 0) ptx::bulk_store(dx + c.head, ptx::smem_u32(data), static_cast<uint32_t>(c.full) * 16u);
        ptx::bulk_commit();
      }
    } else if (dx) {
      const T* from_smem = reinterpret_cast<const T*>(data);
      for (int e = lane; e < c.full * E; e += 32) dx[c.head + e] = from_smem[e];
      __syncwarp();
    }
    s = s1;
    word = word1, word1 = word2, word2 = word3, a = a1, a1 = a2;
    xe = xe1, xe1 = xe2;
  }
  // One term per cluster (or CTA, its warps in their order): its rows' in their order.
  if (SOLO && p.loss_terms) {
    __shared__ float of_warp[R::kWarps];
    if (lane == 0) of_warp[warp] = loss;
    __syncthreads();
    loss = 0.f;
    for (int w = 0; w < R::kWarps; ++w) loss += of_warp[w];
  }
  if (p.loss_terms && unit == 0 && (!SOLO || warp == 0)) leave_term(p, SOLO ? blockIdx.x : first, loss);
  // Rows behind the last are never loaded, so no load is on its way here, unless a wait ran out.
  if (lane == 0) {
    if (*abort_flag)
      for (int q = 0; q < kRingSlots; ++q)
        ptx::wait_bounded(&full[q], (parity >> q) & 1u, abort_flag, p.status, ptx::kDrainLimitNs, false);
    ptx::bulk_wait0();
  }
  __syncwarp();
  if (!SOLO) ptx::cluster_sync_all();  // nobody writes into a CTA that has ended
}

// ---------------------------------------------------------------------------- rows read twice

constexpr int kTwiceThreads = 512;

// One CTA per row: rows beyond a cluster's shared memory (292000 fp32, 585000 bf16 elements). Each thread keeps its
// own maximum and sum, element by element (256 x 600000 fp32: 804 us, 1.4 TB/s, against 4.8 for rows that fit).
template <typename T>
__global__ void __launch_bounds__(kTwiceThreads) policy_twice_kernel(const PolicyLaunch p) {
  __shared__ MaxSum part[kTwiceThreads / 32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t i = blockIdx.x;
  const RowMeta r = row_meta(p, i);
  const T* x = static_cast<const T*>(p.logits) + i * p.ld;
  T* dx = p.dlogits ? static_cast<T*>(p.dlogits) + i * p.ldd : nullptr;
  if (r.a < 0) {
    if (threadIdx.x == 0) row_skipped(p, i);
    if (p.loss_terms && threadIdx.x < 32) leave_term(p, i, 0.f);
    if (dx)
      for (int64_t c = threadIdx.x; c < p.vocab; c += kTwiceThreads) dx[c] = row::from_f<T>(0.f);
    return;
  }
  const float k = p.log2e_over_t;
  MaxSum t{-INFINITY, 0.f};
  float base = 0.f;
  for (int64_t c = threadIdx.x; c < p.vocab; c += kTwiceThreads) {
    const float v = row::to_f(x[c]);
    if (v > t.m) {
      t.s *= pow2((t.m - v) * k);
      t.m = base = v;
    }
    t.s += pow2((v - base) * k);
  }
  t = join_warp(t, k);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = t;
  const float xa = row::to_f(x[r.a]);  // read before any thread writes a gradient over it
  __syncthreads();
  t = part[0];
  for (int w = 1; w < kTwiceThreads / 32; ++w) t = join(t, part[w], k);
  float loss = 0.f;
  const float scale = row_end(p, i, r, xa, t, threadIdx.x == 0, loss);
  if (p.loss_terms && threadIdx.x < 32) leave_term(p, i, loss);
  if (!dx) return;
  base = finite_or_zero(t.m);
  const float per = -scale * __frcp_rn(t.s);
  for (int64_t c = threadIdx.x; c < p.vocab; c += kTwiceThreads) {
    const float e = per * pow2((row::to_f(x[c]) - base) * k);
    dx[c] = row::from_f<T>(c == r.a ? e + scale : e);
  }
}

// ---------------------------------------------------------------------------- launches

// How many clusters of `size` CTAs of the ring kernel fit on the GPU at once. A property of the device: asked for
// once (the caller holds the library's lock), after the kernel's attributes have been set.
template <typename T, int MODE, bool EDGES>
cudaError_t resident_clusters(int dev, int size, int* clusters) {
  constexpr int kMaxDevices = 64;
  static int known[kMaxDevices][kMaxCluster + 1];  // 1 + the number
  int n = dev < kMaxDevices ? known[dev][size] - 1 : -1;
  if (n < 0) {
    auto* kernel = policy_ring_kernel<T, MODE, EDGES>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<MODE>::kSmem);
    if (e == cudaSuccess && MODE == kWide)
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(Ring<MODE>::kThreads);
    cfg.dynamicSmemBytes = Ring<MODE>::kSmem;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(size);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) known[dev][size] = n + 1;
  }
  *clusters = n;
  return cudaSuccess;
}

// A warp's time for a row beside its granules, in granules (about 500 instructions to 65 for 32 of them).
constexpr int kRowCost = 256;

// How rows are shared among clusters: the way that brings the most of them through.
struct RingChoice {
  int mode = 0, cluster = 0, clusters = 0;
  double rate = 0.0;  // clusters at once over time per row
};

// The cluster sizes of one mode that hold a row and fit the GPU. (Larger ones leave fewer SMs over at times, but each
// of their warps pays for the row again.)
template <typename T, int MODE, bool EDGES>
cudaError_t consider(RingChoice& best, int dev, int64_t vocab) {
  using R = Ring<MODE>;
  constexpr int E = 16 / sizeof(T);
  constexpr int64_t per_cta = R::kWarps * kWarpGroups;
  // Two CTAs at least: the sums travel by asynchronous stores, which only a cluster launch has.
  const int64_t groups = (vocab + E - 1) / E, least = std::max<int64_t>(2, (groups + per_cta - 1) / per_cta);
  for (int64_t size = least; size <= R::kCluster; ++size) {
    int n = 0;
    const cudaError_t e = resident_clusters<T, MODE, EDGES>(dev, static_cast<int>(size), &n);
    if (e != cudaSuccess) return e;
    const double rate = n / (kRowCost + static_cast<double>(groups) / (size * R::kWarps));
    // Small CTAs where they gain something: more of them meet for a row (8388 x 32001 fp32: 333 us by four CTAs of 256
    // threads, 354 by seven of 128, at almost equal rates).
    if (rate > best.rate * (MODE == kSmall ? 1.05 : 1.0)) best = {MODE, static_cast<int>(size), n, rate};
  }
  return cudaSuccess;
}

template <typename T, int MODE, bool EDGES>
cudaError_t launch_ring(PolicyLaunch& p, const RingChoice& c, cudaStream_t stream) {
  using R = Ring<MODE>;
  p.slot_bytes = kSlotBytes;
  p.cluster = c.cluster;
  p.terms = std::min<int64_t>(p.n, c.clusters);
  const unsigned ctas = static_cast<unsigned>(p.terms * p.cluster);
  return row::launch(policy_ring_kernel<T, MODE, EDGES>, dim3(ctas), R::kThreads, R::kSmem, stream, p, p.cluster);
}

// Whether a row fits the shared memory of a cluster; if so, launches.
template <typename T, bool EDGES>
cudaError_t launch_shared(PolicyLaunch& p, cudaStream_t stream, bool* launched) {
  int dev = 0;
  RingChoice best;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = consider<T, kShared, EDGES>(best, dev, p.vocab);
  if (e == cudaSuccess) e = consider<T, kSmall, EDGES>(best, dev, p.vocab);
  if (e == cudaSuccess && best.cluster == 0) e = consider<T, kWide, EDGES>(best, dev, p.vocab);
  *launched = e == cudaSuccess && best.cluster > 0;
  if (!*launched) return e;
  return best.mode == kSmall ? launch_ring<T, kSmall, EDGES>(p, best, stream)
       : best.mode == kShared ? launch_ring<T, kShared, EDGES>(p, best, stream)
                              : launch_ring<T, kWide, EDGES>(p, best, stream);
}

template <typename T, bool EDGES>
cudaError_t launch_solo(PolicyLaunch& p, int sms, cudaStream_t stream) {
  using R = Ring<kSolo>;
  auto* kernel = policy_ring_kernel<T, kSolo, EDGES>;
  const size_t smem = static_cast<size_t>(R::kWarps) * kRingSlots * p.slot_bytes + 128;
  cudaError_t e = cudaSuccess;
  if (smem > 40 * 1024)  // beside the static shared memory, what needs no opt-in
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  int64_t ctas = (p.n + R::kWarps - 1) / R::kWarps;
  if (e == cudaSuccess && ctas > sms) {
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, R::kThreads, smem);
    ctas = std::min<int64_t>(ctas, static_cast<int64_t>(sms) * std::max(per_sm, 1));
  }
  if (e != cudaSuccess) return e;
  p.terms = ctas;
  return row::launch(kernel, dim3(static_cast<unsigned>(ctas)), R::kThreads, smem, stream, p);
}

template <typename T>
cudaError_t launch_rows(PolicyLaunch& p, int sms, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  const size_t step = static_cast<size_t>(p.ld) * sizeof(T) % 16;
  const bool aligned = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 && (p.n == 1 || step == 0);
  p.same_cut = p.dlogits && (reinterpret_cast<uintptr_t>(p.dlogits) - reinterpret_cast<uintptr_t>(p.logits)) % 16 == 0 &&
               (p.n == 1 || static_cast<size_t>(p.ldd) * sizeof(T) % 16 == step);
  const bool edges = !aligned || p.vocab % E != 0;
  p.cluster = 1;
  // As a shared row's slot: beside the groups, the rest of the first granule and the one read past the last.
  const int64_t slot = ((p.vocab + E - 1) / E + 2) * 16;
  if (slot <= kSoloSlotBytes) {
    p.slot_bytes = static_cast<int>(slot);
    return edges ? launch_solo<T, true>(p, sms, stream) : launch_solo<T, false>(p, sms, stream);
  }
  bool launched = false;
  const cudaError_t e = edges ? launch_shared<T, true>(p, stream, &launched) : launch_shared<T, false>(p, stream, &launched);
  if (e != cudaSuccess || launched) return e;
  p.terms = p.n;
  return row::launch(policy_twice_kernel<T>, dim3(static_cast<unsigned>(p.n)), kTwiceThreads, 0, stream, p);
}

}  // namespace

int64_t policy_workspace(int64_t n) { return n * static_cast<int64_t>(sizeof(float)); }

cudaError_t launch_policy(PolicyLaunch& p, int sms, cudaStream_t stream) {
  if (p.n == 0) return p.loss ? cudaMemsetAsync(p.loss, 0, sizeof(float), stream) : cudaSuccess;
  return p.dtype == 0 ? launch_rows<float>(p, sms, stream) : launch_rows<__nv_bfloat16>(p, sms, stream);
}

}  // namespace dmuon
