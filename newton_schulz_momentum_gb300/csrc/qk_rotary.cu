// RMS norm of each head's queries and keys with the position rotation in the same pass, and its backward pass.
//
// Per token and head with row x of `dim` elements: z = x rho g with rho = (mean x^2 + eps)^(-1/2) (or z = x without
// the norm); the first rotary_dim columns are pairs, (j, j + rotary_dim / 2) or, interleaved, (2j, 2j + 1), turned by
// the angle a_j = f_j * position:  y1 = z1 cos a - z2 sin a,  y2 = z2 cos a + z1 sin a.  With several axes frequency j
// follows the position of the axis whose section it lies in. The other columns pass.
//
// Backward: d = dy turned by -a, dn = d g, dx = rho dn - x rho^3 / dim sum(dn x), dg = sum over tokens and heads of
// d x rho.
//
// Angles. A frequency is held as its share of a revolution per position in units of 2^-64, so that frequency times
// position modulo one revolution is the low half of one integer product, exact but for the frequency's own rounding
// (2^-53 of it): positions of 2^31 are as good as small ones. fp32 angles would be off by 0.06 at position 10^6.
//
// Each element is read once and written once. A lane holds both ends of its pairs, so a turn needs no exchange, and a
// row's sums are shuffles among the lanes that hold it. A warp takes a token's heads one group after another: the
// angles, their sines and cosines are formed once for all of them, and the next group's elements are on their way while
// this one's are turned. Lanes have 8 columns of a row whose columns come in aligned fours, else single pairs.
#include <algorithm>

#include "row_ops.h"
#include "tc_ptx.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// What one lane holds of a row: item i is 2 V columns, those from lo on and V more from hi on; of interleaved pairs they
// are neighbours (hi = lo + V). They are held by twos, an instruction's worth of fp32 operations; partner(z, k) are the
// other ends of the pairs whose ends are z[k].
template <int V, bool INTER>
__device__ __forceinline__ float2 partner(const float2 (&z)[V], int k) {
  if constexpr (V == 1 || INTER) return make_float2(z[k].y, z[k].x);
  else return z[k ^ (V / 2)];
}
// Whether element e of an item is the first end of its pair, and the pair's number.
template <int V, bool INTER>
__device__ __forceinline__ constexpr bool first_end(int e) { return V == 1 || INTER ? e % 2 == 0 : e < V; }
template <int V, bool INTER>
__device__ __forceinline__ constexpr int pair_of(int e) { return V == 1 || INTER ? e / 2 : e % V; }

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)),
        "l"(reinterpret_cast<const unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 c;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(c))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return c;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// An item as it lies in memory. Of single pairs, neighbours are one access where the array allows it (`wide`).
template <typename T, int V>
struct Raw {
  static constexpr int kWords = V * 2 * static_cast<int>(sizeof(T)) / 4;  // 32-bit words; a pair of bf16 is one
  uint32_t w[kWords];
};

template <typename T, int V, bool INTER>
__device__ __forceinline__ Raw<T, V> load_item(const T* x, int lo, int hi, bool wide) {
  Raw<T, V> r;
  if constexpr (V == 1) {
    if (INTER && wide) {
      if constexpr (sizeof(T) == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(x + lo);
        r.w[0] = u.x, r.w[1] = u.y;
      } else {
        r.w[0] = *reinterpret_cast<const uint32_t*>(x + lo);
      }
    } else if constexpr (sizeof(T) == 4) {
      r.w[0] = *reinterpret_cast<const uint32_t*>(x + lo), r.w[1] = *reinterpret_cast<const uint32_t*>(x + hi);
    } else {
      r.w[0] = *reinterpret_cast<const uint16_t*>(x + lo) |
               static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(x + hi)) << 16;
    }
  } else if constexpr (sizeof(T) == 4) {
    const uint4 a = *reinterpret_cast<const uint4*>(x + lo), b = *reinterpret_cast<const uint4*>(x + hi);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w, r.w[4] = b.x, r.w[5] = b.y, r.w[6] = b.z, r.w[7] = b.w;
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(x + lo), b = *reinterpret_cast<const uint2*>(x + hi);
    r.w[0] = a.x, r.w[1] = a.y, r.w[2] = b.x, r.w[3] = b.y;
  }
  return r;
}

template <typename T, int V>
__device__ __forceinline__ void unpack_item(float2 (&z)[V], const Raw<T, V>& r) {
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if constexpr (sizeof(T) == 4) z[k] = make_float2(__uint_as_float(r.w[2 * k]), __uint_as_float(r.w[2 * k + 1]));
    else z[k] = make_float2(__uint_as_float(r.w[k] << 16), __uint_as_float(r.w[k] & 0xFFFF0000u));
  }
}

template <typename T, int V, bool INTER>
__device__ __forceinline__ void store_item(T* y, int lo, int hi, bool wide, const float2 (&z)[V]) {
  uint32_t w[Raw<T, V>::kWords];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if constexpr (sizeof(T) == 4) {
      w[2 * k] = __float_as_uint(z[k].x), w[2 * k + 1] = __float_as_uint(z[k].y);
    } else {
      const __nv_bfloat162 h = __floats2bfloat162_rn(z[k].x, z[k].y);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  if constexpr (V == 1) {
    if (INTER && wide) {
      if constexpr (sizeof(T) == 4) *reinterpret_cast<uint2*>(y + lo) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(y + lo) = w[0];
    } else if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<uint32_t*>(y + lo) = w[0], *reinterpret_cast<uint32_t*>(y + hi) = w[1];
    } else {
      *reinterpret_cast<uint16_t*>(y + lo) = static_cast<uint16_t>(w[0]);
      *reinterpret_cast<uint16_t*>(y + hi) = static_cast<uint16_t>(w[0] >> 16);
    }
  } else if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<uint4*>(y + lo) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4*>(y + hi) = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
    *reinterpret_cast<uint2*>(y + lo) = make_uint2(w[0], w[1]);
    *reinterpret_cast<uint2*>(y + hi) = make_uint2(w[2], w[3]);
  }
}

// A lane's place in a row and its angles. I items per lane, `lanes` lanes per row.
template <int V, int I, bool INTER>
struct Place {
  int lo[I], hi[I];
  bool live[I];
  uint32_t axis = 0;  // two bits per angle
  uint64_t freq[I * V];

  __device__ __forceinline__ Place(const RotaryLaunch& p, int lane_in_row) {
    const int half = p.rotary_dim / 2, turned = half / V, items = p.dim / (2 * V);
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int it = lane_in_row + i * p.lanes;
      live[i] = it < items;
      if (it < turned) {
        lo[i] = INTER ? 2 * V * it : V * it;
        hi[i] = INTER ? lo[i] + V : lo[i] + half;
      } else {
        lo[i] = p.rotary_dim + (it - turned) * (INTER ? 2 * V : V);
        hi[i] = lo[i] + (INTER ? V : (p.dim - p.rotary_dim) / 2);
      }
#pragma unroll
      for (int m = 0; m < V; ++m) {
        const int j = it * V + m;
        freq[i * V + m] = it < turned ? p.freqs[j] : 0;
        const uint32_t a = j >= p.section_end[0] ? (j >= p.section_end[1] ? (j >= p.section_end[2] ? 3 : 2) : 1) : 0;
        axis |= a << (2 * (i * V + m));
      }
    }
  }

  __device__ __forceinline__ void turns(const RotaryLaunch& p, int64_t token, float (&c)[I * V], float (&s)[I * V]) const {
    int64_t pos[4];
    pos[0] = row::load_id(p.positions, p.id_bytes, token);
#pragma unroll
    for (int a = 1; a < 4; ++a)
      pos[a] = a < p.axes ? row::load_id(p.positions, p.id_bytes, a * p.axis_stride + token) : 0;
#pragma unroll
    for (int k = 0; k < I * V; ++k) {
      int64_t at = pos[0];
      if (p.axes > 1) {
        const uint32_t a = (axis >> (2 * k)) & 3;
        at = a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3];
      }
      const uint64_t share = freq[k] * static_cast<uint64_t>(at);  // of a revolution, modulo 1
      // The nearest of 2^32 steps of a revolution, counted from -1/2 to 1/2: 2^-33 of a revolution off at most.
      const int near = static_cast<int>(static_cast<uint32_t>((share + 0x80000000ull) >> 32));
      sincospif(static_cast<float>(near) * 4.656612873077393e-10f, &s[k], &c[k]);  // 2^-31: halves of a revolution
    }
  }
};

__device__ __forceinline__ float sum_lanes(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A group's rows; zeros where there is no head or no item.
template <typename T, int V, int I, bool INTER>
__device__ __forceinline__ void load_group(Raw<T, V> (&r)[I], const T* x, const Place<V, I, INTER>& at, bool ok, bool wide) {
#pragma unroll
  for (int i = 0; i < I; ++i) {
    if (ok && at.live[i]) {
      r[i] = load_item<T, V, INTER>(x, at.lo[i], at.hi[i], wide);
    } else {
#pragma unroll
      for (int k = 0; k < Raw<T, V>::kWords; ++k) r[i].w[k] = 0u;
    }
  }
}

template <int V, int I, bool INTER>
__device__ __forceinline__ void load_gain(float2 (&g)[I][V], const float* gain, const Place<V, I, INTER>& at) {
#pragma unroll
  for (int i = 0; i < I; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = 2 * k < V || V == 1 ? at.lo[i] + 2 * k : at.hi[i] + 2 * k - V, c1 = V == 1 ? at.hi[i] : c + 1;
      g[i][k] = gain && at.live[i] ? make_float2(__ldg(gain + c), __ldg(gain + c1)) : make_float2(1.f, 1.f);
    }
}

// Work of one warp: units of a token's head groups. A group is the 32 / lanes heads that a warp holds at once; groups
// of queries come before those of keys, and part k of `parts` takes every parts-th of them.
template <typename T, int V, int I, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryLaunch p) {
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane / p.lanes, per_warp = 32 / p.lanes;
  const Place<V, I, INTER> at(p, lane % p.lanes);
  ptx::griddep_wait();
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); unit < p.n * p.parts; unit += warps) {
    const int64_t token = unit / p.parts;
    const int part = static_cast<int>(unit - token * p.parts);
    float c[I * V], s[I * V];
    at.turns(p, token, c, s);
    int before = 0;  // groups before this tensor's
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int heads = p.heads[w], groups = (heads + per_warp - 1) / per_warp;
      int first = (part - before) % p.parts;
      if (first < 0) first += p.parts;
      before += groups;
      if (first >= groups) continue;
      // y = rho (x gain cos + x' gain' sin), with the sign of the pair's end: both products' factors once per token.
      float2 g[I][V], along[I][V], across[I][V];
      load_gain<V, I, INTER>(g, p.gain[w], at);
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float2 other = partner<V, INTER>(g[i], k);
          const int m0 = i * V + pair_of<V, INTER>(2 * k), m1 = i * V + pair_of<V, INTER>(2 * k + 1);
          along[i][k] = make_float2(g[i][k].x * c[m0], g[i][k].y * c[m1]);
          across[i][k] = make_float2(other.x * (first_end<V, INTER>(2 * k) ? -s[m0] : s[m0]),
                                     other.y * (first_end<V, INTER>(2 * k + 1) ? -s[m1] : s[m1]));
        }
      const int64_t step = static_cast<int64_t>(p.parts) * per_warp, h0 = first * per_warp + sub;
      const T* x = static_cast<const T*>(p.x[w]) + token * p.x_token[w] + h0 * p.x_head[w];
      T* y = static_cast<T*>(p.y[w]) + token * p.y_token[w] + h0 * p.y_head[w];
      const int64_t step_x = step * p.x_head[w], step_y = step * p.y_head[w];
      Raw<T, V> next[I];
      load_group<T, V, I, INTER>(next, x, at, h0 < heads, p.wide);
      int h = static_cast<int>(h0);
      for (int group = first; group < groups; group += p.parts) {
        const bool ok = h < heads;
        h += static_cast<int>(step);
        x += step_x;
        float2 z[I][V];
#pragma unroll
        for (int i = 0; i < I; ++i) unpack_item<T, V>(z[i], next[i]);
        if (group + p.parts < groups) load_group<T, V, I, INTER>(next, x, at, h < heads, p.wide);
        float rho = 1.f;
        if (p.norm) {
          float2 sq = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < I; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) sq = fma2(z[i][k], z[i][k], sq);
          rho = rsqrtf(fmaf(sum_lanes(sq.x + sq.y, p.lanes), p.inv_dim, p.eps));
        }
#pragma unroll
        for (int i = 0; i < I; ++i) {
          float2 out[V];
#pragma unroll
          for (int k = 0; k < V; ++k)
            out[k] = mul2(fma2(z[i][k], along[i][k], mul2(partner<V, INTER>(z[i], k), across[i][k])), both(rho));
          if (ok && at.live[i]) store_item<T, V, INTER>(y, at.lo[i], at.hi[i], p.wide, out);
        }
        y += step_y;
      }
    }
  }
}

// y holds dx and x the norm's input; dy the gradient that arrives.
template <typename T, int V, int I, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_grad_kernel(const __grid_constant__ RotaryLaunch p) {
  extern __shared__ float part_sums[];  // 2 x dim of each warp
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / p.lanes, per_warp = 32 / p.lanes;
  const Place<V, I, INTER> at(p, lane % p.lanes);
  ptx::griddep_wait();
  float2 sums[2][I][V] = {};
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp; unit < p.n * p.parts; unit += warps) {
    const int64_t token = unit / p.parts;
    const int part = static_cast<int>(unit - token * p.parts);
    float c[I * V], s[I * V];
    at.turns(p, token, c, s);
    int before = 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int heads = p.heads[w], groups = (heads + per_warp - 1) / per_warp;
      int first = (part - before) % p.parts;
      if (first < 0) first += p.parts;
      before += groups;
      if (first >= groups) continue;
      float2 g[I][V], cos2[I][V], sin2[I][V];
      load_gain<V, I, INTER>(g, p.gain[w], at);
#pragma unroll
      for (int i = 0; i < I; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int m0 = i * V + pair_of<V, INTER>(2 * k), m1 = i * V + pair_of<V, INTER>(2 * k + 1);
          cos2[i][k] = make_float2(c[m0], c[m1]);
          sin2[i][k] = make_float2(first_end<V, INTER>(2 * k) ? s[m0] : -s[m0], first_end<V, INTER>(2 * k + 1) ? s[m1] : -s[m1]);
        }
      const int64_t step = static_cast<int64_t>(p.parts) * per_warp, h0 = first * per_warp + sub;
      const T* dy = static_cast<const T*>(p.dy[w]) + token * p.dy_token[w] + h0 * p.dy_head[w];
      const T* x = static_cast<const T*>(p.x[w]) + token * p.x_token[w] + h0 * p.x_head[w];
      T* dx = static_cast<T*>(p.y[w]) + token * p.y_token[w] + h0 * p.y_head[w];
      const int64_t step_dy = step * p.dy_head[w], step_x = step * p.x_head[w], step_dx = step * p.y_head[w];
      Raw<T, V> next_d[I], next_x[I];
      load_group<T, V, I, INTER>(next_d, dy, at, h0 < heads, p.wide);
      load_group<T, V, I, INTER>(next_x, x, at, p.norm && h0 < heads, p.wide);
      int h = static_cast<int>(h0);
      for (int group = first; group < groups; group += p.parts) {
        const bool ok = h < heads;
        h += static_cast<int>(step);
        dy += step_dy, x += step_x;
        float2 in[I][V], z[I][V], d[I][V];
#pragma unroll
        for (int i = 0; i < I; ++i) unpack_item<T, V>(in[i], next_d[i]), unpack_item<T, V>(z[i], next_x[i]);
        if (group + p.parts < groups) {
          load_group<T, V, I, INTER>(next_d, dy, at, h < heads, p.wide);
          load_group<T, V, I, INTER>(next_x, x, at, p.norm && h < heads, p.wide);
        }
#pragma unroll
        for (int i = 0; i < I; ++i)
#pragma unroll
          for (int k = 0; k < V; ++k) d[i][k] = fma2(in[i][k], cos2[i][k], mul2(partner<V, INTER>(in[i], k), sin2[i][k]));
        if (p.norm) {
          float2 sq = make_float2(0.f, 0.f), along = sq;
#pragma unroll
          for (int i = 0; i < I; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
              sq = fma2(z[i][k], z[i][k], sq);
              along = fma2(mul2(d[i][k], g[i][k]), z[i][k], along);
            }
          const float rho = rsqrtf(fmaf(sum_lanes(sq.x + sq.y, p.lanes), p.inv_dim, p.eps));
          const float back = -rho * rho * (sum_lanes(along.x + along.y, p.lanes) * p.inv_dim);
#pragma unroll
          for (int i = 0; i < I; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) {
              const float2 hat = mul2(z[i][k], both(rho));
              sums[w][i][k] = fma2(d[i][k], hat, sums[w][i][k]);
              d[i][k] = fma2(hat, both(back), mul2(mul2(d[i][k], g[i][k]), both(rho)));
            }
        }
#pragma unroll
        for (int i = 0; i < I; ++i)
          if (ok && at.live[i]) store_item<T, V, INTER>(dx, at.lo[i], at.hi[i], p.wide, d[i]);
        dx += step_dx;
      }
    }
  }
  if (!p.partials) return;
  // The warp's heads, then the CTA's warps, in fixed orders; the CTAs' sums are joined by rotary_gain_kernel.
#pragma unroll
  for (int w = 0; w < 2; ++w)
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int m = 0; m < 2 * V; ++m) {
        float v = m % 2 ? sums[w][i][m / 2].y : sums[w][i][m / 2].x;
        for (int o = 16; o >= p.lanes; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (sub == 0 && at.live[i])
          part_sums[(warp * 2 + w) * p.dim + (m < V ? at.lo[i] + m : at.hi[i] + m - V)] = v;
      }
  __syncthreads();
  for (int k = threadIdx.x; k < 2 * p.dim; k += kThreads) {
    float v = 0.f;
    for (int q = 0; q < kWarps; ++q) v += part_sums[q * 2 * p.dim + k];
    p.partials[static_cast<int64_t>(blockIdx.x) * 2 * p.dim + k] = v;
  }
}

constexpr int kJoinThreads = 1024;

// Sums of the gains' gradients over the CTAs of rotary_grad_kernel: 32 columns a CTA, warp q adds rows q, q + 32, ...
__global__ void __launch_bounds__(kJoinThreads) rotary_gain_kernel(const __grid_constant__ RotaryLaunch p) {
  __shared__ float part[32][33];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (k < 2 * p.dim)
    for (int r = warp; r < p.npartials; r += 32) v += p.partials[static_cast<int64_t>(r) * 2 * p.dim + k];
  part[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || k >= 2 * p.dim) return;
  v = 0.f;
  for (int q = 0; q < 32; ++q) v += part[q][lane];
  float* out = p.dgain[k / p.dim];
  if (out) out[k % p.dim] = v;
}

// Whether every row of every array starts at a multiple of `bytes`.
bool aligned_rows(const RotaryLaunch& p, size_t bytes) {
  const size_t size = p.dtype == 0 ? 4 : 2;
  auto fits = [&](const void* ptr, int64_t token, int64_t head) {
    return reinterpret_cast<uintptr_t>(ptr) % bytes == 0 && token * size % bytes == 0 && head * size % bytes == 0;
  };
  for (int w = 0; w < 2; ++w) {
    if (p.heads[w] == 0) continue;
    if (!fits(p.y[w], p.y_token[w], p.y_head[w])) return false;
    if (p.x[w] && !fits(p.x[w], p.x_token[w], p.x_head[w])) return false;
    if (p.dy[w] && !fits(p.dy[w], p.dy_token[w], p.dy_head[w])) return false;
  }
  return true;
}

// Lanes per row, a power of two, for `each` items a lane.
int lanes_for(int items, int each) {
  int lanes = 1;
  while (lanes * each < items) lanes *= 2;
  return lanes;
}

constexpr int kMaxDevices = 64;

// `known` holds what a kernel's occupancy on a device was found to be, for the largest `smem` (the caller holds the
// library's lock).
template <typename K>
cudaError_t set_grid(RotaryLaunch& p, K* kernel, int (&known)[kMaxDevices], size_t smem, int sms, int64_t* ctas) {
  int dev = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices) per_sm = known[dev];
  if (per_sm == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) known[dev] = per_sm;
  }
  const int64_t resident = static_cast<int64_t>(sms) * std::max(per_sm, 1);
  // A token's heads are shared out where there are fewer tokens than warps.
  const int per_warp = 32 / p.lanes;
  const int64_t groups = (p.heads[0] + per_warp - 1) / per_warp + (p.heads[1] + per_warp - 1) / per_warp;
  p.parts = static_cast<int>(std::max<int64_t>(1, std::min(groups, resident * kWarps / p.n)));
  *ctas = std::min(resident, (p.n * p.parts + kWarps - 1) / kWarps);
  return cudaSuccess;
}

template <typename T, int V, int I, bool INTER>
cudaError_t launch_as(RotaryLaunch& p, int sms, cudaStream_t stream) {
  static int known[2][kMaxDevices];
  int64_t ctas = 0;
  if (!p.grad) {
    const cudaError_t e = set_grid(p, rotary_kernel<T, V, I, INTER>, known[0], 0, sms, &ctas);
    if (e != cudaSuccess) return e;
    return row::launch(rotary_kernel<T, V, I, INTER>, dim3(static_cast<unsigned>(ctas)), kThreads, 0, stream, p);
  }
  const size_t smem = sizeof(float) * 2 * p.dim * kWarps;
  cudaError_t e = set_grid(p, rotary_grad_kernel<T, V, I, INTER>, known[1], sizeof(float) * 2 * 256 * kWarps, sms, &ctas);
  if (e != cudaSuccess) return e;
  p.npartials = static_cast<int>(ctas);
  if (p.planning) return cudaSuccess;
  e = row::launch(rotary_grad_kernel<T, V, I, INTER>, dim3(static_cast<unsigned>(ctas)), kThreads, smem, stream, p);
  if (e != cudaSuccess || !p.partials) return e;
  return row::launch(rotary_gain_kernel, dim3(static_cast<unsigned>((2 * p.dim + 31) / 32)), kJoinThreads, 0, stream, p);
}

template <typename T, bool INTER>
cudaError_t launch_type(RotaryLaunch& p, int sms, cudaStream_t stream) {
  // Fours of bf16 rather than eights: half the registers, and twice the warps (16384 x 40 x 128: forward 90 us with
  // eights, backward 245).
  if (p.rotary_dim % 8 == 0 && p.dim % 8 == 0 && aligned_rows(p, 4 * sizeof(T))) {
    p.lanes = lanes_for(p.dim / 8, 1);  // dim <= 256: at most 32
    p.wide = 1;
    return launch_as<T, 4, 1, INTER>(p, sms, stream);
  }
  // Pairs: as many to a lane as leave the fewest lanes idle (78 columns: 16 lanes of 3).
  p.wide = aligned_rows(p, 2 * sizeof(T));
  const int items = p.dim / 2;
  int each = 4;
  for (int e = 3; e >= 1; --e)
    if (lanes_for(items, e) <= 32 && lanes_for(items, e) * e <= lanes_for(items, each) * each) each = e;
  p.lanes = lanes_for(items, each);
  switch (each) {
    case 1: return launch_as<T, 1, 1, INTER>(p, sms, stream);
    case 2: return launch_as<T, 1, 2, INTER>(p, sms, stream);
    case 3: return launch_as<T, 1, 3, INTER>(p, sms, stream);
    default: return launch_as<T, 1, 4, INTER>(p, sms, stream);
  }
}

}  // namespace

int64_t rotary_workspace(RotaryLaunch& p, char* ws) {
  if (!p.dgain[0] && !p.dgain[1]) return 0;
  if (ws) p.partials = reinterpret_cast<float*>(ws);
  return static_cast<int64_t>(sizeof(float)) * p.npartials * 2 * p.dim;
}

cudaError_t launch_rotary(RotaryLaunch& p, int sms, cudaStream_t stream) {
  p.inv_dim = static_cast<float>(1.0 / p.dim);
  if (p.dtype == 0)
    return p.interleaved ? launch_type<float, true>(p, sms, stream) : launch_type<float, false>(p, sms, stream);
  return p.interleaved ? launch_type<__nv_bfloat16, true>(p, sms, stream)
                       : launch_type<__nv_bfloat16, false>(p, sms, stream);
}

}  // namespace dmuon
