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
// row's sums are shuffles among the lanes that hold it. A warp takes a token's heads one batch of groups after another:
// the angles, their sines and cosines are formed once for all of them, and the next batches' elements are on their way
// while this one's are turned. Lanes have 8 columns of a row whose columns come in aligned fours, else single pairs.
//
// What bounds it is memory, as far as enough of it is asked for ahead. Measured, 16384 tokens, 32 + 8 heads of 128 bf16
// columns, three axes: forward 58 us, 5.8 TB/s (0.86 of a copy's rate); backward 93 us, 5.4 TB/s (0.81), where the sums
// of the gains' gradients leave registers for 16 warps an SM. 8191 tokens, 9 + 3 heads of 78 fp32 columns of which 20
// turn, backward: 35 to 39 us, of which the kernel is 27, instructions of 39 pairs on 16 lanes.
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

// Each of the sums over the lanes of a row.
template <int N>
__device__ __forceinline__ void sum_lanes(float (&v)[N], int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
}

// The first group of tensor w that part `part` of a token's heads has.
__device__ __forceinline__ int first_group(const RotaryLaunch& p, int w, int part, int per_warp) {
  if (p.parts == 1) return 0;
  const int first = (part - (w ? (p.heads[0] + per_warp - 1) / per_warp : 0)) % p.parts;
  return first < 0 ? first + p.parts : first;
}

// 4, 8 or 16 bytes into shared memory, asynchronously; zeros if not `ok`, whatever is at src.
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool ok) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(__cvta_generic_to_global(src)), "n"(kBytes),
               "r"(ok ? kBytes : 0)
               : "memory");
}

// The rows of `kArrays` arrays that a warp takes: batches of G groups of a tensor's heads, across tensors and tokens alike,
// so that a token's first rows are on their way while the last of the one before are turned. They come through shared
// memory, kStages batches ahead, every lane its own (so a lane waits for its copies alone); single pairs of bf16, whose
// ends may be 2 bytes each, through registers, one batch ahead.
template <typename T, int V, int I, bool INTER, int G, int kStages, int kArrays>
struct Rows {
  static constexpr bool kShared = V > 1 || sizeof(T) == 4;
  static constexpr int kPiece = V * sizeof(T);                      // of a lane's item, twice
  static constexpr int kOther = V == 1 ? 4 : kPiece * 32;           // from a lane's lower piece to its upper one
  static constexpr int kBatch = kArrays * G * I * 2 * kPiece * 32;  // bytes of a warp's batch
  int64_t unit;
  int w, group, h, slot;
  const T* at[kArrays];
  uint32_t ring;
  Raw<T, V> next[kShared ? 1 : kArrays][kShared ? 1 : G][I];

  // Array 0 of two is dy; x is the other, or the only one.
  __device__ __forceinline__ static const void* base(const RotaryLaunch& p, int a, int w) {
    return a || kArrays == 1 ? p.x[w] : p.dy[w];
  }
  __device__ __forceinline__ static int64_t token_stride(const RotaryLaunch& p, int a, int w) {
    return a || kArrays == 1 ? p.x_token[w] : p.dy_token[w];
  }
  __device__ __forceinline__ static int64_t head_stride(const RotaryLaunch& p, int a, int w) {
    return a || kArrays == 1 ? p.x_head[w] : p.dy_head[w];
  }
  // The next tensor of which this warp has groups, from w of the current unit on.
  __device__ __forceinline__ void find(const RotaryLaunch& p, int64_t units, int64_t warps, int per_warp, int sub) {
    for (; unit < units; unit += warps, w = 0) {
      const int64_t token = p.parts == 1 ? unit : unit / p.parts;
      const int part = static_cast<int>(unit - token * p.parts);
      for (; w < 2; ++w) {
        const int first = first_group(p, w, part, per_warp);
        if (first * per_warp >= p.heads[w]) continue;
        group = first, h = first * per_warp + sub;
#pragma unroll
        for (int a = 0; a < kArrays; ++a)
          at[a] = static_cast<const T*>(base(p, a, w)) + token * token_stride(p, a, w) + h * head_stride(p, a, w);
        return;
      }
    }
  }
  __device__ __forceinline__ void ask(const RotaryLaunch& p, const Place<V, I, INTER>& place, int64_t units, int64_t warps,
                                      int per_warp, int sub) {
    if (unit < units) {
      const int step = p.parts * per_warp;
#pragma unroll
      for (int u = 0; u < G; ++u) {
        const bool ok = h + u * step < p.heads[w];
#pragma unroll
        for (int a = 0; a < kArrays; ++a) {
          const bool wanted = ok && (a == 0 || p.norm);
          const T* row = at[a] + static_cast<int64_t>(u * step) * head_stride(p, a, w);
          if constexpr (kShared) {
#pragma unroll
            for (int i = 0; i < I; ++i) {
              const uint32_t dst = ring + slot * kBatch + ((a * G + u) * I + i) * 2 * kPiece * 32;
              const bool live = wanted && place.live[i];
              const void* lo = live ? static_cast<const void*>(row + place.lo[i]) : base(p, 0, 0);
              if (V == 1 && INTER && p.wide) {
                copy_async<8>(dst, lo, live);
              } else {
                copy_async<kPiece>(dst, lo, live);
                copy_async<kPiece>(dst + kOther, live ? static_cast<const void*>(row + place.hi[i]) : lo, live);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < I; ++i) {
              if (wanted && place.live[i]) {
                next[a][u][i] = load_item<T, V, INTER>(row, place.lo[i], place.hi[i], p.wide);
              } else {
#pragma unroll
                for (int k = 0; k < Raw<T, V>::kWords; ++k) next[a][u][i].w[k] = 0u;
              }
            }
          }
        }
      }
      group += G * p.parts, h += G * step;
      if (group * per_warp >= p.heads[w]) {
        ++w;
        find(p, units, warps, per_warp, sub);
      } else {
#pragma unroll
        for (int a = 0; a < kArrays; ++a) at[a] += static_cast<int64_t>(G * step) * head_stride(p, a, w);
      }
    }
    if constexpr (kShared) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (++slot == kStages) slot = 0;
    }
  }
  __device__ __forceinline__ Rows(const RotaryLaunch& p, const Place<V, I, INTER>& place, uint8_t* smem, int64_t first_unit,
                                  int64_t units, int64_t warps, int per_warp, int sub)
      : unit(first_unit), w(0), slot(0) {
    if constexpr (kShared)
      ring = ptx::smem_u32(smem) + (threadIdx.x >> 5) * kStages * kBatch + (threadIdx.x & 31) * (V == 1 ? 8 : kPiece);
    find(p, units, warps, per_warp, sub);
#pragma unroll 1
    for (int k = 0; k < (kShared ? kStages : 1); ++k) ask(p, place, units, warps, per_warp, sub);
  }
  // The oldest batch, as fp32; and another is asked for in its place.
  __device__ __forceinline__ void take(float2 (&z)[kArrays][G][I][V], const RotaryLaunch& p, const Place<V, I, INTER>& place,
                                       int64_t units, int64_t warps, int per_warp, int sub) {
    if constexpr (kShared) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      Raw<T, V> raw[kArrays][G][I];
#pragma unroll
      for (int a = 0; a < kArrays; ++a)
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int i = 0; i < I; ++i)
#pragma unroll
            for (int side = 0; side < (V == 1 ? 1 : 2); ++side) {
              const uint32_t src = ring + slot * kBatch + ((a * G + u) * I + i) * 2 * kPiece * 32 + side * kOther;
              uint32_t* to = raw[a][u][i].w + side * kPiece / 4;
              if constexpr (V == 1 || kPiece == 8)
                asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(to[0]), "=r"(to[1]) : "r"(src) : "memory");
              else
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(to[0]), "=r"(to[1]), "=r"(to[2]), "=r"(to[3])
                             : "r"(src)
                             : "memory");
            }
#pragma unroll
      for (int a = 0; a < kArrays; ++a)
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int i = 0; i < I; ++i) unpack_item<T, V>(z[a][u][i], raw[a][u][i]);
    } else {
#pragma unroll
      for (int a = 0; a < kArrays; ++a)
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int i = 0; i < I; ++i) unpack_item<T, V>(z[a][u][i], next[a][u][i]);
    }
    ask(p, place, units, warps, per_warp, sub);
  }
};

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

// Groups of a batch, whose sums run side by side, and batches ahead. At the sizes above, forward: one group through
// registers 85 us, two in a batch of four stages 63, four in two or three stages 58, eight 84 (one CTA per SM for want of
// registers). Backward: through registers 128 us, one group in four stages 106, two in two to four stages 93 to 95, two
// without the limit of 128 registers 117.
template <typename T, int V> constexpr int kGroups = V > 1 ? 4 : sizeof(T) == 4 ? 2 : 1;
template <typename T, int V> constexpr int kGradGroups = V > 1 ? 2 : sizeof(T) == 4 ? 2 : 1;
constexpr int kStages = 2, kGradStages = 2;

// Work of one warp: units of a token's head groups. A group is the 32 / lanes heads that a warp holds at once; groups
// of queries come before those of keys, and part k of `parts` takes every parts-th of them.
template <typename T, int V, int I, bool INTER, int G>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryLaunch p) {
  extern __shared__ __align__(16) uint8_t smem[];
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, sub = lane / p.lanes, per_warp = 32 / p.lanes;
  const Place<V, I, INTER> at(p, lane % p.lanes);
  ptx::griddep_wait();
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps, units = p.n * p.parts;
  int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  Rows<T, V, I, INTER, G, kStages, 1> rows(p, at, smem, unit, units, warps, per_warp, sub);
  for (; unit < units; unit += warps) {
    const int64_t token = p.parts == 1 ? unit : unit / p.parts;
    const int part = static_cast<int>(unit - token * p.parts);
    float c[I * V], s[I * V];
    at.turns(p, token, c, s);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int heads = p.heads[w], first = first_group(p, w, part, per_warp), step = p.parts * per_warp;
      int h = first * per_warp + sub;
      if (first * per_warp >= heads) continue;
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
      T* y = static_cast<T*>(p.y[w]) + token * p.y_token[w] + h * p.y_head[w];
      const int64_t step_y = step * p.y_head[w];
      for (int head = first * per_warp; head < heads; head += G * step) {
        float2 z[1][G][I][V];
        rows.take(z, p, at, units, warps, per_warp, sub);
        float rho[G];
        if (p.norm) {
#pragma unroll
          for (int u = 0; u < G; ++u) {
            float2 sq = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
              for (int k = 0; k < V; ++k) sq = fma2(z[0][u][i][k], z[0][u][i][k], sq);
            rho[u] = sq.x + sq.y;
          }
          sum_lanes(rho, p.lanes);
#pragma unroll
          for (int u = 0; u < G; ++u) rho[u] = rsqrtf(fmaf(rho[u], p.inv_dim, p.eps));
        }
#pragma unroll
        for (int u = 0; u < G; ++u) {
          const bool ok = h + u * step < heads;
#pragma unroll
          for (int i = 0; i < I; ++i) {
            float2 out[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
              out[k] = fma2(z[0][u][i][k], along[i][k], mul2(partner<V, INTER>(z[0][u][i], k), across[i][k]));
              if (p.norm) out[k] = mul2(out[k], both(rho[u]));
            }
            if (ok && at.live[i]) store_item<T, V, INTER>(y + u * step_y, at.lo[i], at.hi[i], p.wide, out);
          }
        }
        h += G * step;
        y += G * step_y;
      }
    }
  }
}

// y holds dx and x the norm's input; dy the gradient that arrives.
template <typename T, int V, int I, bool INTER, int G>
__global__ void __launch_bounds__(kThreads, 2) rotary_grad_kernel(const __grid_constant__ RotaryLaunch p) {
  extern __shared__ __align__(16) uint8_t smem[];
  ptx::griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / p.lanes, per_warp = 32 / p.lanes;
  const Place<V, I, INTER> at(p, lane % p.lanes);
  ptx::griddep_wait();
  float2 sums[2][I][V] = {};
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarps, units = p.n * p.parts;
  int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  using Stream = Rows<T, V, I, INTER, G, kGradStages, 2>;
  Stream rows(p, at, smem, unit, units, warps, per_warp, sub);
  for (; unit < units; unit += warps) {
    const int64_t token = p.parts == 1 ? unit : unit / p.parts;
    const int part = static_cast<int>(unit - token * p.parts);
    float c[I * V], s[I * V];
    at.turns(p, token, c, s);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int heads = p.heads[w], first = first_group(p, w, part, per_warp), step = p.parts * per_warp;
      int h = first * per_warp + sub;
      if (first * per_warp >= heads) continue;
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
      T* dx = static_cast<T*>(p.y[w]) + token * p.y_token[w] + h * p.y_head[w];
      const int64_t step_dx = step * p.y_head[w];
      for (int head = first * per_warp; head < heads; head += G * step) {
        float2 in[2][G][I][V], d[G][I][V];
        rows.take(in, p, at, units, warps, per_warp, sub);
        auto& z = in[1];
#pragma unroll
        for (int u = 0; u < G; ++u)
#pragma unroll
          for (int i = 0; i < I; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k)
              d[u][i][k] = fma2(in[0][u][i][k], cos2[i][k], mul2(partner<V, INTER>(in[0][u][i], k), sin2[i][k]));
        if (p.norm) {
          float rho[2 * G];  // the sums of squares; those of dn . x
#pragma unroll
          for (int u = 0; u < G; ++u) {
            float2 sq = make_float2(0.f, 0.f), along = sq;
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
              for (int k = 0; k < V; ++k) {
                sq = fma2(z[u][i][k], z[u][i][k], sq);
                along = fma2(mul2(d[u][i][k], g[i][k]), z[u][i][k], along);
              }
            rho[u] = sq.x + sq.y, rho[G + u] = along.x + along.y;
          }
          sum_lanes(rho, p.lanes);
#pragma unroll
          for (int u = 0; u < G; ++u) {
            const float r = rsqrtf(fmaf(rho[u], p.inv_dim, p.eps)), back = -r * r * (rho[G + u] * p.inv_dim);
#pragma unroll
            for (int i = 0; i < I; ++i)
#pragma unroll
              for (int k = 0; k < V; ++k) {
                const float2 hat = mul2(z[u][i][k], both(r));
                sums[w][i][k] = fma2(d[u][i][k], hat, sums[w][i][k]);
                d[u][i][k] = fma2(hat, both(back), mul2(mul2(d[u][i][k], g[i][k]), both(r)));
              }
          }
        }
#pragma unroll
        for (int u = 0; u < G; ++u) {
          const bool ok = h + u * step < heads;
#pragma unroll
          for (int i = 0; i < I; ++i)
            if (ok && at.live[i]) store_item<T, V, INTER>(dx + u * step_dx, at.lo[i], at.hi[i], p.wide, d[u][i]);
        }
        h += G * step;
        dx += G * step_dx;
      }
    }
  }
  if (!p.partials) return;
  float* part_sums = reinterpret_cast<float*>(smem + (Stream::kShared ? kWarps * kGradStages * Stream::kBatch : 0));
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
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
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

template <typename T, int V, int I, bool INTER, int G>
cudaError_t launch_forward(RotaryLaunch& p, int sms, cudaStream_t stream) {
  static int known[kMaxDevices];
  int64_t ctas = 0;
  using Stream = Rows<T, V, I, INTER, G, kStages, 1>;
  constexpr size_t smem = Stream::kShared ? kWarps * kStages * Stream::kBatch : 0;
  const cudaError_t e = set_grid(p, rotary_kernel<T, V, I, INTER, G>, known, smem, sms, &ctas);
  if (e != cudaSuccess) return e;
  return row::launch(rotary_kernel<T, V, I, INTER, G>, dim3(static_cast<unsigned>(ctas)), kThreads, smem, stream, p);
}

template <typename T, int V, int I, bool INTER, int G>
cudaError_t launch_backward(RotaryLaunch& p, int sms, cudaStream_t stream) {
  static int known[kMaxDevices];
  int64_t ctas = 0;
  using Stream = Rows<T, V, I, INTER, G, kGradStages, 2>;
  constexpr size_t ring = Stream::kShared ? kWarps * kGradStages * Stream::kBatch : 0;
  const size_t smem = ring + sizeof(float) * 2 * p.dim * kWarps;
  cudaError_t e =
      set_grid(p, rotary_grad_kernel<T, V, I, INTER, G>, known, ring + sizeof(float) * 2 * 256 * kWarps, sms, &ctas);
  if (e != cudaSuccess) return e;
  p.npartials = static_cast<int>(ctas);
  if (p.planning) return cudaSuccess;
  e = row::launch(rotary_grad_kernel<T, V, I, INTER, G>, dim3(static_cast<unsigned>(ctas)), kThreads, smem, stream, p);
  if (e != cudaSuccess || !p.partials) return e;
  return row::launch(rotary_gain_kernel, dim3(static_cast<unsigned>((2 * p.dim + 31) / 32)), kJoinThreads, 0, stream, p);
}

template <typename T, int V, int I, bool INTER>
cudaError_t launch_as(RotaryLaunch& p, int sms, cudaStream_t stream) {
  // Up to three groups of a tensor's heads that a warp has of a token: batches of one, which leave none of a batch empty.
  // 32768 tokens, bf16, us in batches of one and of more: 2 + 1 heads of 128 30.5, 46.3 (backward 40, 50), 6 + 2 45.9, 50.8
  // (59, 66), 8 + 2 52.1, 51.7 (67, 67), 16 + 4 66, 56 (88, 79); 200 tokens of 32 + 8 5.0, 5.9 (9.3, 10.2).
  const int per_warp = 32 / p.lanes, most = (std::max(p.heads[0], p.heads[1]) + per_warp - 1) / per_warp;
  const int64_t warps = 16 * static_cast<int64_t>(sms), each = most * std::min(p.n, warps) / warps;
  if (!p.grad)
    return each <= 3 ? launch_forward<T, V, I, INTER, 1>(p, sms, stream)
                     : launch_forward<T, V, I, INTER, kGroups<T, V>>(p, sms, stream);
  return each <= 3 ? launch_backward<T, V, I, INTER, 1>(p, sms, stream)
                   : launch_backward<T, V, I, INTER, kGradGroups<T, V>>(p, sms, stream);
}

template <typename T, bool INTER>
cudaError_t launch_type(RotaryLaunch& p, int sms, cudaStream_t stream) {
  // Fours of bf16 rather than eights: half the registers, and twice the warps (through registers, 16384 x 40 x 128:
  // forward 90 us with eights, 87 with fours; backward 245, 138).
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
