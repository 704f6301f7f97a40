// Residual addition with RMS norm, h = x + r, y = h * rho * gain with rho = (mean(h^2) + eps)^(-1/2), and
// its backward pass.
//
// The norm is formed from h before h is rounded to its stored type; sums are fp32. With an 8-bit output
// each group of consecutive columns (or the whole row) has scale = max |y| / 448 (1 for a group of zeros)
// and q = e4m3(y / scale).
//
// Backward, for the stored h: with d = dy * gain,
//   dx = dh + rho d - h rho^3 / dim * sum(d h),   dgain = sum over rows of dy h rho.
//
// Each element is read once and written once. A row is held in the registers of `tpr` threads, K 16-byte granules
// of it in each, so one read serves the sums and the outputs. Rows need not
// start on 16 bytes: granules are cut where the addresses are aligned, and the up to 2 (E - 1) elements before
// and behind them are held one per thread. CTAs stay and take every (gridDim.x * rows per CTA)-th row, a multiple
// of 8, so all rows of a thread start at the same offset from 16 bytes whatever their length: its columns, and
// with them its gains and its sums for dgain, stay the same.
//
// The forward sum has one order for every layout: thread t of sum_threads adds groups of E elements t,
// t + sum_threads, ... counted from the row's first element, then the threads join. Rows that are not whole
// granules pass through shared memory for it, so a value's bits do not depend on where it lies.
//
// Bounds. Rows of whole granules: memory, forward at 16384 x 4096 bf16 85 us (6.3 TB/s), fp32 171 (6.3), backward
// 92 (5.8) and 168 (6.4). Rows with edges: the instructions that cut and realign them, forward at 65344 x 1027 bf16
// 121 us (4.4 TB/s), fp32 180 (6.0), backward 111 (4.8) and 168 (6.4). 8-bit outputs: the chain from the row's sum
// over the group's maximum to the bytes, with two or three rows at a time per SM: 16384 x 4096 bf16 83 us (5.7
// TB/s), 3001 x 8200 fp32 60 (5.4); with edges, where groups pass through shared memory twice, 65344 x 1027 bf16
// 187 (2.5). One row: latency, 4 us on the device, and the launch.
#include <algorithm>

#include <cuda_fp8.h>

#include "row_ops.h"
#include "tc_ptx.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;  // of a CTA that holds short rows, and of the kernels for the longest ones
constexpr int kMaxThreads = 1024;
constexpr int kHugeThreads = 576;  // of two CTAs per SM that hold 16 elements of a long fp32 row in each thread
constexpr float kFp8Max = 448.f;  // largest finite e4m3
constexpr float kMinScale = 1.17549435e-38f;

// top / 448, rounded once, for the bits of a group's largest |y|: the product with 1 / 448 held in two parts (Brisebarre,
// Muller and Raina, "Accelerating correctly rounded floating-point division when the divisor is known in advance",
// 2004; equal to the quotient for all 2^23 significands). The bound on the second part keeps an infinity one.
__device__ __forceinline__ float scale_of(unsigned top_bits) {
  constexpr float kHigh = 0x1.24924ap-9f, kLow = -0x1.b6db6ep-34f;
  const float top = __uint_as_float(top_bits), quotient = fmaf(top, kHigh, fmaxf(top * kLow, -1e38f));
  return top == 0.f ? 1.f : (top < kFp8Max * kMinScale ? kMinScale : quotient);
}

// Largest |y| of the block as the bits of a non-negative float; a NaN is larger than every number.
__device__ __forceinline__ unsigned block_top(unsigned v, unsigned* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return __reduce_max_sync(0xffffffffu, (threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0u);
}

// ---------------------------------------------------------------------------- granules

template <typename T>
constexpr int kPer = 16 / sizeof(T);  // elements of a granule

template <typename T>
__device__ __forceinline__ void store_granule(T* dst, const float (&v)[kPer<T>]) {
  __stcs(reinterpret_cast<uint4*>(dst), row::pack16(v));
}

// Where a row lies: `head` elements before the first 16-byte address, `full` granules, `tail` elements.
template <typename T>
struct Cut {
  int head, full, tail;
  __device__ __forceinline__ Cut(const T* x, int dim) {
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    head = min((kPer<T> - off) & (kPer<T> - 1), dim);
    full = (dim - head) / kPer<T>;
    tail = dim - head - full * kPer<T>;
  }
  // The element outside the granules that thread t of a row (16 threads at least) holds, or -1.
  __device__ __forceinline__ int edge(int t) const {
    if (t < head) return t;
    if (t >= 8 && t - 8 < tail) return head + full * kPer<T> + t - 8;
    return -1;
  }
};

// Gains [e0, e0 + E), ones outside the row or without gains.
template <int E>
__device__ __forceinline__ void load_gain(float (&g)[E], const float* gain, int e0, int dim) {
  if (gain && e0 + E <= dim && (reinterpret_cast<uintptr_t>(gain + e0) & 15) == 0) {
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(gain + e0 + j));
      g[j] = u.x, g[j + 1] = u.y, g[j + 2] = u.z, g[j + 3] = u.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < E; ++j) g[j] = gain && e0 + j < dim ? __ldg(gain + e0 + j) : 1.f;
}

// Sums over the `tpr` threads of a row. `red` alternates between two halves from row to row, so one barrier
// per row is enough. All threads of the CTA call it.
template <int N>
__device__ __forceinline__ void row_sum(float (&s)[N], int tpr, float (*red)[32][N], int half) {
  if (tpr >= 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  } else {
    for (int o = tpr / 2; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < N; ++k) s[k] += __shfl_xor_sync(0xffffffffu, s[k], o);
  }
  if (tpr <= 32) {
    __syncwarp();  // as the barrier below does for wider rows: what a row left in shared memory is there for the next
    return;
  }
  const int warp = threadIdx.x >> 5, warps = tpr >> 5, first = warp / warps * warps;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) red[half][warp][k] = s[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) s[k] = 0.f;
  for (int w = first; w < first + warps; ++w)
#pragma unroll
    for (int k = 0; k < N; ++k) s[k] += red[half][w][k];
}

// The threads of a row meet.
__device__ __forceinline__ void row_sync(int tpr) {
  if (tpr <= 32)
    __syncwarp();
  else
    __syncthreads();
}

// ---------------------------------------------------------------------------- forward

// max that gives NaN for NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float c;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(c) : "f"(a), "f"(b));
  return c;
}

// Within one unit of the last place, against e4m3's four significant bits: a quotient by the scale is within 2^-22 of
// itself, so a value that close to a border between two e4m3 numbers may fall on its other side (__fdiv_rn for the scale
// and __frcp_rn here, within 2^-23: 67108 x 1000 bf16 82 -> 92 us). The same for every layout, so that the bytes are.
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// E elements as e4m3 bytes.
template <int E>
__device__ __forceinline__ void pack_fp8(uint32_t (&w)[E / 4], const float (&v)[E], float inv) {
#pragma unroll
  for (int j = 0; j < E; j += 4) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[j] * inv, v[j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[j + 2] * inv, v[j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    w[j / 4] = lo | hi << 16;
  }
}

// THREADS: the most of a CTA. HELD: gains stay in registers and the next row is loaded early; without it, for
// longer rows, a thread has fewer registers, more CTAs overlap, and the next row is asked into L2 (16-byte
// pieces of it, by one copy instruction; 5460 x 12289 bf16: 179 us without, 153 with; fp32 rows with edges gain
// too, 65344 x 1027 210 -> 182 us, and all others lose, 16384 x 4096 bf16 85 -> 91). EDGES: rows that are not
// whole granules. CTAs of 256 threads that registers leave room for: four with one aligned granule a thread
// (1048576 x 64 bf16: 92 us with three, 84 with four), three and two where there is more to hold (65344 x 1027
// bf16: 126 us with three, 148 with four). Of longer rows one or two: fp32 rows with edges would spill at two (8183 x
// 8201: 218 us with two, 192 with one; to e4m3 249 and 201).
template <typename T, int K, bool FP8, int THREADS, bool HELD, bool EDGES>
__global__ void __launch_bounds__(THREADS, HELD ? (FP8 || EDGES ? (K > 1 ? 2 : 3) : K > 1 ? 3 : 4)
                                                : EDGES && sizeof(T) == 4 ? 1
                                                : THREADS <= 320 || THREADS == kHugeThreads ? 2 : 1)
    add_rmsnorm_rows_kernel(const RmsNormLaunch p) {
  constexpr int E = kPer<T>;
  __shared__ float red[2][32][1];
  extern __shared__ __align__(16) uint8_t dyn[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tpr = p.tpr, rows = blockDim.x / tpr, slot = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int dim = static_cast<int>(p.dim);
  const int64_t step = p.step, first = static_cast<int64_t>(blockIdx.x) * rows;
  const T* x = static_cast<const T*>(p.x) + (first + slot) * p.ldx;
  const T* r = p.residual ? static_cast<const T*>(p.residual) + (first + slot) * p.ldr : nullptr;
  T* h = p.h ? static_cast<T*>(p.h) + (first + slot) * p.ldh : nullptr;
  const Cut<T> cut(x, dim);
  const int full = EDGES ? cut.full : dim / E, edge = EDGES ? cut.edge(t) : -1;
  auto start = [&](int k) { return (EDGES ? cut.head : 0) + (t + k * tpr) * E; };
  auto holds = [&](int k) { return t + k * tpr < full; };
  // 8-bit outputs of such rows are formed from the line below, by groups of elements from the row's first one.
  constexpr bool LINED = FP8 && EDGES;
  auto first_out = [&](int k) { return LINED ? (t + k * tpr) * E : start(k); };
  float gain[HELD ? K : 1][E];
  if (HELD)
#pragma unroll
    for (int k = 0; k < K; ++k) load_gain(gain[k], p.gain, first_out(k), dim);
  const float gain_edge = EDGES && !FP8 && edge >= 0 && p.gain ? __ldg(p.gain + edge) : 1.f;

  // For a group that is not within a warp, the largest |y| of each (as bits, which order as the values do),
  // alternating between two halves. Then a row of bytes. Then h in the order of its elements, a word left out
  // after every 32, so that lanes E elements apart use different banks.
  const int group_bits = p.group ? 31 - __clz(static_cast<int>(p.group)) : 30;  // log2 of a group, longer than the row without
  const int parts = FP8 ? p.parts : 0, top_bytes = FP8 && p.lanes == 0 ? (2 * rows * parts * 4 + 15) / 16 * 16 : 0;
  unsigned* tops = reinterpret_cast<unsigned*>(dyn);
  uint8_t* bytes = dyn + top_bytes + slot * p.stage;
  float* line = reinterpret_cast<float*>(dyn + top_bytes + rows * p.stage) + slot * p.line;
  if (top_bytes) {
    for (int k = threadIdx.x; k < 2 * rows * parts; k += blockDim.x) tops[k] = 0;
    __syncthreads();
  }

  uint4 xr[K], rr[K];
  T xe{}, re{};
  auto fetch = [&](int64_t i) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool in = i < p.n && holds(k);
      xr[k] = in ? __ldcs(reinterpret_cast<const uint4*>(x + start(k))) : make_uint4(0, 0, 0, 0);
      rr[k] = in && r ? __ldcs(reinterpret_cast<const uint4*>(r + start(k))) : make_uint4(0, 0, 0, 0);
    }
    if (EDGES && i < p.n && edge >= 0) {
      xe = x[edge];
      if (r) re = r[edge];
    }
  };
  if (HELD) fetch(first + slot);
  int half = 0;
  for (int64_t base = first; base < p.n; base += step, half ^= 1) {
    const int64_t i = base + slot;
    if (!HELD) fetch(i);
    float v[K][E], ve = 0.f;
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float a[E], b[E];
      row::unpack16<T>(a, xr[k]);
      row::unpack16<T>(b, rr[k]);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        v[k][j] = a[j] + b[j];
        if (!EDGES) s[0] = fmaf(v[k][j], v[k][j], s[0]);
      }
    }
    if (EDGES) ve = row::to_f(xe) + row::to_f(re);
    x += p.step_x;
    if (r) r += p.step_r;
    if (HELD && base + step < p.n) fetch(i + step);
    if ((!HELD || (EDGES && sizeof(T) == 4 && !FP8)) && t == 0 && full > 0 && i + (HELD ? 2 : 1) * step < p.n) {
      const int head = EDGES ? cut.head : 0;
      ptx::prefetch_l2(x + (HELD ? p.step_x : 0) + head, full * 16);
      if (r) ptx::prefetch_l2(r + (HELD ? p.step_r : 0) + head, full * 16);
    }
    if (h && i < p.n) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (holds(k)) store_granule(h + start(k), v[k]);
      if (edge >= 0) h[edge] = row::from_f<T>(ve);
    }
    if (h) h += p.step_h;
    if (EDGES) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (holds(k)) {
          const int e0 = start(k), border = 32 - (e0 & 31);  // where a granule crosses a left-out word
          float* to = line + e0 + (e0 >> 5);
#pragma unroll
          for (int j = 0; j < E; ++j) to[j + (j >= border ? 1 : 0)] = v[k][j];
        }
      if (edge >= 0) line[edge + (edge >> 5)] = ve;
      row_sync(tpr);
      // Group t + k tpr from the row's first element: tpr is sum_threads, or the row has fewer groups than either.
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int e0 = (t + k * tpr) * E;
        const float* from = line + e0 + (e0 >> 5);
        float u[E];
#pragma unroll
        for (int j = 0; j < E; ++j) u[j] = 0.f;
        if (e0 + E <= dim) {
#pragma unroll
          for (int j = 0; j < E; ++j) u[j] = from[j];
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j)
            if (e0 + j < dim) u[j] = from[j];
        }
#pragma unroll
        for (int j = 0; j < E; ++j) {
          s[0] = fmaf(u[j], u[j], s[0]);
          if (LINED) v[k][j] = u[j];
        }
      }
    }
    row_sum(s, tpr, red, half);
    const float rho = rsqrtf(fmaf(s[0], p.inv_dim, p.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!HELD) load_gain(gain[0], p.gain, first_out(k), dim);
#pragma unroll
      for (int j = 0; j < E; ++j) v[k][j] = v[k][j] * rho * gain[HELD ? k : 0][j];
    }
    if constexpr (!FP8) {
      T* y = static_cast<T*>(p.y) + i * p.ldy;
      if (i < p.n) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (holds(k)) store_granule(y + start(k), v[k]);
        if (edge >= 0) y[edge] = row::from_f<T>(ve * rho * gain_edge);
      }
    } else {
      unsigned* top = tops + (half * rows + slot) * parts;
      float most[K];  // of the granule, then of its group
#pragma unroll
      for (int k = 0; k < K; ++k) {
        most[k] = 0.f;
#pragma unroll
        for (int j = 0; j < E; ++j) most[k] = max_nan(most[k], fabsf(v[k][j]));
      }
      if (p.group == 0) {
#pragma unroll
        for (int k = 1; k < K; ++k) most[0] = max_nan(most[0], most[k]);
#pragma unroll
        for (int k = 1; k < K; ++k) most[k] = most[0];
      }
      for (int o = (p.lanes ? p.lanes : 32) / 2; o > 0; o >>= 1)  // a group's lanes, or a part of them
#pragma unroll
        for (int k = 0; k < K; ++k) most[k] = max_nan(most[k], __shfl_xor_sync(0xffffffffu, most[k], o));
      if (p.lanes == 0)
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (i < p.n && first_out(k) < dim && (threadIdx.x & 31) == 0)
            atomicMax(top + (first_out(k) >> group_bits), __float_as_uint(most[k]));
      if (p.lanes == 0) {
        row_sync(tpr);
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (first_out(k) < dim) most[k] = __uint_as_float(top[first_out(k) >> group_bits]);
        for (int k = t; k < parts; k += tpr) {
          if (i < p.n) p.scales[i * parts + k] = scale_of(top[k]);
          tops[((half ^ 1) * rows + slot) * parts + k] = 0;  // for the next row; its readers are a barrier behind
        }
      }
      uint8_t* q = static_cast<uint8_t*>(p.y) + i * p.ldy;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int e0 = first_out(k);
        if (i >= p.n || e0 >= dim) continue;
        const float scale = scale_of(__float_as_uint(most[k]));
        if (p.lanes && (t & (p.lanes - 1)) == 0) p.scales[i * parts + (e0 >> group_bits)] = scale;
        uint32_t w[E / 4];
        pack_fp8(w, v[k], reciprocal(scale));
        uint8_t* to = p.stage ? bytes + e0 : q + e0;
        if constexpr (E == 8)
          *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
        else
          *reinterpret_cast<uint32_t*>(to) = w[0];
      }
      if (p.stage) {
        row_sync(tpr);
        // The row goes out by 16-byte addresses, what lies there beginning between words of the bytes; up to 15 bytes
        // on either side one per thread.
        const int head = min(static_cast<int>((0 - reinterpret_cast<uintptr_t>(q)) & 15), dim), whole = (dim - head) >> 4;
        if (i < p.n) {
#pragma unroll 1
          for (int c = t; c < whole; c += tpr) {
            const int lo = head + 16 * c, bits = (lo & 3) * 8;
            const uint32_t* from = reinterpret_cast<const uint32_t*>(bytes) + (lo >> 2);
            uint4 o;
            o.x = __funnelshift_r(from[0], from[1], bits), o.y = __funnelshift_r(from[1], from[2], bits);
            o.z = __funnelshift_r(from[2], from[3], bits), o.w = __funnelshift_r(from[3], from[4], bits);
            __stcs(reinterpret_cast<uint4*>(q + lo), o);
          }
#pragma unroll 1
          for (int b = t; b < head; b += tpr) q[b] = bytes[b];
#pragma unroll 1
          for (int b = head + 16 * whole + t; b < dim; b += tpr) q[b] = bytes[b];
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------- backward

// The sums for dgain of a thread's columns, and its gains, stay in registers (REGS) or in shared memory.
// AHEAD: the next row is loaded early. PER_SM: CTAs that registers are to leave room for.
template <typename T, int K, int THREADS, int PER_SM, bool REGS, bool AHEAD, bool EDGES>
__global__ void __launch_bounds__(THREADS, PER_SM) add_rmsnorm_grad_rows_kernel(const RmsNormGradLaunch p) {
  constexpr int E = kPer<T>;
  __shared__ float red[2][32][2];
  extern __shared__ __align__(16) uint8_t dyn[];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tpr = p.tpr, rows = blockDim.x / tpr, slot = threadIdx.x / tpr, t = threadIdx.x % tpr;
  const int dim = static_cast<int>(p.dim);
  const int64_t step = p.step, first = static_cast<int64_t>(blockIdx.x) * rows;
  const T* dy = static_cast<const T*>(p.dy) + (first + slot) * p.lddy;
  const T* h = static_cast<const T*>(p.h) + (first + slot) * p.ldh;
  const T* dh = p.dh ? static_cast<const T*>(p.dh) + (first + slot) * p.lddh : nullptr;
  T* dx = static_cast<T*>(p.dx) + (first + slot) * p.lddx;
  const Cut<T> cut(dy, dim);
  const int full = EDGES ? cut.full : dim / E, edge = EDGES ? cut.edge(t) : -1;
  auto start = [&](int k) { return (EDGES ? cut.head : 0) + (t + k * tpr) * E; };
  auto holds = [&](int k) { return t + k * tpr < full; };
  float gain[REGS ? K : 1][E], acc[REGS ? K : 1][E], acc_edge = 0.f;
  const float gain_edge = edge >= 0 && p.gain ? __ldg(p.gain + edge) : 1.f;
  // Without REGS a thread's sums, then its gains: four columns at [quarter][granule], so that a warp's accesses do
  // not conflict. (Gains loaded from memory at each use: 8192 x 8192 bf16 107 us, 98 with them here.)
  const int granules = K * tpr, held = REGS ? 0 : E / 4 * granules * 2;  // of a row
  float4* sums = reinterpret_cast<float4*>(dyn) + slot * held;
  float4* gains = sums + E / 4 * granules;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float g[E];
    load_gain(g, p.gain, start(k), dim);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (REGS) {
        gain[k][j] = g[j];
        acc[k][j] = 0.f;
      } else if (j % 4 == 0) {
        sums[j / 4 * granules + t + k * tpr] = make_float4(0.f, 0.f, 0.f, 0.f);
        gains[j / 4 * granules + t + k * tpr] = make_float4(g[j], g[j + 1], g[j + 2], g[j + 3]);
      }
    }
  }
  // Into gain[0], without REGS.
  auto gains_of = [&](int k) {
#pragma unroll
    for (int j = 0; j < E; j += 4) {
      const float4 u = gains[j / 4 * granules + t + k * tpr];
      gain[0][j] = u.x, gain[0][j + 1] = u.y, gain[0][j + 2] = u.z, gain[0][j + 3] = u.w;
    }
  };
  struct Row {
    uint4 y[K], h[K], t[K];
    T ye, he, te;
  };
  Row now{}, next{};
  const bool leads = t == 0 && full > 0;
  auto fetch = [&](Row& to, int64_t i) {
    const bool live = i < p.n;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const bool in = live && holds(k);
      to.y[k] = in ? __ldcs(reinterpret_cast<const uint4*>(dy + start(k))) : make_uint4(0, 0, 0, 0);
      to.h[k] = in ? __ldcs(reinterpret_cast<const uint4*>(h + start(k))) : make_uint4(0, 0, 0, 0);
      to.t[k] = in && dh ? __ldcs(reinterpret_cast<const uint4*>(dh + start(k))) : make_uint4(0, 0, 0, 0);
    }
    if (EDGES) {
      to.ye = to.he = to.te = row::from_f<T>(0.f);
      if (live && edge >= 0) {
        to.ye = dy[edge];
        to.he = h[edge];
        if (dh) to.te = dh[edge];
      }
    }
    dy += p.step_dy;
    h += p.step_h;
    if (dh) dh += p.step_dh;
    // Into L2 the row after it (16372 x 4099 fp32: 186 -> 168 us, 4194 x 16000 bf16 146 -> 116; bf16 rows that are
    // loaded early lose, 16384 x 4096 103 -> 107).
    if ((!AHEAD || sizeof(T) == 4) && leads && i + step < p.n) {
      const int head = EDGES ? cut.head : 0;
      ptx::prefetch_l2(dy + head, full * 16);
      ptx::prefetch_l2(h + head, full * 16);
      if (dh) ptx::prefetch_l2(dh + head, full * 16);
    }
  };
  if (AHEAD) fetch(next, first + slot);
  int half = 0;
  for (int64_t base = first; base < p.n; base += step, half ^= 1) {
    const int64_t i = base + slot;
    const bool live = i < p.n;
    if (AHEAD) {
      now = next;
      if (base + step < p.n) fetch(next, i + step);
    } else {
      fetch(now, i);
    }
    float s[2] = {0.f, 0.f};  // sum of h^2, sum of d h
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float a[E], b[E];
      row::unpack16<T>(a, now.y[k]);
      row::unpack16<T>(b, now.h[k]);
      if (!REGS) gains_of(k);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        s[0] = fmaf(b[j], b[j], s[0]);
        s[1] = fmaf(a[j] * gain[REGS ? k : 0][j], b[j], s[1]);
      }
    }
    const float he = EDGES ? row::to_f(now.he) : 0.f, de = EDGES ? row::to_f(now.ye) * gain_edge : 0.f;
    if (EDGES) {
      s[0] = fmaf(he, he, s[0]);
      s[1] = fmaf(de, he, s[1]);
    }
    row_sum(s, tpr, red, half);
    // Behind the last row everything is 0, rho too.
    const float rho = live ? rsqrtf(fmaf(s[0], p.inv_dim, p.eps)) : 0.f;
    const float back = s[1] * p.inv_dim * rho * rho * rho;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float a[E], b[E], c[E];
      row::unpack16<T>(a, now.y[k]);
      row::unpack16<T>(b, now.h[k]);
      row::unpack16<T>(c, now.t[k]);
      if (!REGS) gains_of(k);
      float4 sum;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        const float hat = b[j] * rho;
        if (REGS) {
          acc[k][j] = fmaf(a[j], hat, acc[k][j]);
        } else {
          if (j % 4 == 0) sum = sums[j / 4 * granules + t + k * tpr];
          float& to = j % 4 == 0 ? sum.x : j % 4 == 1 ? sum.y : j % 4 == 2 ? sum.z : sum.w;
          to = fmaf(a[j], hat, to);
          if (j % 4 == 3) sums[j / 4 * granules + t + k * tpr] = sum;
        }
        c[j] = fmaf(rho, a[j] * gain[REGS ? k : 0][j], fmaf(-back, b[j], c[j]));
      }
      if (live && holds(k)) store_granule(dx + start(k), c);
    }
    if (EDGES && live && edge >= 0) {
      acc_edge = fmaf(row::to_f(now.ye), he * rho, acc_edge);
      dx[edge] = row::from_f<T>(fmaf(rho, de, fmaf(-back, he, row::to_f(now.te))));
    }
    dx += p.step_dx;
  }
  if (!p.dgain) return;
  // This CTA's sums, one row of the workspace. The row slots of a CTA start at different offsets, so they join
  // by column, in their order.
  float* out = p.partials + static_cast<int64_t>(blockIdx.x) * p.dim;
  float* line = reinterpret_cast<float*>(reinterpret_cast<float4*>(dyn) + rows * held);
  for (int turn = 0; turn < rows; ++turn) {
    if (rows > 1) __syncthreads();
    if (turn != slot) continue;
    auto put = [&](int e, float v) {
      if (rows > 1) {
        if (turn > 0) v += line[e];
        line[e] = v;
      }
      if (turn == rows - 1) out[e] = v;
    };
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (holds(k))
#pragma unroll
        for (int j = 0; j < E; ++j) {
          if (REGS) {
            put(start(k) + j, acc[k][j]);
          } else {
            const float4 sum = sums[j / 4 * granules + t + k * tpr];
            put(start(k) + j, j % 4 == 0 ? sum.x : j % 4 == 1 ? sum.y : j % 4 == 2 ? sum.z : sum.w);
          }
        }
    if (edge >= 0) put(edge, acc_edge);
  }
}

// dgain from the CTAs' sums: a CTA takes 32 columns, its warps every 32nd row of the workspace, then a column each.
// Latency of the loads of a warp bounds it. The sums are added by pairs: one after the other they were most of dgain's
// error (65537 x 129 fp32: 1.54e-7 of itself, one after the other 1.70e-7; 16384 x 4096 fp32 1.63e-7 and 1.88e-7; 27.5 us
// for the former's gradient, 26.5 so).
__global__ void __launch_bounds__(kMaxThreads) rmsnorm_dgain_kernel(const RmsNormGradLaunch p) {
  constexpr int kWarps = kMaxThreads / 32;
  static_assert(kWarps == 32, "a warp's lanes are the warps' sums");
  __shared__ float sums[kWarps][33];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * 32, c = first + lane;
  float acc = 0.f;
  if (c < p.dim) {
    const float* from = p.partials + warp * p.dim + c;
    const int64_t step = kWarps * p.dim;
#pragma unroll 1
    for (int left = p.npartials - warp; left > 0; left -= 8 * kWarps) {
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = k * kWarps < left ? __ldcg(from) : 0.f;
        from += step;
      }
      acc += ((v[0] + v[4]) + (v[1] + v[5])) + ((v[2] + v[6]) + (v[3] + v[7]));
    }
  }
  sums[warp][lane] = acc;
  __syncthreads();
  acc = sums[lane][warp];
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0 && first + warp < p.dim) {
    float* to = p.dgain + first + warp;
    *to = p.accumulate ? *to + acc : acc;
  }
}

// ---------------------------------------------------------------------------- the longest rows

// One CTA per row, each element read again for every use: rows beyond what registers hold (3000 x 20000 bf16: 133 us
// forward, 427 backward), and arrays that start at different offsets from 16 bytes, whose granules no one cut fits.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) add_rmsnorm_kernel(const RmsNormLaunch p) {
  __shared__ float red[2][32][1];
  __shared__ unsigned redu[32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  constexpr int E = kPer<T>;
  const int threads = blockDim.x;
  const int64_t i = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + i * p.ldx;
  const T* r = p.residual ? static_cast<const T*>(p.residual) + i * p.ldr : nullptr;
  T* h = p.h ? static_cast<T*>(p.h) + i * p.ldh : nullptr;
  float sq[1] = {0.f};
  if (threadIdx.x < p.sum_threads)
    for (int64_t c0 = threadIdx.x * E; c0 < p.dim; c0 += p.sum_threads * E)
      for (int64_t c = c0; c < min(c0 + E, p.dim); ++c) {
        const float v = row::to_f(x[c]) + (r ? row::to_f(r[c]) : 0.f);
        sq[0] = fmaf(v, v, sq[0]);
      }
  row_sum(sq, threads, red, 0);
  const float rho = rsqrtf(fmaf(sq[0], p.inv_dim, p.eps));
  auto value = [&](int64_t c) {
    const float v = row::to_f(x[c]) + (r ? row::to_f(r[c]) : 0.f);
    return v * rho * (p.gain ? p.gain[c] : 1.f);
  };
  if (!p.scales) {
    T* y = static_cast<T*>(p.y) + i * p.ldy;
    for (int64_t c = threadIdx.x; c < p.dim; c += threads) {
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
    for (int64_t c = begin + threadIdx.x; c < end; c += threads) top = max(top, __float_as_uint(fabsf(value(c))));
    const float scale = scale_of(block_top(top, redu));
    const float inv = reciprocal(scale);
    if (threadIdx.x == 0) p.scales[i * parts + k] = scale;
    for (int64_t c = begin + threadIdx.x; c < end; c += threads) {
      const float v = row::to_f(x[c]) + (r ? row::to_f(r[c]) : 0.f);
      q[c] = __nv_cvt_float_to_fp8(value(c) * inv, __NV_SATFINITE, __NV_E4M3);
      if (h) h[c] = row::from_f<T>(v);
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) add_rmsnorm_grad_kernel(const RmsNormGradLaunch p) {
  __shared__ float red[32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
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
  const float rho = rsqrtf(fmaf(sq, p.inv_dim, p.eps));
  const float back = along * p.inv_dim * rho * rho * rho;
  if (!p.dx) {
    if (threadIdx.x == 0) p.rho[i] = rho;
    return;
  }
  for (int64_t c = threadIdx.x; c < p.dim; c += kThreads) {
    const float d = row::to_f(dy[c]) * (p.gain ? p.gain[c] : 1.f);
    static_cast<T*>(p.dx)[i * p.lddx + c] = row::from_f<T>(rho * d - back * row::to_f(h[c]) + (dh ? row::to_f(dh[c]) : 0.f));
  }
}

// dgain for them: a CTA takes 32 columns over a stretch of rows, its warps every eighth row of it, and leaves
// their sums in the workspace.
template <typename T>
__global__ void __launch_bounds__(kThreads) rmsnorm_columns_kernel(const RmsNormGradLaunch p) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float sums[kWarps][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  const int64_t begin = p.n * blockIdx.y / gridDim.y, end = p.n * (blockIdx.y + 1) / gridDim.y;
  float acc = 0.f;
  if (c < p.dim)
    for (int64_t i = begin + warp; i < end; i += kWarps)
      acc = fmaf(row::to_f(static_cast<const T*>(p.dy)[i * p.lddy + c]) * p.rho[i],
                 row::to_f(static_cast<const T*>(p.h)[i * p.ldh + c]), acc);
  sums[warp][lane] = acc;
  __syncthreads();
  if (warp == 0 && c < p.dim) {
    for (int w = 1; w < kWarps; ++w) acc += sums[w][lane];
    p.partials[blockIdx.y * p.dim + c] = acc;
  }
}

// ---------------------------------------------------------------------------- launches

constexpr int kMaxHeld = 16384;    // elements of a row held in registers: 32 or 16 by 512 or 1024 threads
constexpr int kColumnSplits = 32;  // stretches of rows of rmsnorm_columns_kernel

// A row's arrays and their strides, to see whether their granules coincide.
struct Array {
  const void* ptr;
  int64_t ld;
};

// Whether every array starts its rows at the same offsets from 16 bytes as the first one.
bool same_offsets(std::initializer_list<Array> arrays, int64_t n, size_t elem) {
  const Array& a = *arrays.begin();
  for (const Array& b : arrays)
    if (b.ptr && ((reinterpret_cast<uintptr_t>(b.ptr) - reinterpret_cast<uintptr_t>(a.ptr)) % 16 != 0 ||
                  (n > 1 && (static_cast<size_t>(b.ld) - static_cast<size_t>(a.ld)) * elem % 16 != 0)))
      return false;
  return true;
}

// Whether rows are not whole granules.
bool has_edges(const Array& a, int64_t n, int64_t dim, size_t elem) {
  return reinterpret_cast<uintptr_t>(a.ptr) % 16 != 0 || (n > 1 && static_cast<size_t>(a.ld) * elem % 16 != 0) ||
         static_cast<size_t>(dim) * elem % 16 != 0;
}

// Threads of a row for K granules each: whole warps, or a power of two below one.
int row_threads(int granules, int k) {
  const int need = (granules + k - 1) / k;
  if (need > 16) return (need + 31) / 32 * 32;
  int t = 1;
  while (t < need) t *= 2;
  return t;
}

constexpr size_t kPlainSmem = 40 * 1024;  // dynamic shared memory that needs no opt-in, beside the static one
constexpr int kMaxPerSm = 16;  // CTAs (of 160 threads at least)

struct RowGrid {
  int tpr, threads, rows;
  unsigned ctas;
};

// Resident CTAs of a kernel, all over the GPU and a multiple of 8 (152 SMs are), or fewer where the rows run out.
template <typename P>
cudaError_t row_grid(RowGrid& g, void (*kernel)(P), int tpr, int64_t n, size_t smem, int sms) {
  g.tpr = tpr;
  g.rows = g.tpr >= kThreads ? 1 : kThreads / g.tpr;
  g.threads = g.tpr * g.rows;
  const int64_t turns = (n + g.rows - 1) / g.rows;
  if (turns <= sms) {
    g.ctas = static_cast<unsigned>(turns);
    return cudaSuccess;
  }
  int per_sm = 0;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, g.threads, smem);
  if (e != cudaSuccess) return e;
  const int64_t most = std::max<int64_t>(8, static_cast<int64_t>(sms) * std::min(per_sm, kMaxPerSm) / 8 * 8);
  g.ctas = static_cast<unsigned>(std::min<int64_t>(most, turns));
  return cudaSuccess;
}

template <typename T, int K, bool FP8, int THREADS, bool HELD, bool EDGES>
cudaError_t launch_rows(RmsNormLaunch& p, int sms, cudaStream_t stream) {
  auto* kernel = add_rmsnorm_rows_kernel<T, K, FP8, THREADS, HELD, EDGES>;
  constexpr int E = kPer<T>;
  const int tpr = std::max(p.sum_threads, EDGES ? 16 : 1);
  size_t per_row = 0;
  p.parts = 0, p.stage = 0, p.lanes = 0;
  if (FP8) {
    p.parts = p.group ? static_cast<int>((p.dim + p.group - 1) / p.group) : 1;
    // Lanes that share a scale, where that is a part of a warp; a group may be longer than the row.
    const int lanes = p.group ? std::min(static_cast<int>(p.group) / E, tpr < 32 ? tpr : 1 << 30) : tpr;
    p.lanes = lanes <= 32 ? lanes : 0;
    if (p.lanes == 0) per_row += static_cast<size_t>(2 * p.parts * 4 + 16);
    // A granule's bytes are stored as such where they are aligned in every row.
    const bool direct = !EDGES && (reinterpret_cast<uintptr_t>(p.y) | static_cast<uintptr_t>(p.n == 1 ? 0 : p.ldy)) % E == 0;
    p.stage = direct ? 0 : static_cast<int>((p.dim + 15) / 16 * 16 + 32);
    per_row += static_cast<size_t>(p.stage);
  }
  p.line = EDGES ? static_cast<int>(p.dim + p.dim / 32 + 1) : 0;
  per_row += static_cast<size_t>(p.line) * 4;
  const size_t smem = per_row * (tpr >= kThreads ? 1 : kThreads / tpr);
  if (smem > kPlainSmem) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  RowGrid g;
  const cudaError_t e = row_grid(g, kernel, tpr, p.n, smem, sms);
  if (e != cudaSuccess) return e;
  p.tpr = g.tpr;
  p.step = static_cast<int64_t>(g.ctas) * g.rows;
  p.step_x = p.step * p.ldx, p.step_r = p.step * p.ldr, p.step_h = p.step * p.ldh;
  return row::launch(kernel, dim3(g.ctas), g.threads, smem, stream, p);
}

// Granules per thread: up to 64 granules a row is one warp's, so that it needs no barrier of the CTA (129 fp32
// columns backward: 52 us with two warps, 31 with one); then CTAs of 256 threads as long as that is 16 elements
// per thread. Beyond, fp32 rows of up to 2304 granules keep 16 elements per thread in CTAs of up to 576, two of
// which fit an SM (3001 x 8200 to e4m3: 84 us with 32 elements, 76 with 16), and the rest 32 elements. 8-bit outputs
// meet more often, so their rows are a warp's or two warps' for longer (67108 x 1000 to e4m3: bf16 95 us with one
// granule a thread, 89 with four, fp32 173 and 139; but 65344 x 1027 bf16 200 and 236); and of fp32 rows just above
// 128 granules a fifth warp would hold next to nothing (130308 x 515: 233 us with one, 171 with four).
template <typename T, bool FP8>
int granules_each(int granules) {
  constexpr int kHeld = sizeof(T) == 4 ? 4 : 2, kLong = sizeof(T) == 4 ? 8 : 4;
  constexpr int kFours = sizeof(T) == 4 ? (FP8 ? 256 : 160) : FP8 ? 128 : 64;  // rows up to which four gain
  if (granules > 64 && granules <= kFours) return 4;
  return granules <= 32 ? 1 : granules <= 64 ? 2 : granules <= 256 ? 1 : granules <= 512 ? 2
       : granules <= 256 * kHeld || (sizeof(T) == 4 && granules <= kHeld * kHugeThreads) ? kHeld : kLong;
}

template <typename T, bool FP8, bool EDGES>
cudaError_t launch_held_norm(RmsNormLaunch& p, int each, int sms, cudaStream_t stream) {
  constexpr int kHeld = sizeof(T) == 4 ? 4 : 2, kLong = sizeof(T) == 4 ? 8 : 4;
  if (each == 1) return launch_rows<T, 1, FP8, 256, true, EDGES>(p, sms, stream);
  if (each == 2) return launch_rows<T, 2, FP8, 256, true, EDGES>(p, sms, stream);
  if constexpr (sizeof(T) == 4) {
    if (each == kHeld && p.sum_threads > 256) return launch_rows<T, kHeld, FP8, kHugeThreads, false, EDGES>(p, sms, stream);
  }
  if (each == kHeld) return launch_rows<T, kHeld, FP8, 256, true, EDGES>(p, sms, stream);
  // Two CTAs of up to 320 threads fit an SM; rows for more are alone on it.
  if (p.sum_threads <= 320) return launch_rows<T, kLong, FP8, 320, false, EDGES>(p, sms, stream);
  return launch_rows<T, kLong, FP8, 512, false, EDGES>(p, sms, stream);
}

template <typename T, bool FP8>
cudaError_t launch_norm(RmsNormLaunch& p, int sms, cudaStream_t stream) {
  const int granules = static_cast<int>((p.dim + kPer<T> - 1) / kPer<T>), each = granules_each<T, FP8>(granules);
  p.sum_threads = std::min(row_threads(granules, each), kMaxThreads);
  // The mean of the squares is within two units of the last place by it. (With 1 / dim in two parts, which rounds as a
  // division does, no gradient's error was smaller, and 520223 x 129 bf16 took 160.4 us in place of 159.0.)
  p.inv_dim = 1.f / static_cast<float>(p.dim);
  const Array x{p.x, p.ldx};
  if (p.dim > kMaxHeld ||
      !same_offsets({x, {p.residual, p.ldr}, {p.h, p.ldh}, {FP8 ? nullptr : p.y, p.ldy}}, p.n, sizeof(T)))
    return row::launch(add_rmsnorm_kernel<T>, dim3(static_cast<unsigned>(p.n)), std::max(32, p.sum_threads), 0, stream, p);
  return has_edges(x, p.n, p.dim, sizeof(T)) ? launch_held_norm<T, FP8, true>(p, each, sms, stream)
                                             : launch_held_norm<T, FP8, false>(p, each, sms, stream);
}

template <typename T, int K, int THREADS, int PER_SM, bool REGS, bool AHEAD, bool EDGES>
cudaError_t launch_grad_rows(RmsNormGradLaunch& p, int granules, int sms, cudaStream_t stream) {
  auto* kernel = add_rmsnorm_grad_rows_kernel<T, K, THREADS, PER_SM, REGS, AHEAD, EDGES>;
  // Sums of long rows, or the line in which a CTA's short rows join.
  const int tpr = std::max(row_threads(granules, K), EDGES ? 16 : 1), rows = tpr >= kThreads ? 1 : kThreads / tpr;
  const size_t smem = (rows > 1 ? static_cast<size_t>(p.dim) * 4 : 0) +
                      (REGS ? 0 : static_cast<size_t>(rows) * K * tpr * kPer<T> * 4 * 2);
  if (p.planning) {
    if (smem > kPlainSmem) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) return e;
    }
    RowGrid g;
    const cudaError_t e = row_grid(g, kernel, tpr, p.n, smem, sms);
    if (e != cudaSuccess) return e;
    p.tpr = tpr;
    p.step = static_cast<int64_t>(g.ctas) * rows;
    p.step_dy = p.step * p.lddy, p.step_h = p.step * p.ldh, p.step_dh = p.step * p.lddh, p.step_dx = p.step * p.lddx;
    p.npartials = static_cast<int>(g.ctas);
    return cudaSuccess;
  }
  return row::launch(kernel, dim3(static_cast<unsigned>(p.npartials)), tpr * rows, smem, stream, p);
}

// A row's whole granules, K a thread, in CTAs that leave a thread the registers for them: 256 threads twice per SM,
// then one CTA per SM whose threads are as many as the row needs, since registers are divided among them. What
// spills loses; all at 67 million elements:
// - bf16, two granules: three CTAs 122 us, two 94 (dim 4096), with the sums in shared memory; in registers 95 (and of
//   rows up to 512 columns, a warp's, the same).
// - fp32 with edges, as of 65 granules two: dim 1027 225 us with one, 169 with two.
// - bf16 with edges, 513 to 1024 granules: four and two CTAs of 256 131 us, two in 512 and the next row ahead 112
//   (dim 6005); aligned rows the other way, 101 and 127 (dim 5000). To 1280 granules four in 320 threads 164 us, two in
//   640 133 (dim 8201).
// - fp32 beyond 2048 granules: four in 576 to 768 threads while that holds them (aligned, dim 10000: 181 us, 194 with
//   eight in 416; with edges, dim 8201: 189, 224), then eight in 512 (aligned, dim 16000: 175, 184 with four in 1024;
//   with edges, dim 11003: 210, 253).
// Sums of rows with edges lie in shared memory where that saves a spill or a CTA: with one granule (dim 129: bf16 110
// us in registers, 102; fp32 183, 174) and of bf16 rows (dim 515: 153, 98; dim 4099 172, 98).
template <typename T, bool EDGES>
cudaError_t launch_held_grad(RmsNormGradLaunch& p, int granules, int sms, cudaStream_t stream) {
  if (granules <= 32) return launch_grad_rows<T, 1, 256, 3, !EDGES, true, EDGES>(p, granules, sms, stream);
  if (granules <= 64) return launch_grad_rows<T, 2, 256, 2, !EDGES || sizeof(T) == 4, true, EDGES>(p, granules, sms, stream);
  if (granules <= 256 && !(EDGES && sizeof(T) == 4))
    return launch_grad_rows<T, 1, 256, 3, !EDGES, true, EDGES>(p, granules, sms, stream);
  if (granules <= 512) return launch_grad_rows<T, 2, 256, 2, sizeof(T) == 4, true, EDGES>(p, granules, sms, stream);
  if constexpr (EDGES && sizeof(T) == 2) {
    if (granules <= 1024) return launch_grad_rows<T, 2, 512, 1, false, true, EDGES>(p, granules, sms, stream);
    if (granules <= 1280) return launch_grad_rows<T, 2, 640, 1, false, false, EDGES>(p, granules, sms, stream);
  } else {
    if (granules <= 1024) return launch_grad_rows<T, 4, 256, 2, false, false, EDGES>(p, granules, sms, stream);
    if (granules <= 1280) return launch_grad_rows<T, 4, 320, 2, false, false, EDGES>(p, granules, sms, stream);
  }
  if (granules <= 2048) return launch_grad_rows<T, 4, 512, 1, false, false, EDGES>(p, granules, sms, stream);
  if constexpr (sizeof(T) == 4) {
    if constexpr (EDGES) {
      if (granules <= 2304) return launch_grad_rows<T, 4, kHugeThreads, 1, false, false, EDGES>(p, granules, sms, stream);
    } else {
      if (granules <= 3072) return launch_grad_rows<T, 4, 768, 1, false, false, EDGES>(p, granules, sms, stream);
    }
    return launch_grad_rows<T, 8, 512, 1, false, false, EDGES>(p, granules, sms, stream);
  }
  return cudaErrorInvalidValue;  // kMaxHeld bf16 are 2048 granules
}

template <typename T>
cudaError_t launch_grad(RmsNormGradLaunch& p, int sms, cudaStream_t stream) {
  const Array dy{p.dy, p.lddy};
  p.inv_dim = 1.f / static_cast<float>(p.dim);
  cudaError_t e;
  if (p.dim > kMaxHeld || !same_offsets({dy, {p.h, p.ldh}, {p.dh, p.lddh}, {p.dx, p.lddx}}, p.n, sizeof(T))) {
    const dim3 grid(static_cast<unsigned>(p.n));
    if (p.planning) {
      p.npartials = kColumnSplits;
      p.rhos = p.n;
      return cudaSuccess;
    }
    if (p.dgain) {  // before dx, which may be written over dy
      RmsNormGradLaunch only_rho = p;
      only_rho.dx = nullptr;
      e = row::launch(add_rmsnorm_grad_kernel<T>, grid, kThreads, 0, stream, only_rho);
      if (e != cudaSuccess) return e;
      e = row::launch(rmsnorm_columns_kernel<T>, dim3(static_cast<unsigned>((p.dim + 31) / 32), kColumnSplits), kThreads, 0,
                      stream, p);
      if (e != cudaSuccess) return e;
    }
    e = row::launch(add_rmsnorm_grad_kernel<T>, grid, kThreads, 0, stream, p);
  } else {
    const int granules = std::max(1, static_cast<int>(p.dim / kPer<T>));  // at most, whole ones
    e = has_edges(dy, p.n, p.dim, sizeof(T)) ? launch_held_grad<T, true>(p, granules, sms, stream)
                                             : launch_held_grad<T, false>(p, granules, sms, stream);
  }
  if (e != cudaSuccess || p.planning || !p.dgain) return e;
  return row::launch(rmsnorm_dgain_kernel, dim3(static_cast<unsigned>((p.dim + 31) / 32)), kMaxThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_add_rmsnorm(RmsNormLaunch& p, int sms, cudaStream_t stream) {
  if (p.scales)
    return p.dtype == 0 ? launch_norm<float, true>(p, sms, stream) : launch_norm<__nv_bfloat16, true>(p, sms, stream);
  return p.dtype == 0 ? launch_norm<float, false>(p, sms, stream) : launch_norm<__nv_bfloat16, false>(p, sms, stream);
}

cudaError_t plan_add_rmsnorm_grad(RmsNormGradLaunch& p, int sms) {
  p.planning = 1, p.rhos = 0;
  const cudaError_t e = launch_add_rmsnorm_grad(p, sms, nullptr);
  p.planning = 0;
  return e;
}

// Rows of sums, one per CTA or kColumnSplits; then a rho per row for the longest rows. Both are for dgain.
int64_t rmsnorm_grad_workspace(RmsNormGradLaunch& p, char* ws) {
  if (!p.dgain) return 0;
  const int64_t sums = (p.npartials * p.dim * 4 + 255) / 256 * 256;
  if (ws) {
    p.partials = reinterpret_cast<float*>(ws);
    p.rho = reinterpret_cast<float*>(ws + sums);
  }
  return sums + p.rhos * 4;
}

cudaError_t launch_add_rmsnorm_grad(RmsNormGradLaunch& p, int sms, cudaStream_t stream) {
  return p.dtype == 0 ? launch_grad<float>(p, sms, stream) : launch_grad<__nv_bfloat16>(p, sms, stream);
}

}  // namespace dmuon
