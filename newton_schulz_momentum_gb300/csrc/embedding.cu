// Embedding lookup with scaling, out[i, :] = scale * table[id_i, :], and its gradient,
// grad[v, :] = scale * sum over the tokens i with id_i = v of grad_out[i, :], added in the order of i.
//
// The gradient of up to kDirectTokens tokens takes two launches: zeros, then a CTA per token that adds its row's tokens
// unless an earlier one of them does. Of more tokens, four:
//   1. one cluster sorts the tokens by id (stable);
//   2. meanwhile, on the other SMs, the table is filled with zeros, which at a language model's sizes is most
//      of the bytes (not run where the caller adds to the gradient);
//   3. the sorted list is cut into chunks of equal length, whatever the ids' frequencies: a CTA adds a
//      chunk's rows and writes each table row that begins and ends inside it; a row that crosses a chunk's
//      border leaves its sum over the chunk in the workspace;
//   4. the rows that cross borders are put together from their chunks' sums, in order.
// Bound by memory where the table is large: 16384 x 4096 bf16 tokens into 128256 rows take 348 us, 2.1 GB of them
// zeros and rows (6.4 TB/s in all). Small ones by the sort's latency, which is that of its passes and not of its
// tokens: 20011 x 1027 fp32 into 5003 rows take 44 us, the sort (two passes) 16 of them beside the zeros, the
// chunks' sums 19 and their joining 12. Equal ids in a row cost nothing more, nor do ids that are all the same.
#include <algorithm>

#include "row_ops.h"
#include "tc_ptx.h"

namespace dmuon {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------- lookup

constexpr int kLookup = 8;  // consecutive columns of a thread at a time

// Eight consecutive elements by 16-byte loads and stores.
__device__ __forceinline__ void load8(float (&v)[8], const float* src) {
  float lo[4], hi[4];
  row::unpack16<float>(lo, __ldg(reinterpret_cast<const uint4*>(src)));
  row::unpack16<float>(hi, __ldg(reinterpret_cast<const uint4*>(src) + 1));
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = lo[k], v[k + 4] = hi[k];
}
__device__ __forceinline__ void load8(float (&v)[8], const __nv_bfloat16* src) {
  row::unpack16<__nv_bfloat16>(v, __ldg(reinterpret_cast<const uint4*>(src)));
}
__device__ __forceinline__ void store8(float* dst, const float (&v)[8]) {
  __stcs(reinterpret_cast<float4*>(dst), make_float4(v[0], v[1], v[2], v[3]));
  __stcs(reinterpret_cast<float4*>(dst) + 1, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&v)[8]) {
  __stcs(reinterpret_cast<uint4*>(dst), row::pack16(v));
}

// Token i's row of the table (null for an id outside it, which is recorded) and of the output (null beyond the
// last token).
template <typename TI, typename TO>
__device__ __forceinline__ void source_row(const EmbeddingLaunch& p, int64_t i, int t, const TI*& src, TO*& dst) {
  src = nullptr, dst = nullptr;
  if (i >= p.n) return;
  const int64_t id = row::load_id(p.ids, p.id_bytes, i);
  if (id >= 0 && id < p.rows)
    src = static_cast<const TI*>(p.table) + id * p.ld_table;
  else if (t == 0)
    atomicOr(p.status, kDevIndex);
  dst = static_cast<TO*>(p.out) + i * p.ld_out;
}

// `tpr` threads take two tokens, so that twice as much is on its way (16384 x 4096 fp32 to bf16: 43 us with one, 41
// with two). Bound by memory: each row is read once (a row that several tokens name comes from L2 again) and the output
// is written once: 16384 x 4096 bf16 out of 128256 rows 35 us, 5.4 TB/s. A single token is bound by the launch.
template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) embedding_kernel(const EmbeddingLaunch p) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tpr = p.tpr, t = threadIdx.x % tpr;
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / tpr) + threadIdx.x / tpr) * 2;
  const TI* src[2];
  TO* dst[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) source_row(p, i0 + r, t, src[r], dst[r]);
  for (int64_t c = t * kLookup; c < p.dim; c += tpr * kLookup) {
    float v[2][kLookup];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int k = 0; k < kLookup; ++k) v[r][k] = 0.f;
      if (src[r]) load8(v[r], src[r] + c);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (!dst[r]) continue;
#pragma unroll
      for (int k = 0; k < kLookup; ++k) v[r][k] = src[r] ? p.scale * v[r][k] : 0.f;
      store8(dst[r] + c, v[r]);
    }
  }
}

// Rows that do not start on 16 bytes, or are not whole granules. The output is written in 16-byte granules at
// aligned addresses; a granule's elements begin anywhere in the table's row, so the aligned 16-byte words
// around them are read and shifted. Where those would reach beyond the row, and in the up to 2 (E - 1) elements
// beside the granules, single elements are read. (8193 x 8191 bf16: 41 us, 4.7 TB/s; 87 with single elements.)
template <typename TI, typename TO>
__global__ void __launch_bounds__(kThreads) embedding_shift_kernel(const EmbeddingLaunch p) {
  constexpr int E = 16 / sizeof(TO), BYTES = E * sizeof(TI), LOADS = (BYTES + 15) / 16 + 1, WORDS = LOADS * 4;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tpr = p.tpr, t = threadIdx.x % tpr, dim = static_cast<int>(p.dim);
  const int64_t i0 = (static_cast<int64_t>(blockIdx.x) * (kThreads / tpr) + threadIdx.x / tpr) * 2;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const TI* src;
    TO* dst;
    source_row(p, i0 + r, t, src, dst);
    if (!dst) continue;
    const int off = static_cast<int>((reinterpret_cast<uintptr_t>(dst) & 15) / sizeof(TO));
    const int head = min((E - off) & (E - 1), dim), full = (dim - head) / E, tail = dim - head - full * E;
    const int edge = t < head ? t : t >= 8 && t - 8 < tail ? head + full * E + t - 8 : -1;
    if (edge >= 0) dst[edge] = row::from_f<TO>(src ? p.scale * row::to_f(__ldg(src + edge)) : 0.f);
    const char* begin = reinterpret_cast<const char*>(src);
    const char* end = begin + static_cast<int64_t>(dim) * sizeof(TI);
    for (int q = t; q < full; q += tpr) {
      float v[E];
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = 0.f;
      if (src) {
        const TI* at = src + head + q * E;
        const int a = static_cast<int>(reinterpret_cast<uintptr_t>(at) & 15);
        const char* base = reinterpret_cast<const char*>(at) - a;
        if (base >= begin && base + LOADS * 16 <= end) {
          uint32_t w[WORDS];
#pragma unroll
          for (int l = 0; l < LOADS; ++l) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(base) + l);
            w[4 * l] = u.x, w[4 * l + 1] = u.y, w[4 * l + 2] = u.z, w[4 * l + 3] = u.w;
          }
          if (a & 8)
#pragma unroll
            for (int k = 0; k + 2 < WORDS; ++k) w[k] = w[k + 2];
          if (a & 4)
#pragma unroll
            for (int k = 0; k + 1 < WORDS; ++k) w[k] = w[k + 1];
          if (sizeof(TI) == 2 && (a & 2))
#pragma unroll
            for (int k = 0; k + 1 < WORDS; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
#pragma unroll
          for (int k = 0; k < E; ++k)
            v[k] = p.scale * (sizeof(TI) == 4 ? __uint_as_float(w[k])
                                              : __uint_as_float(k % 2 ? w[k / 2] & 0xffff0000u : w[k / 2] << 16));
        } else {
#pragma unroll
          for (int k = 0; k < E; ++k) v[k] = p.scale * row::to_f(__ldg(at + k));
        }
      }
      __stcs(reinterpret_cast<uint4*>(dst + head + q * E), row::pack16(v));
    }
  }
}

// ---------------------------------------------------------------------------- 1. sort

constexpr int kSortCtas = 8;  // one portable cluster
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;
constexpr int kHeldTokens = 4;  // per lane: all of them up to 32768
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr size_t kSortSmem = sizeof(uint32_t) * (kSortWarps + 2) * kMaxDigits;

// Token i's sort key: its id, or `rows` (behind every row) for padding and ids outside the table.
__device__ __forceinline__ uint32_t sort_key(const EmbeddingGradLaunch& p, int64_t i) {
  const int64_t id = row::load_id(p.ids, p.id_bytes, i);
  if (id < 0 || id >= p.rows) atomicOr(p.status, kDevIndex);
  return id >= 0 && id < p.rows && id != p.padding_idx ? static_cast<uint32_t>(id) : static_cast<uint32_t>(p.rows);
}

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Radix sort of the tokens, least significant digit first, by the CTAs of one cluster. Every warp holds a
// run of consecutive tokens; a token's place is the number of tokens with a smaller digit, plus those with
// the same digit in earlier CTAs, earlier warps and earlier in its warp, so equal ids keep their order. Bound by
// the latency of a pass, about 8 us: its tokens' loads, two barriers of the cluster, and the chains of shared
// memory between them. Digits have up to 9 bits, as few passes as that allows and of equal width: two of 9 bits for
// 128256 rows, two of 7 for 5003. Eight CTAs are the largest cluster of a portable size.
__device__ void sort_tokens(const EmbeddingGradLaunch& p, uint32_t* smem) {
  const int digits = 1 << p.digit_bits;
  uint32_t* count = smem;                               // [warp][digit]
  uint32_t* total = smem + kSortWarps * kMaxDigits;     // this CTA's tokens per digit, read by the cluster
  uint32_t* base = total + kMaxDigits;                  // first place of this CTA's tokens per digit
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const int64_t steps = (p.n + kSortCtas * kSortThreads - 1) / (kSortCtas * kSortThreads);  // per warp, 32 tokens each
  const int64_t first = (static_cast<int64_t>(rank) * kSortWarps + warp) * steps * 32;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.digit_bits;
    const uint2* in = p.sorted[(p.passes - pass) & 1];
    uint2* out = p.sorted[(p.passes - pass - 1) & 1];
    for (int k = threadIdx.x; k < kSortWarps * kMaxDigits; k += kSortThreads) count[k] = 0;
    __syncthreads();
    uint32_t* mine = count + warp * kMaxDigits;
    auto token = [&](int64_t i) {
      if (i >= p.n) return make_uint2(0xffffffffu, 0);
      return pass == 0 ? make_uint2(sort_key(p, i), static_cast<uint32_t>(i)) : __ldcg(in + i);
    };
    // The first tokens stay in registers for the second look at them, and which lanes have the same digit.
    uint2 held[kHeldTokens];
    unsigned alike[kHeldTokens];
#pragma unroll
    for (int s = 0; s < kHeldTokens; ++s) held[s] = s < steps ? token(first + s * 32 + lane) : make_uint2(0, 0);
    auto digit = [&](int64_t i, const uint2& t) { return i < p.n ? (t.x >> shift) & (digits - 1) : 0xffffffffu; };
    auto count_one = [&](int64_t i, const uint2& t) {
      const uint32_t d = digit(i, t);
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (d != 0xffffffffu && lane == __ffs(same) - 1) mine[d] += __popc(same);
      __syncwarp();
      return same;
    };
#pragma unroll
    for (int s = 0; s < kHeldTokens; ++s)
      if (s < steps) alike[s] = count_one(first + s * 32 + lane, held[s]);
    for (int64_t s = kHeldTokens; s < steps; ++s) count_one(first + s * 32 + lane, token(first + s * 32 + lane));
    __syncthreads();
    if (threadIdx.x < digits) {
      uint32_t of_warp[kSortWarps], sum = 0;
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) of_warp[w] = count[w * kMaxDigits + threadIdx.x];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        count[w * kMaxDigits + threadIdx.x] = sum;
        sum += of_warp[w];
      }
      total[threadIdx.x] = sum;
    }
    ptx::cluster_sync_all();
    // Exclusive sum over the digits of the cluster's totals: a warp's digits by shuffles, the warps in order.
    uint32_t all = 0, before = 0;
    if (threadIdx.x < digits) {
      const uint32_t at = ptx::smem_u32(total + threadIdx.x);
#pragma unroll
      for (uint32_t r = 0; r < kSortCtas; ++r) {
        const uint32_t c = ld_cluster(ptx::map_shared(at, r));
        all += c;
        if (r < rank) before += c;
      }
    }
    uint32_t upto = all;
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    __shared__ uint32_t warp_sum[kSortWarps];
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    if (threadIdx.x < digits) {
      uint32_t start = 0;
      for (int w = 0; w < warp; ++w) start += warp_sum[w];
      base[threadIdx.x] = start + upto - all + before;
    }
    __syncthreads();
    auto place_one = [&](int64_t i, const uint2& t, unsigned same) {
      const uint32_t d = digit(i, t);
      if (d != 0xffffffffu) {
        const uint32_t at = base[d] + mine[d] + __popc(same & ((1u << lane) - 1));
        if (dev_check(at < p.n, p.status)) __stcg(out + at, t);
      }
      __syncwarp();
      if (d != 0xffffffffu && lane == __ffs(same) - 1) mine[d] += __popc(same);
      __syncwarp();
    };
#pragma unroll
    for (int s = 0; s < kHeldTokens; ++s)
      if (s < steps) place_one(first + s * 32 + lane, held[s], alike[s]);
    for (int64_t s = kHeldTokens; s < steps; ++s) {
      const int64_t i = first + s * 32 + lane;
      const uint2 t = token(i);
      place_one(i, t, __match_any_sync(0xffffffffu, digit(i, t)));
    }
    // The next pass reads what the whole cluster wrote, and reuses the counts others have read.
    ptx::cluster_sync_all();
  }
}

__global__ void __cluster_dims__(kSortCtas) __launch_bounds__(kSortThreads, 1)
    embedding_sort_kernel(const EmbeddingGradLaunch p) {
  extern __shared__ __align__(16) uint32_t smem[];
  // The zeroing launch may start once every CTA has passed this wait: then the work before this launch is over,
  // and that is all it depends on.
  ptx::griddep_wait();
  ptx::griddep_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.crossing_count = 0;
  sort_tokens(p, smem);
}

// ---------------------------------------------------------------------------- 2. zeros

constexpr int kZeroThreads = 512;
constexpr int kZeroPer = 2;  // 16-byte stores of a thread
constexpr int64_t kZeroBlock = int64_t(kZeroThreads) * kZeroPer * 4;  // elements of a CTA

// One short CTA per 16 KB of the table. They start in the order of the addresses, so the stores in flight stay
// close together: 2.1 GB take 270 us (7.8 TB/s), against 312-323 us for CTAs that stay and walk over it.
__global__ void __launch_bounds__(kZeroThreads) embedding_zero_kernel(const EmbeddingGradLaunch p) {
  ptx::griddep_launch_dependents();
  if (p.direct) ptx::griddep_wait();  // no sort has waited for the work before
  // Rows that follow one another are one long row.
  const bool flat = p.ld_grad == p.dim;
  const int64_t len = flat ? p.rows * p.dim : p.dim;
  const int64_t blocks = (len + kZeroBlock - 1) / kZeroBlock;
  const int64_t begin = blockIdx.x % blocks * kZeroBlock, end = min(begin + kZeroBlock, len);
  float* dst = p.grad + blockIdx.x / blocks * p.ld_grad;
  if (p.vec_grad) {
#pragma unroll
    for (int k = 0; k < kZeroPer; ++k) {
      const int64_t c = begin + (k * kZeroThreads + threadIdx.x) * 4;
      if (c + 4 <= end)
        __stcs(reinterpret_cast<float4*>(dst + c), make_float4(0.f, 0.f, 0.f, 0.f));
      else
        for (int64_t e = c; e < end; ++e) dst[e] = 0.f;
    }
  } else {
    for (int64_t c = begin + threadIdx.x; c < end; c += kZeroThreads) __stcs(dst + c, 0.f);
  }
  // The next launch waits for this one, and may need the sort's result.
  ptx::griddep_wait();
}

// ---------------------------------------------------------------------------- few tokens

constexpr int kDirectTokens = kThreads;  // a thread looks at each
constexpr int kDirectCols = 2;           // of a thread, kThreads apart
constexpr int kDirectAhead = 16;         // rows loaded at a time

// A CTA per token and 512 columns. The first token of an id adds that id's rows, in the tokens' order; the others'
// CTAs end. Bound by latency: the ids, then its rows 16 at a time: 256 x 8000 fp32 into 2000 rows 26 us, 28 by the sort's
// way; 256 x 300 bf16 18, 22; at worst, 256 tokens all alike, 23, 22.
template <typename TG>
__global__ void __launch_bounds__(kThreads) embedding_direct_kernel(const EmbeddingGradLaunch p) {
  __shared__ unsigned same_of[kThreads / 32];
  __shared__ int list[kDirectTokens];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31, me = static_cast<int>(blockIdx.x);
  const uint32_t key = sort_key(p, me);
  const unsigned same = __ballot_sync(0xffffffffu, t < p.n && sort_key(p, t) == key);
  if (lane == 0) same_of[warp] = same;
  __syncthreads();
  if (key == static_cast<uint32_t>(p.rows)) return;
  int before = 0, count = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += __popc(same_of[w]);
    if (w == me / 32 && same_of[w] & ((1u << (me % 32)) - 1)) return;
    if (w < me / 32 && same_of[w]) return;
    count += __popc(same_of[w]);
  }
  if ((same >> lane) & 1u) list[before + __popc(same & ((1u << lane) - 1))] = t;
  __syncthreads();
  const int64_t col = static_cast<int64_t>(blockIdx.y) * (kThreads * kDirectCols) + t;
  const TG* src = static_cast<const TG*>(p.grad_out) + col;
  float acc[kDirectCols] = {};
  for (int i = 0; i < count; i += kDirectAhead) {
    TG v[kDirectAhead][kDirectCols];
#pragma unroll
    for (int a = 0; a < kDirectAhead; ++a)
#pragma unroll
      for (int k = 0; k < kDirectCols; ++k)
        v[a][k] = i + a < count && col + k * kThreads < p.dim ? __ldcs(src + list[i + a] * p.ld_grad_out + k * kThreads)
                                                              : row::from_f<TG>(0.f);
#pragma unroll
    for (int a = 0; a < kDirectAhead; ++a)
#pragma unroll
      for (int k = 0; k < kDirectCols; ++k) acc[k] += row::to_f(v[a][k]);
  }
  float* dst = p.grad + static_cast<int64_t>(key) * p.ld_grad + col;
#pragma unroll
  for (int k = 0; k < kDirectCols; ++k)
    if (col + k * kThreads < p.dim) {
      float* at = dst + k * kThreads;
      *at = fmaf(p.scale, acc[k], p.accumulate ? *at : 0.f);
    }
}

// ---------------------------------------------------------------------------- 3. sums by chunk

// A group of `tpr` threads adds the rows of one chunk over tpr * kCols consecutive columns, kAhead rows loaded at a
// time. With 16-byte rows (VEC) a thread holds consecutive columns, one 16-byte load of a row; otherwise a warp
// holds 32 * kCols consecutive columns and a thread every 32nd of them, so that a warp's loads lie side by side
// (20011 x 1027 fp32: 44 us; with a thread's columns consecutive 61).
template <typename TG, bool VEC>
struct Columns;

template <typename TG>
struct Columns<TG, true> {
  static constexpr int kCols = 16 / sizeof(TG), kAhead = 8;
  uint4 raw;
  // From this thread's first column on; `left` columns of the row lie there.
  __device__ __forceinline__ void load(const TG* src, int64_t) { raw = __ldcs(reinterpret_cast<const uint4*>(src)); }
  __device__ __forceinline__ void add_to(float (&acc)[kCols]) const {
    float v[kCols];
    row::unpack16<TG>(v, raw);
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] += v[k];
  }
};

template <typename TG>
struct Columns<TG, false> {
  static constexpr int kCols = 8, kAhead = 4;
  TG raw[kCols];
  __device__ __forceinline__ void load(const TG* src, int64_t left) {
    if (left > 32 * (kCols - 1)) {
#pragma unroll
      for (int k = 0; k < kCols; ++k) raw[k] = __ldcs(src + 32 * k);
    } else {
#pragma unroll
      for (int k = 0; k < kCols; ++k) raw[k] = 32 * k < left ? __ldcs(src + 32 * k) : row::from_f<TG>(0.f);
    }
  }
  __device__ __forceinline__ void add_to(float (&acc)[kCols]) const {
#pragma unroll
    for (int k = 0; k < kCols; ++k) acc[k] += row::to_f(raw[k]);
  }
};

// dst = scale * acc, or dst += scale * acc, from this thread's first column on.
template <bool VEC, int COLS>
__device__ __forceinline__ void store_columns(float* dst, const float (&acc)[COLS], float scale, bool add, int64_t left) {
  if constexpr (VEC) {
#pragma unroll
    for (int k = 0; k < COLS; k += 4) {
      float4* at = reinterpret_cast<float4*>(dst + k);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (add) o = *at;
      o.x = fmaf(scale, acc[k], o.x), o.y = fmaf(scale, acc[k + 1], o.y);
      o.z = fmaf(scale, acc[k + 2], o.z), o.w = fmaf(scale, acc[k + 3], o.w);
      __stcs(at, o);
    }
  } else {
#pragma unroll
    for (int k = 0; k < COLS; ++k)
      if (32 * k < left) dst[32 * k] = fmaf(scale, acc[k], add ? dst[32 * k] : 0.f);
  }
}

// Rows of this many chunks' heads or more are listed, to be joined by more threads: a warp of the short rows' adds
// them eight at a time, one after the other.
constexpr int kLongSpan = 32;

template <typename TG, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_chunk_kernel(const EmbeddingGradLaunch p) {
  using Cols = Columns<TG, VEC>;
  constexpr int COLS = Cols::kCols, kAhead = Cols::kAhead;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tpr = p.tpr, groups = blockDim.x / tpr;
  const int64_t chunk = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / tpr;
  if (chunk >= p.chunks) return;
  const int t = threadIdx.x % tpr;
  const int64_t col = static_cast<int64_t>(blockIdx.y) * tpr * COLS + (VEC ? t * COLS : t / 32 * 32 * COLS + t % 32);
  const int64_t left = p.dim - col;
  const bool active = left > 0;
  const bool first_slice = blockIdx.y == 0 && t == 0;
  const uint2* tokens = p.sorted[0];
  const int64_t begin = chunk * p.chunk_len, end = min(begin + p.chunk_len, p.n);
  const uint32_t none = static_cast<uint32_t>(p.rows);
  const TG* src = static_cast<const TG*>(p.grad_out) + col;
  // Tokens that add nothing sort behind every row; their rows are not read.
  uint2 tok[kAhead];
  auto fetch_tokens = [&](uint2 (&to)[kAhead], int64_t i) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) to[a] = i + a < end ? __ldcg(tokens + i + a) : make_uint2(none, 0);
  };
  fetch_tokens(tok, begin);
  const uint32_t key_before = begin > 0 ? __ldcg(&tokens[begin - 1].x) : none;
  const uint32_t key_after = end < p.n ? __ldcg(&tokens[end].x) : none;
  const int64_t far = (chunk + kLongSpan) * p.chunk_len;
  const uint32_t key_far = far < p.n ? __ldcg(&tokens[far].x) : none;
  uint32_t key = tok[0].x;
  bool from_before = key == key_before && key != none;
  // Bit 0: the chunk begins inside a row; bit 1: that row also fills the chunk and goes on.
  if (first_slice) p.chunk_state[chunk] = (from_before ? 1 : 0) | (from_before && key == key_after ? 2 : 0);
  float acc[COLS];
#pragma unroll
  for (int k = 0; k < COLS; ++k) acc[k] = 0.f;
  auto flush = [&](bool goes_on) {
    if (from_before || goes_on) {
      // Head sums lie in the even rows of the workspace, tail sums in the odd ones.
      float* part = p.partials + (chunk * 2 + (from_before ? 0 : 1)) * p.ld_partials;
      if (active) store_columns<VEC>(part + col, acc, 1.f, false, left);
      if (!from_before && key == key_far && first_slice) {
        const unsigned at = atomicAdd(p.crossing_count, 1u);
        if (dev_check(at < p.chunks, p.status)) p.crossing[at] = make_uint2(static_cast<uint32_t>(chunk), key);
      }
    } else if (active) {
      store_columns<VEC>(p.grad + static_cast<int64_t>(key) * p.ld_grad + col, acc, p.scale, p.accumulate != 0, left);
    }
  };
  // A chunk's length is a multiple of kAhead: only the list's last chunk has places without tokens.
  for (int64_t i = begin; i < end && key != none; i += kAhead) {
    Cols val[kAhead];
    uint2 next[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (active && tok[a].x != none) val[a].load(src + tok[a].y * p.ld_grad_out, left);
    fetch_tokens(next, i + kAhead);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (tok[a].x != key) {
        if (key != none) flush(false);
        key = tok[a].x;
        from_before = false;
#pragma unroll
        for (int k = 0; k < COLS; ++k) acc[k] = 0.f;
      }
      if (key != none) val[a].add_to(acc);
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) tok[a] = next[a];
  }
  if (key != none) flush(key == key_after);
}

// ---------------------------------------------------------------------------- 4. rows across chunks

constexpr int kJoinWarps = kThreads / 32;
constexpr int kJoinCols = 128;  // columns of a warp, four per lane
constexpr int kLongCtas = 304;  // that join listed rows, beside those that look at the chunks

__device__ __forceinline__ void add4(float4& a, const float4& b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }

// Adds the heads of chunks [lo, hi) at a column.
__device__ __forceinline__ void add_heads(float4& acc, const EmbeddingGradLaunch& p, int64_t lo, int64_t hi, int64_t col) {
  const float* part = p.partials + col;
  int64_t c = lo;
  for (; c + 8 <= hi; c += 8) {
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __ldcg(reinterpret_cast<const float4*>(part + (c + k) * 2 * p.ld_partials));
#pragma unroll
    for (int k = 0; k < 8; ++k) add4(acc, v[k]);
  }
  for (; c < hi; ++c) add4(acc, __ldcg(reinterpret_cast<const float4*>(part + c * 2 * p.ld_partials)));
}

__device__ __forceinline__ void store_joined(const EmbeddingGradLaunch& p, uint32_t key, int64_t col, const float4& acc) {
  float* dst = p.grad + static_cast<int64_t>(key) * p.ld_grad + col;
  const float v[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (col + k < p.dim) dst[k] = fmaf(p.scale, v[k], p.accumulate ? dst[k] : 0.f);
}

// The last chunk that the row which `first` leaves open reaches into: the first one behind it that the row does
// not fill. Called by whole warps.
__device__ __forceinline__ int64_t last_chunk(const EmbeddingGradLaunch& p, int64_t first) {
  const int lane = threadIdx.x & 31;
  for (int64_t last = first;; last += 32) {
    const int64_t c = last + 1 + lane;
    const unsigned ends = __ballot_sync(0xffffffffu, c >= p.chunks || __ldcg(p.chunk_state + c) != 3);
    if (ends) {
      const int64_t stop = last + __ffs(ends);
      return stop < p.chunks && (__ldcg(p.chunk_state + stop) & 1) ? stop : stop - 1;
    }
  }
}

// The first CTAs take the chunks, p.join_warps warps for each: where a chunk leaves a row open that it does not
// begin inside of, they add the row's heads to its tail, a warp for 128 columns at a time. The last kLongCtas
// take the listed rows, 128 columns of one at a time, the heads split over the CTA's warps.
__global__ void __launch_bounds__(kThreads) embedding_join_kernel(const EmbeddingGradLaunch p) {
  __shared__ float4 sums[kJoinWarps][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t per_cta = kJoinWarps / p.join_warps, short_ctas = (p.chunks + per_cta - 1) / per_cta;
  if (blockIdx.x < short_ctas) {
    const int64_t c = blockIdx.x * per_cta + warp / p.join_warps;
    if (c + 1 >= p.chunks) return;
    const int here = __ldcg(p.chunk_state + c), next = __ldcg(p.chunk_state + c + 1);
    const uint32_t key = __ldcg(&p.sorted[0][(c + 1) * p.chunk_len].x);
    if (!(next & 1) || here == 3) return;
    const int64_t last = last_chunk(p, c);
    if (last - c >= kLongSpan) return;
    const float* tail = p.partials + (c * 2 + 1) * p.ld_partials;
    for (int64_t col = (warp % p.join_warps) * kJoinCols + lane * 4; col < p.dim; col += p.join_warps * kJoinCols) {
      float4 acc = __ldcg(reinterpret_cast<const float4*>(tail + col));
      add_heads(acc, p, c + 1, last + 1, col);
      store_joined(p, key, col, acc);
    }
    return;
  }
  const int64_t blocks = (p.dim + kJoinCols - 1) / kJoinCols;
  const int64_t items = static_cast<int64_t>(__ldcg(p.crossing_count)) * blocks;
  for (int64_t item = blockIdx.x - short_ctas; item < items; item += kLongCtas) {
    const uint2 row = p.crossing[item / blocks];
    const int64_t first = row.x, col = item % blocks * kJoinCols + lane * 4, span = last_chunk(p, first) - first;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < p.dim) {
      if (warp == 0) acc = __ldcg(reinterpret_cast<const float4*>(p.partials + (first * 2 + 1) * p.ld_partials + col));
      add_heads(acc, p, first + 1 + span * warp / kJoinWarps, first + 1 + span * (warp + 1) / kJoinWarps, col);
    }
    sums[warp][lane] = acc;
    __syncthreads();
    if (warp == 0 && col < p.dim) {
      for (int w = 1; w < kJoinWarps; ++w) add4(acc, sums[w][lane]);
      store_joined(p, row.y, col, acc);
    }
    __syncthreads();
  }
}

template <typename TG, bool VEC>
cudaError_t launch_chunks(const EmbeddingGradLaunch& p, cudaStream_t stream) {
  const int64_t slice = int64_t(p.tpr) * Columns<TG, VEC>::kCols, groups = kThreads / p.tpr;
  const dim3 grid(static_cast<unsigned>((p.chunks + groups - 1) / groups),
                  static_cast<unsigned>((p.dim + slice - 1) / slice));
  return row::launch(embedding_chunk_kernel<TG, VEC>, grid, static_cast<int>(groups * p.tpr), 0, stream, p);
}

bool aligned16(const void* p, int64_t ld, size_t elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && static_cast<size_t>(ld) * elem % 16 == 0;
}

// How the sums by chunk are split: threads per row, and tokens per chunk. Short chunks spread few tokens over
// many SMs; long ones leave fewer sums in the workspace (a chunk writes two fp32 rows of them at worst). So
// chunks are 16 tokens long, and longer once that still leaves a CTA for each of 1024 places (about 7 per SM). A
// slice of the columns is a CTA's at most, and all slices are alike: 1027 fp32 columns, off 16 bytes, are one of 160
// threads.
void split_tokens(EmbeddingGradLaunch& p) {
  const int cols = p.vec ? (p.grad_dtype == 1 ? Columns<__nv_bfloat16, true>::kCols : Columns<float, true>::kCols)
                         : Columns<float, false>::kCols;
  // Slices of equal length: whole warps, or with VEC a power of two of threads below one.
  const int64_t slices = (p.dim + kThreads * cols - 1) / (kThreads * cols);
  const int need = static_cast<int>(((p.dim + slices - 1) / slices + cols - 1) / cols);
  p.tpr = (need + 31) / 32 * 32;
  if (p.vec && need <= 16)
    for (p.tpr = 1; p.tpr < need;) p.tpr *= 2;
  const int64_t groups = kThreads / p.tpr;
  p.chunk_len = 16;
  while (p.n / (2 * p.chunk_len) * slices >= 1024 * groups) p.chunk_len *= 2;
  p.chunks = (p.n + p.chunk_len - 1) / p.chunk_len;
}

int64_t padded(int64_t bytes) { return (bytes + 255) / 256 * 256; }

}  // namespace

cudaError_t launch_embedding(EmbeddingLaunch& p, cudaStream_t stream) {
  const size_t ti = p.table_dtype == 0 ? 4 : 2, to = p.out_dtype == 0 ? 4 : 2;
  const bool vec = p.dim % kLookup == 0 && aligned16(p.table, p.ld_table, ti) && aligned16(p.out, p.ld_out, to);
  const int each = vec ? kLookup : static_cast<int>(16 / to);
  p.tpr = vec ? 1 : 16;
  while (p.tpr < kThreads && p.tpr * each < p.dim) p.tpr *= 2;
  const int64_t tokens = kThreads / p.tpr * 2;  // of a CTA
  const dim3 grid(static_cast<unsigned>((p.n + tokens - 1) / tokens));
  auto run = [&](auto kernel) { return row::launch(kernel, grid, kThreads, 0, stream, const_cast<const EmbeddingLaunch&>(p)); };
  using B = __nv_bfloat16;
  if (p.table_dtype == 0 && p.out_dtype == 0) return run(vec ? embedding_kernel<float, float> : embedding_shift_kernel<float, float>);
  if (p.table_dtype == 0) return run(vec ? embedding_kernel<float, B> : embedding_shift_kernel<float, B>);
  if (p.out_dtype == 0) return run(vec ? embedding_kernel<B, float> : embedding_shift_kernel<B, float>);
  return run(vec ? embedding_kernel<B, B> : embedding_shift_kernel<B, B>);
}

int64_t embedding_grad_workspace(EmbeddingGradLaunch& p, char* ws) {
  p.vec_grad = aligned16(p.grad, p.ld_grad, sizeof(float));
  p.direct = p.n <= kDirectTokens;
  if (p.direct) return 0;
  p.vec = p.vec_grad && p.dim % (p.grad_dtype == 1 ? 8 : 4) == 0 &&
          aligned16(p.grad_out, p.ld_grad_out, p.grad_dtype == 1 ? 2 : 4);
  split_tokens(p);
  p.ld_partials = (p.dim + 3) / 4 * 4;
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    char* at = ws ? ws + off : nullptr;
    off += padded(bytes);
    return at;
  };
  p.crossing_count = reinterpret_cast<unsigned*>(take(sizeof(unsigned)));
  for (auto& s : p.sorted) s = reinterpret_cast<uint2*>(take(p.n * static_cast<int64_t>(sizeof(uint2))));
  p.crossing = reinterpret_cast<uint2*>(take(p.chunks * static_cast<int64_t>(sizeof(uint2))));
  p.chunk_state = reinterpret_cast<int*>(take(p.chunks * static_cast<int64_t>(sizeof(int))));
  p.partials = reinterpret_cast<float*>(take(p.chunks * 2 * p.ld_partials * static_cast<int64_t>(sizeof(float))));
  return off;
}

cudaError_t launch_embedding_zeros(const EmbeddingGradLaunch& p, cudaStream_t stream) {
  const bool flat = p.ld_grad == p.dim;
  const int64_t len = flat ? p.rows * p.dim : p.dim;
  const int64_t blocks = (len + kZeroBlock - 1) / kZeroBlock * (flat ? 1 : p.rows);
  if (blocks >= int64_t(1) << 31) return cudaErrorInvalidConfiguration;
  return row::launch(embedding_zero_kernel, dim3(static_cast<unsigned>(blocks)), kZeroThreads, 0, stream, p);
}

cudaError_t launch_embedding_grad(EmbeddingGradLaunch& p, int sms, cudaStream_t stream) {
  if (p.direct) {
    const cudaError_t e = p.accumulate ? cudaSuccess : launch_embedding_zeros(p, stream);
    if (e != cudaSuccess || p.n == 0) return e;
    constexpr int64_t slice = kThreads * kDirectCols;
    const dim3 grid(static_cast<unsigned>(p.n), static_cast<unsigned>((p.dim + slice - 1) / slice));
    return row::launch(p.grad_dtype == 0 ? embedding_direct_kernel<float> : embedding_direct_kernel<__nv_bfloat16>, grid,
                       kThreads, 0, stream, const_cast<const EmbeddingGradLaunch&>(p));
  }
  int bits = 1;
  while ((int64_t(1) << bits) <= p.rows) ++bits;  // keys go up to `rows`
  p.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  cudaError_t e = cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSortSmem));
  if (e != cudaSuccess) return e;
  e = row::launch(embedding_sort_kernel, dim3(kSortCtas), kSortThreads, kSortSmem, stream, p);
  if (e != cudaSuccess) return e;
  if (!p.accumulate) e = launch_embedding_zeros(p, stream);
  if (e != cudaSuccess) return e;
  if (p.grad_dtype == 0)
    e = p.vec ? launch_chunks<float, true>(p, stream) : launch_chunks<float, false>(p, stream);
  else
    e = p.vec ? launch_chunks<__nv_bfloat16, true>(p, stream) : launch_chunks<__nv_bfloat16, false>(p, stream);
  if (e != cudaSuccess) return e;
  p.join_warps = 1;
  while (p.join_warps < kJoinWarps && p.join_warps * kJoinCols < p.dim) p.join_warps *= 2;
  const int64_t per_cta = kJoinWarps / p.join_warps;
  const int64_t ctas = (p.chunks + per_cta - 1) / per_cta + (p.chunks > kLongSpan ? kLongCtas : 0);
  return row::launch(embedding_join_kernel, dim3(static_cast<unsigned>(ctas)), kThreads, 0, stream, p);
}

}  // namespace dmuon
