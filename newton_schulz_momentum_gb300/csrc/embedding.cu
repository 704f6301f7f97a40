// Embedding lookup with scaling, out[i, :] = scale * table[id_i, :], and its gradient,
// grad[v, :] = scale * sum over the tokens i with id_i = v of grad_out[i, :], added in the order of i.
//
// The gradient takes four launches:
//   1. one cluster sorts the tokens by id (stable);
//   2. meanwhile, on the other SMs, the table rows that no token falls on are written with zeros, which at a
//      language model's sizes is most of the bytes (not run where the caller adds to the gradient);
//   3. the sorted list is cut into chunks of equal length, whatever the ids' frequencies: a CTA adds a
//      chunk's rows and writes each table row that begins and ends inside it; a row that crosses a chunk's
//      border leaves its sum over the chunk in the workspace;
//   4. the rows that cross borders are put together from their chunks' sums, in order.
#include <algorithm>

#include "row_ops.h"
#include "tc_ptx.h"

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

// ---------------------------------------------------------------------------- 1. sort

constexpr int kSortCtas = 8;  // one portable cluster
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr size_t kSortSmem = sizeof(uint32_t) * (kSortWarps + 2) * kMaxDigits;

// Token i's sort key: its id, or `rows` (behind every row) for padding and ids outside the table.
__device__ __forceinline__ uint32_t sort_key(const EmbeddingGradLaunch& p, int64_t i) {
  const int64_t id = row::load_id(p.ids, p.id_bytes, i);
  return id >= 0 && id < p.rows && id != p.padding_idx ? static_cast<uint32_t>(id) : static_cast<uint32_t>(p.rows);
}

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Radix sort of the tokens, least significant digit first, by the CTAs of one cluster. Every warp holds a
// run of consecutive tokens; a token's place is the number of tokens with a smaller digit, plus those with
// the same digit in earlier CTAs, earlier warps and earlier in its warp, so equal ids keep their order.
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
    for (int64_t s = 0; s < steps; ++s) {
      const int64_t i = first + s * 32 + lane;
      const uint32_t d = i < p.n ? (token(i).x >> shift) & (digits - 1) : 0xffffffffu;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (d != 0xffffffffu && lane == __ffs(same) - 1) mine[d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    if (threadIdx.x < digits) {
      uint32_t sum = 0;
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = count[w * kMaxDigits + threadIdx.x];
        count[w * kMaxDigits + threadIdx.x] = sum;
        sum += c;
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
    for (int64_t s = 0; s < steps; ++s) {
      const int64_t i = first + s * 32 + lane;
      const uint2 t = token(i);
      const uint32_t d = i < p.n ? (t.x >> shift) & (digits - 1) : 0xffffffffu;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (d != 0xffffffffu) {
        const uint32_t at = base[d] + mine[d] + __popc(same & ((1u << lane) - 1));
        if (dev_check(at < p.n, p.status)) __stcg(out + at, t);
      }
      __syncwarp();
      if (d != 0xffffffffu && lane == __ffs(same) - 1) mine[d] += __popc(same);
      __syncwarp();
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
  for (int64_t i = blockIdx.x * kSortThreads + threadIdx.x; i < p.n; i += kSortCtas * kSortThreads) {
    const int64_t id = row::load_id(p.ids, p.id_bytes, i);
    if (id < 0 || id >= p.rows) atomicOr(p.status, kDevIndex);
  }
  sort_tokens(p, smem);
}

// ---------------------------------------------------------------------------- 2. rows without tokens

constexpr int kZeroThreads = 512;
constexpr int kMarkWords = 8192;  // a CTA marks the rows with tokens in a bitmap over 2^18 of its rows at a time

__global__ void __launch_bounds__(kZeroThreads) embedding_zero_kernel(const EmbeddingGradLaunch p) {
  __shared__ uint32_t marks[kMarkWords];
  ptx::griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t begin = p.rows * blockIdx.x / gridDim.x, end = p.rows * (blockIdx.x + 1) / gridDim.x;
  for (int64_t r0 = begin; r0 < end; r0 += kMarkWords * 32) {
    const int here = static_cast<int>(min(static_cast<int64_t>(kMarkWords) * 32, end - r0));
    for (int k = threadIdx.x; k < (here + 31) / 32; k += kZeroThreads) marks[k] = 0;
    __syncthreads();
    for (int64_t i = threadIdx.x; i < p.n; i += kZeroThreads) {
      const int64_t at = static_cast<int64_t>(sort_key(p, i)) - r0;
      if (at >= 0 && at < here) atomicOr(marks + (at >> 5), 1u << (at & 31));
    }
    __syncthreads();
    for (int r = warp; r < here; r += kZeroThreads / 32) {
      if (marks[r >> 5] >> (r & 31) & 1) continue;
      float* dst = p.grad + (r0 + r) * p.ld_grad;
      int64_t c = lane;
      if (p.vec_grad) {
        float4* dst4 = reinterpret_cast<float4*>(dst);
        for (; c < p.dim / 4; c += 32) __stcs(dst4 + c, make_float4(0.f, 0.f, 0.f, 0.f));
        c = p.dim / 4 * 4 + lane;
      }
      for (; c < p.dim; c += 32) __stcs(dst + c, 0.f);
    }
    __syncthreads();
  }
  // The next launch waits for this one, and needs the sort's result.
  ptx::griddep_wait();
}

// ---------------------------------------------------------------------------- 3. sums by chunk

// A group of `tpr` threads adds the rows of one chunk over tpr * COLS consecutive columns.
// VEC: a thread's COLS columns are one 16-byte load; otherwise they lie tpr apart.
template <typename TG, bool VEC>
struct ChunkColumns {
  static constexpr int kCols = VEC ? 16 / sizeof(TG) : 4;
};

template <typename TG, bool VEC, int COLS>
__device__ __forceinline__ void load_columns(float (&v)[COLS], const TG* src, int64_t col, int tpr, int64_t dim) {
  if constexpr (VEC) {
    row::load16(v, src + col);
  } else {
#pragma unroll
    for (int k = 0; k < COLS; ++k) v[k] = col + k * tpr < dim ? row::to_f(__ldcs(src + col + k * tpr)) : 0.f;
  }
}

// dst = scale * acc, or dst += scale * acc.
template <bool VEC, int COLS>
__device__ __forceinline__ void store_columns(float* dst, const float (&acc)[COLS], float scale, bool add, int64_t col,
                                              int tpr, int64_t dim) {
  if constexpr (VEC) {
#pragma unroll
    for (int k = 0; k < COLS; k += 4) {
      float4* at = reinterpret_cast<float4*>(dst + col + k);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
      if (add) o = *at;
      o.x = fmaf(scale, acc[k], o.x), o.y = fmaf(scale, acc[k + 1], o.y);
      o.z = fmaf(scale, acc[k + 2], o.z), o.w = fmaf(scale, acc[k + 3], o.w);
      __stcs(at, o);
    }
  } else {
#pragma unroll
    for (int k = 0; k < COLS; ++k)
      if (col + k * tpr < dim) {
        float* at = dst + col + k * tpr;
        *at = fmaf(scale, acc[k], add ? *at : 0.f);
      }
  }
}

constexpr int kAhead = 4;  // rows in flight per thread

template <typename TG, bool VEC>
__global__ void __launch_bounds__(kThreads) embedding_chunk_kernel(const EmbeddingGradLaunch p) {
  constexpr int COLS = ChunkColumns<TG, VEC>::kCols;
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int tpr = p.tpr, groups = kThreads / tpr;
  const int64_t chunk = static_cast<int64_t>(blockIdx.x) * groups + threadIdx.x / tpr;
  if (chunk >= p.chunks) return;
  const int t = threadIdx.x % tpr;
  const int64_t col = static_cast<int64_t>(blockIdx.y) * tpr * COLS + (VEC ? t * COLS : t);
  const bool first_slice = blockIdx.y == 0 && t == 0;
  const uint2* tokens = p.sorted[0];
  const int64_t begin = chunk * p.chunk_len, end = min(begin + p.chunk_len, p.n);
  const uint32_t none = static_cast<uint32_t>(p.rows);
  const uint32_t key_before = begin > 0 ? __ldcg(&tokens[begin - 1].x) : none;
  const uint32_t key_after = end < p.n ? __ldcg(&tokens[end].x) : none;
  uint32_t key = __ldcg(&tokens[begin].x);
  const bool head_comes_in = key == key_before && key != none;
  // Bit 0: the chunk begins inside a row; bit 1: that row also fills the chunk and goes on.
  if (first_slice) {
    const bool through = head_comes_in && key == key_after;
    p.chunk_state[chunk] = (head_comes_in ? 1 : 0) | (through ? 2 : 0);
  }
  if (key == none) return;  // padding sorts behind every row
  const TG* src = static_cast<const TG*>(p.grad_out);
  const bool active = col < p.dim;
  float acc[COLS];
#pragma unroll
  for (int k = 0; k < COLS; ++k) acc[k] = 0.f;
  bool from_before = head_comes_in;
  auto flush = [&](bool goes_on) {
    if (from_before || goes_on) {
      // Head sums lie in the even slots of the workspace, tail sums in the odd ones.
      float* part = p.partials + (chunk * 2 + (from_before ? 0 : 1)) * p.ld_partials;
      if (active) store_columns<VEC>(part, acc, 1.f, false, col, tpr, p.dim);
      if (!from_before && first_slice) {
        const unsigned at = atomicAdd(p.crossing_count, 1u);
        if (dev_check(at < p.chunks, p.status)) p.crossing[at] = make_uint2(static_cast<uint32_t>(chunk), key);
      }
    } else if (active) {
      store_columns<VEC>(p.grad + static_cast<int64_t>(key) * p.ld_grad, acc, p.scale, p.accumulate != 0, col, tpr, p.dim);
    }
  };
  for (int64_t i = begin; i < end; i += kAhead) {
    uint2 tok[kAhead];
    float v[kAhead][COLS];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) tok[a] = i + a < end ? __ldcg(tokens + i + a) : make_uint2(none, 0);
#pragma unroll
    for (int a = 0; a < kAhead; ++a)
      if (active && tok[a].x != none) load_columns<TG, VEC>(v[a], src + tok[a].y * p.ld_grad_out, col, tpr, p.dim);
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (tok[a].x == none) {
        if (key != none) flush(false);
        key = none;
        continue;
      }
      if (tok[a].x != key) {
        flush(false);
        key = tok[a].x;
        from_before = false;
#pragma unroll
        for (int k = 0; k < COLS; ++k) acc[k] = 0.f;
      }
      if (active) {
#pragma unroll
        for (int k = 0; k < COLS; ++k) acc[k] += v[a][k];
      }
    }
    if (key == none) return;
  }
  flush(key == key_after);
}

// ---------------------------------------------------------------------------- 4. rows across chunks

constexpr int kJoinCols = 64;                       // columns of a CTA, one per thread of a group
constexpr int kJoinGroups = kThreads / kJoinCols;   // a row's chunks are split over the groups

__global__ void __launch_bounds__(kThreads) embedding_join_kernel(const EmbeddingGradLaunch p) {
  __shared__ float sums[kJoinGroups][kJoinCols];
  ptx::griddep_wait();
  const int lane = threadIdx.x & 31, group = threadIdx.x / kJoinCols, t = threadIdx.x % kJoinCols;
  const int64_t slices = (p.dim + kJoinCols - 1) / kJoinCols;
  const int64_t items = static_cast<int64_t>(*p.crossing_count) * slices;
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const uint2 row = p.crossing[item / slices];
    const int64_t col = item % slices * kJoinCols + t;
    // The last chunk that the row reaches into: the first one behind row.x that it does not fill.
    int64_t last = row.x;
    for (;;) {
      const int64_t c = last + 1 + lane;
      const unsigned ends = __ballot_sync(0xffffffffu, c >= p.chunks || p.chunk_state[c] != 3);
      if (ends) {
        const int64_t stop = last + __ffs(ends);
        last = stop < p.chunks && (p.chunk_state[stop] & 1) ? stop : stop - 1;
        break;
      }
      last += 32;
    }
    const int64_t span = last - row.x;  // heads to add
    const int64_t lo = row.x + 1 + span * group / kJoinGroups, hi = row.x + 1 + span * (group + 1) / kJoinGroups;
    float acc = 0.f;
    if (col < p.dim) {
      const float* part = p.partials + col;
      if (group == 0) acc = __ldcg(part + (static_cast<int64_t>(row.x) * 2 + 1) * p.ld_partials);
      int64_t c = lo;
      for (; c + 8 <= hi; c += 8) {
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = __ldcg(part + (c + k) * 2 * p.ld_partials);
#pragma unroll
        for (int k = 0; k < 8; ++k) acc += v[k];
      }
      for (; c < hi; ++c) acc += __ldcg(part + c * 2 * p.ld_partials);
    }
    sums[group][t] = acc;
    __syncthreads();
    if (group == 0 && col < p.dim) {
#pragma unroll
      for (int g = 1; g < kJoinGroups; ++g) acc += sums[g][t];
      float* dst = p.grad + static_cast<int64_t>(row.y) * p.ld_grad + col;
      *dst = fmaf(p.scale, acc, p.accumulate ? *dst : 0.f);
    }
    __syncthreads();
  }
}

template <typename TG, bool VEC>
cudaError_t launch_chunks(EmbeddingGradLaunch& p, cudaStream_t stream) {
  constexpr int COLS = ChunkColumns<TG, VEC>::kCols;
  p.tpr = 1;
  while (p.tpr < kThreads && p.tpr * COLS < p.dim) p.tpr *= 2;
  const int groups = kThreads / p.tpr;
  const dim3 grid(static_cast<unsigned>((p.chunks + groups - 1) / groups),
                  static_cast<unsigned>((p.dim + p.tpr * COLS - 1) / (p.tpr * COLS)));
  return row::launch(embedding_chunk_kernel<TG, VEC>, grid, kThreads, 0, stream, p);
}

bool aligned16(const void* p, int64_t ld, size_t elem) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && static_cast<size_t>(ld) * elem % 16 == 0;
}

// Tokens per chunk: at least 16, so that the sums over chunks stay well under the tokens' own rows (two fp32
// rows of sums for 16 rows read, at worst), and about a thousand chunks from there on.
int64_t chunk_length(int64_t n) {
  int64_t len = 16;
  while (len * 1024 < n) len *= 2;
  return len;
}

int64_t padded(int64_t bytes) { return (bytes + 255) / 256 * 256; }

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

int64_t embedding_grad_workspace(EmbeddingGradLaunch& p, char* ws) {
  p.chunk_len = chunk_length(p.n);
  p.chunks = (p.n + p.chunk_len - 1) / p.chunk_len;
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

cudaError_t launch_embedding_grad(EmbeddingGradLaunch& p, int sms, cudaStream_t stream) {
  int bits = 1;
  while ((int64_t(1) << bits) <= p.rows) ++bits;  // keys go up to `rows`
  p.passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
  p.digit_bits = (bits + p.passes - 1) / p.passes;
  p.vec_grad = aligned16(p.grad, p.ld_grad, sizeof(float));
  const bool vec = p.vec_grad && p.dim % (p.grad_dtype == 1 ? 8 : 4) == 0 &&
                   aligned16(p.grad_out, p.ld_grad_out, p.grad_dtype == 1 ? 2 : 4);
  cudaError_t e = cudaFuncSetAttribute(embedding_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSortSmem));
  if (e != cudaSuccess) return e;
  e = row::launch(embedding_sort_kernel, dim3(kSortCtas), kSortThreads, kSortSmem, stream, p);
  if (e != cudaSuccess) return e;
  if (!p.accumulate) e = row::launch(embedding_zero_kernel, dim3(2 * sms), kZeroThreads, 0, stream, p);
  if (e != cudaSuccess || p.n == 0) return e;
  if (p.grad_dtype == 0)
    e = vec ? launch_chunks<float, true>(p, stream) : launch_chunks<float, false>(p, stream);
  else
    e = vec ? launch_chunks<__nv_bfloat16, true>(p, stream) : launch_chunks<__nv_bfloat16, false>(p, stream);
  if (e != cudaSuccess) return e;
  const int64_t items = p.chunks * ((p.dim + kJoinCols - 1) / kJoinCols);
  return row::launch(embedding_join_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(items, 4 * sms))), kThreads, 0,
                     stream, p);
}

}  // namespace dmuon
