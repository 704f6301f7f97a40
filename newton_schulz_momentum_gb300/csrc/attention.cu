// Attention over whole prompts, sequences packed one behind the other, query heads in groups that share a key head; and
// its backward pass.
//
// Per sequence and query head, over the keys j of the same sequence (j <= i if causal): x_ij = scale q_i . k_j,
// p = softmax of a row of x, o_i = sum p_ij v_j, lse_i = log sum exp x_ij. Backward, with D_i = do_i . o_i:
//   dv_j = sum p_ij do_i,  ds_ij = p_ij (do_i . v_j - D_i),  dq_i = scale sum ds_ij k_j,  dk_j = scale sum ds_ij q_i,
// the last two of a key head over all of its query heads.
//
// Forward. A unit is 128 consecutive queries of one head. A CTA takes two units of a key head's group, whose keys and
// values (tiles of 128) come by tensor-map copies into a ring of four slots. Scores and outputs of both units lie in
// tensor memory (fp32, 512 columns); four warps per unit turn scores into probabilities, one row a thread, written
// back as bf16 over the scores they come from, the left operand of the product with the values. While one unit's warps
// form probabilities the tensor cores multiply for the other. The running maximum that probabilities are taken from is
// raised (and sums and outputs scaled down) only where a row's maximum has grown by more than 2^8 beyond it: results do
// not change but for rounding, fp32 sums and bf16 probabilities being floating point.
#include <algorithm>
#include <cstring>

#include "row_ops.h"
#include "tc_ptx.h"

namespace dmuon {
namespace {

using namespace ptx;
using bf16 = __nv_bfloat16;

constexpr int kTile = 128;           // queries of a unit, keys of a tile
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;        // how far (log2) a row's maximum may grow beyond the one in use

__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 c;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(c))
      : "l"(reinterpret_cast<const unsigned long long&>(a)), "l"(reinterpret_cast<const unsigned long long&>(b)));
  return c;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------------------- sequences

// Sequence s, [*begin, *begin + length); an empty one where the offsets are not in order or leave the arrays.
__device__ __forceinline__ int64_t sequence_length(const AttentionLaunch& p, int64_t s, int64_t* begin) {
  if (!p.offsets) {
    const int64_t len = p.n / p.sequences;
    *begin = s * len;
    return len;
  }
  const int64_t b = row::load_id(p.offsets, p.id_bytes, s), e = row::load_id(p.offsets, p.id_bytes, s + 1);
  *begin = b;
  if (b < 0 || e > p.n || e < b) {
    atomicOr(p.status, kDevIndex);
    return 0;
  }
  return e - b;
}

// A CTA's place: the `slot`-th of the pieces that all sequences are cut into (`per`(length) of each).
struct Place {
  int64_t begin, length, piece;  // length 0: there are fewer pieces
};

// By one warp. Without offsets the sequences are equal; otherwise 32 of them at a time.
template <typename F>
__device__ __forceinline__ Place find_place(const AttentionLaunch& p, int64_t slot, F&& per) {
  const int lane = threadIdx.x & 31;
  Place at{0, 0, 0};
  if (!p.offsets) {
    const int64_t len = p.n / p.sequences, pieces = per(len), s = slot / pieces;
    if (s < p.sequences) at = {s * len, len, slot - s * pieces};
    return at;
  }
  for (int64_t s0 = 0; s0 < p.sequences; s0 += 32) {
    int64_t begin = 0;
    const int64_t len = s0 + lane < p.sequences ? sequence_length(p, s0 + lane, &begin) : 0;
    const int64_t pieces = len > 0 ? per(len) : 0;
    int64_t sum = pieces;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t left = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += left;
    }
    const unsigned behind = __ballot_sync(0xffffffffu, slot < sum);
    if (behind) {
      const int l = __ffs(behind) - 1;
      at.begin = __shfl_sync(0xffffffffu, begin, l);
      at.length = __shfl_sync(0xffffffffu, len, l);
      at.piece = slot - __shfl_sync(0xffffffffu, sum - pieces, l);
      return at;
    }
    slot -= __shfl_sync(0xffffffffu, sum, 31);
  }
  return at;
}

__device__ __forceinline__ const bf16* at(const HeadArray& a, int64_t token, int64_t head) {
  return static_cast<const bf16*>(a.data) + token * a.token + head * a.head;
}
__device__ __forceinline__ bf16* out_at(const HeadArray& a, int64_t token, int64_t head) {
  return static_cast<bf16*>(const_cast<void*>(a.data)) + token * a.token + head * a.head;
}

// Zeros in the rows of tokens that belong to no sequence, spread over the grid's CTAs and their threads.
__device__ __forceinline__ void zero_rows_outside(const AttentionLaunch& p, const HeadArray& a, int heads, float* lse) {
  if (!p.offsets || !p.zero_outside) return;
  const int64_t first = row::load_id(p.offsets, p.id_bytes, 0), last = row::load_id(p.offsets, p.id_bytes, p.sequences);
  const int64_t before = first < 0 ? 0 : first > p.n ? p.n : first, from = last < before ? before : last > p.n ? p.n : last;
  const int64_t rows = (before + p.n - from) * heads;
  const int64_t thread = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t r = thread; r < rows; r += static_cast<int64_t>(gridDim.x) * gridDim.y * blockDim.x) {
    const int64_t k = r / heads, head = r - k * heads, token = k < before ? k : from + (k - before);
    bf16* x = out_at(a, token, head);
    for (int c = 0; c < p.dim; c += 8) *reinterpret_cast<uint4*>(x + c) = make_uint4(0, 0, 0, 0);
    if (lse) lse[head * p.n + token] = 0.f;
  }
}

// ---------------------------------------------------------------------------- forward

// kD: columns of a head, padded with zeros to 64 or 128.
template <int kD>
struct Fwd {
  static constexpr int kSlots = 4;
  static constexpr int kTileBytes = kTile * kD * 2;
  static constexpr int kBoxes = kD / 64, kBoxBytes = kTile * 128;
  static constexpr int kThreads = 320;  // warps 0-3 and 4-7: a unit's rows each; 8: copies; 9: products
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + 1024 + 256;
  static constexpr uint32_t kCols = 512;
  static constexpr uint32_t kScores = 0, kOut = 256;  // of the first unit; the second's are kTile columns behind
};

// How many tiles of keys the unit's rows meet, and where the unit lies.
struct Unit {
  int head, tiles;
  int64_t row;  // first row within the sequence
};

__device__ __forceinline__ Unit unit_at(const AttentionLaunch& p, int64_t length, int64_t unit, int kv) {
  const int group = p.heads / p.kv_heads;
  const int64_t blocks = (length + kTile - 1) / kTile, back = unit / group, block = blocks - 1 - back;
  if (block < 0) return {0, 0, 0};
  return {static_cast<int>(kv * group + unit - back * group), static_cast<int>(p.causal ? block + 1 : blocks), block * kTile};
}

// Scores of one row times log2(e) |scale|, made probabilities; see softmax_rows.
template <int kD>
__device__ __forceinline__ void scale_outputs(uint32_t tmem_out, float f) {
#pragma unroll
  for (int c = 0; c < kD; c += 32) {
    uint32_t r[32];
    tmem_ld32_issue(tmem_out + c, r);
    tmem_ld_wait(r);
#pragma unroll
    for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * f);
    tmem_st32(tmem_out + c, r);
  }
  tmem_st_wait();
}

template <int kD>
__global__ void __launch_bounds__(Fwd<kD>::kThreads, 1) attention_kernel(const __grid_constant__ AttentionLaunch p) {
  using F = Fwd<kD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * F::kTileBytes;
  uint64_t* q_full = reinterpret_cast<uint64_t*>(ring + F::kSlots * F::kTileBytes);
  uint64_t* full = q_full + 1;
  uint64_t* empty = full + F::kSlots;
  uint64_t* patched = empty + F::kSlots;
  uint64_t* s_full = patched + 1;   // scores of a unit are there
  uint64_t* p_full = s_full + 2;    // probabilities are
  uint64_t* o_full = p_full + 2;    // the outputs are
  uint64_t* drain = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ Place place;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, kv = blockIdx.y;
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < F::kSlots; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
    mbar_init(patched, 1);
    for (int j = 0; j < 2; ++j) mbar_init(&s_full[j], 1), mbar_init(&p_full[j], 4), mbar_init(&o_full[j], 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8 && lane == 0) prefetch_tensormap(&p.map_q), prefetch_tensormap(&p.map_k), prefetch_tensormap(&p.map_v);
  griddep_wait();
  const int group = p.heads / p.kv_heads;
  if (warp == 9) {
    const Place found = find_place(p, blockIdx.x, [&](int64_t len) { return ((len + kTile - 1) / kTile * group + 1) / 2; });
    if (lane == 0) place = found;
    if (found.length > 0) tmem_alloc(tmem_slot, F::kCols);
  }
  zero_rows_outside(p, p.out, p.heads, p.lse);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int64_t begin = place.begin, length = place.length;
  if (length == 0) return;
  const uint32_t tmem = *tmem_slot;
  const Unit units[2] = {unit_at(p, length, 2 * place.piece, kv), unit_at(p, length, 2 * place.piece + 1, kv)};
  const int tiles = max(units[0].tiles, units[1].tiles);
  // Of the last tile's values the rows behind the sequence are someone else's: whatever they hold meets probabilities of
  // 0, and must be 0 too.
  const bool patch = static_cast<int64_t>(tiles) * kTile > length;

  if (warp == 8) {
    // ------------------------------------------------------------------ copies
    bool ok = true;
    uint32_t issued = 0, parity = 0;
    int slot = 0;
    uint32_t phase = 0;
    if (lane == 0) {
      const int present = units[1].tiles > 0 ? 2 : 1;
      mbar_arrive_expect_tx(q_full, present * F::kTileBytes);
      for (int j = 0; j < present; ++j)
        for (int b = 0; b < F::kBoxes; ++b)
          tma_load_3d(smem_u32(smem + j * F::kTileBytes + b * F::kBoxBytes), &p.map_q, b * 64, units[j].head,
                      static_cast<int>(begin + units[j].row), q_full);
      for (int t = 0; ok && t < 2 * tiles; ++t) {  // keys and values of a tile in turn
        if (!wait_fast(&empty[slot], phase ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[slot], F::kTileBytes);
        for (int b = 0; b < F::kBoxes; ++b)
          tma_load_3d(smem_u32(ring + slot * F::kTileBytes + b * F::kBoxBytes), t & 1 ? &p.map_v : &p.map_k, b * 64, kv,
                      static_cast<int>(begin + static_cast<int64_t>(t >> 1) * kTile), &full[slot]);
        issued |= 1u << slot;
        parity = (parity & ~(1u << slot)) | (phase << slot);
        if (++slot == F::kSlots) slot = 0, phase ^= 1u;
      }
    }
    __syncwarp();
    if (patch) {
      const int last = (2 * tiles - 1) % F::kSlots;
      const uint32_t ph = ((2 * tiles - 1) / F::kSlots) & 1;
      ok = __all_sync(0xffffffffu, ok && wait_bounded(&full[last], ph, abort_flag, p.status, kWaitLimitNs, true));
      if (ok) {
        const int valid = static_cast<int>(length - static_cast<int64_t>(tiles - 1) * kTile);
        for (int b = 0; b < F::kBoxes; ++b)
          for (int i = valid * 8 + lane; i < kTile * 8; i += 32)
            *reinterpret_cast<uint4*>(ring + last * F::kTileBytes + b * F::kBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(patched);
      }
    }
    if (lane == 0 && (!ok || *abort_flag)) {
      wait_bounded(q_full, 0, abort_flag, p.status, kDrainLimitNs, false);
      for (int s = 0; s < F::kSlots; ++s)
        if ((issued >> s) & 1u) wait_bounded(&full[s], (parity >> s) & 1u, abort_flag, p.status, kDrainLimitNs, false);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ products
    if (lane == 0) {
      const uint32_t qk_desc = instr_desc_bf16<kTile, kTile>(false), pv_desc = instr_desc_bf16<kTile, kD>(true);
      int slot = 0;
      uint32_t phase = 0;
      auto next = [&] {
        if (++slot == F::kSlots) slot = 0, phase ^= 1u;
      };
      auto wait = [&](uint64_t* bar, uint32_t ph) { return wait_fast(bar, ph, abort_flag, p.status); };
      auto scores = [&](int j, int key_slot) {
        const uint32_t q = smem_u32(smem + j * F::kTileBytes), k = smem_u32(ring + key_slot * F::kTileBytes);
#pragma unroll
        for (int s = 0; s < kD / 16; ++s) {
          const uint32_t off = (s >> 2) * F::kBoxBytes + (s & 3) * 32;
          mma_f16(tmem + F::kScores + j * kTile, smem_desc(q + off, 16, 1024), smem_desc(k + off, 16, 1024), qk_desc, s > 0);
        }
        mma_commit(&s_full[j]);
      };
      bool ok = wait(q_full, 0) && wait(&full[0], 0);
      if (ok) {
        tc_fence_after();
        for (int j = 0; j < 2; ++j)
          if (units[j].tiles > 0) scores(j, 0);
        mma_commit(&empty[0]);
        next();
      }
      for (int i = 0; ok && i < tiles; ++i) {
        const int v_slot = slot;
        ok = wait(&full[v_slot], phase);
        if (ok && patch && i + 1 == tiles) ok = wait(patched, 0);
        next();
        const int k_slot = slot;
        const uint32_t k_phase = phase;
        if (i + 1 < tiles) next();
        bool have_keys = false;
        for (int j = 0; ok && j < 2; ++j) {
          if (i < units[j].tiles) {
            if (!(ok = wait(&p_full[j], i & 1))) break;
            tc_fence_after();
            const uint32_t v = smem_u32(ring + v_slot * F::kTileBytes);
#pragma unroll
            for (int s = 0; s < kTile / 16; ++s)
              mma_tmem_a(tmem + F::kOut + j * kTile, tmem + F::kScores + j * kTile + s * 8,
                         smem_desc(v + s * 2048, F::kBoxBytes, 1024), pv_desc, i > 0 || s > 0);
            if (i + 1 == units[j].tiles) mma_commit(&o_full[j]);
          }
          if (j == 1) mma_commit(&empty[v_slot]);
          if (i + 1 < units[j].tiles) {
            if (!have_keys && !(ok = wait(&full[k_slot], k_phase))) break;
            have_keys = true;
            tc_fence_after();
            scores(j, k_slot);
          }
        }
        if (ok && i + 1 < tiles) mma_commit(&empty[k_slot]);
      }
      mma_commit(drain);
      wait_bounded(drain, 0, abort_flag, p.status, kDrainLimitNs, false);
    }
  } else {
    // ------------------------------------------------------------------ softmax: one row a thread
    const int j = warp >> 2, r = (warp & 3) * 32 + lane;
    const Unit u = units[j];
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + F::kScores + j * kTile, t_o = tmem + lanes + F::kOut + j * kTile;
    const float sl2 = p.scale_log2;
    const bool negative = p.scale < 0.f;
    float top = -INFINITY;  // the maximum in use
    float2 sum = make_float2(0.f, 0.f);
    bool ok = true;
    for (int i = 0; i < u.tiles; ++i) {
      ok = wait_fast(&s_full[j], i & 1, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      // Keys that this row meets of the tile.
      const int64_t key0 = static_cast<int64_t>(i) * kTile;
      const bool masked = (p.causal && key0 == u.row) || key0 + kTile > length;
      const int keys = masked ? static_cast<int>((p.causal && u.row + r < length ? u.row + r + 1 : length) - key0) : kTile;
      uint32_t x[2][32];
      auto scores_of = [&](uint32_t (&v)[32], int c) {  // chunk c of the row, which has arrived
        if (negative) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] ^= 0x80000000u;
        }
        if (masked) {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = c * 32 + e < keys ? v[e] : 0xff800000u;
        }
      };
      // The scores are read twice, a quarter of a row at a time and the next one under way: 128 of them and their
      // probabilities are more registers than a thread has.
      float m4[4] = {top, top, top, top};
      tmem_ld32_issue(t_s, x[0]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tmem_ld_wait(x[c & 1]);
        if (c < 3) tmem_ld32_issue(t_s + (c + 1) * 32, x[(c + 1) & 1]);
        scores_of(x[c & 1], c);
#pragma unroll
        for (int e = 0; e < 32; e += 8)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            m4[q] = fmaxf(m4[q], fmaxf(__uint_as_float(x[c & 1][e + 2 * q]), __uint_as_float(x[c & 1][e + 2 * q + 1])));
      }
      const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      if (__any_sync(0xffffffffu, (m - top) * sl2 > kRaise)) {
        const float f = top == m ? 1.f : pow2((top - m) * sl2);
        top = m;
        sum = mul2(sum, make_float2(f, f));
        if (i > 0) scale_outputs<kD>(t_o, f);
      }
      const float shift = top == -INFINITY ? 0.f : -top * sl2;
      tmem_ld32_issue(t_s, x[0]);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        tmem_ld_wait(x[c & 1]);
        if (c < 3) tmem_ld32_issue(t_s + (c + 1) * 32, x[(c + 1) & 1]);
        scores_of(x[c & 1], c);
        uint32_t half[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float2 y = fma2(make_float2(__uint_as_float(x[c & 1][e]), __uint_as_float(x[c & 1][e + 1])), make_float2(sl2, sl2),
                          make_float2(shift, shift));
          y = make_float2(pow2(y.x), pow2(y.y));
          sum = add2(sum, y);
          half[e / 2] = pack_bf16(y.x, y.y);
        }
        // Over columns that have been read: probabilities take half of their scores' place, from its start on.
        tmem_st16(t_s + c * 16, half);
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[j]);
    }
    if (u.tiles > 0 && ok) {
      ok = wait_fast(&o_full[j], 0, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        tc_fence_after();
        const float total = sum.x + sum.y, inverse = 1.f / total;
        const bool live = u.row + r < length;
        const int64_t token = begin + u.row + r;
        bf16* out = out_at(p.out, live ? token : begin, u.head);
#pragma unroll
        for (int c = 0; c < kD; c += 32) {
          uint32_t o[32];
          tmem_ld32_issue(t_o + c, o);
          tmem_ld_wait(o);
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[k + e]) * inverse;
            if (live && c + k < p.dim) *reinterpret_cast<uint4*>(out + c + k) = row::pack16(v);
          }
        }
        if (live) p.lse[static_cast<int64_t>(u.head) * p.n + token] =
            kLn2 * ((top == -INFINITY ? 0.f : top * sl2) + log2f(total));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, F::kCols);
}

// ---------------------------------------------------------------------------- backward

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

template <int kD>
cudaError_t launch_forward(AttentionLaunch& p, cudaStream_t stream) {
  using F = Fwd<kD>;
  const char* why = nullptr;
  if (!encode_heads(&p.map_q, p.q, p.dim, p.heads, p.n, kTile, &why) ||
      !encode_heads(&p.map_k, p.k, p.dim, p.kv_heads, p.n, kTile, &why) ||
      !encode_heads(&p.map_v, p.v, p.dim, p.kv_heads, p.n, kTile, &why))
    return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(attention_kernel<kD>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t group = p.heads / p.kv_heads, filled = std::min(p.sequences, p.n);
  // Pairs of units: of equal sequences exactly; of others at most, every sequence having one unit per head more than
  // its tokens fill, and one unit alone.
  int64_t slots = 0;
  if (!p.offsets) slots = p.sequences * (((p.n / p.sequences + kTile - 1) / kTile * group + 1) / 2);
  else slots = ((p.n / kTile + filled) * group + filled) / 2 + 1;
  if (slots > 0x7fffffff) return cudaErrorInvalidValue;
  return row::launch(attention_kernel<kD>, dim3(static_cast<unsigned>(slots), static_cast<unsigned>(p.kv_heads)), F::kThreads,
                     F::kSmem, stream, p);
}

}  // namespace

int64_t attention_workspace(AttentionLaunch& p, char* ws) {
  if (ws) p.delta = reinterpret_cast<float*>(ws);
  return static_cast<int64_t>(sizeof(float)) * p.n * p.heads;
}

cudaError_t launch_attention(AttentionLaunch& p, int sms, cudaStream_t stream) {
  p.scale_log2 = fabsf(p.scale) * kLog2e;
  return p.dim <= 64 ? launch_forward<64>(p, stream) : launch_forward<128>(p, stream);
}

cudaError_t launch_attention_grad(AttentionLaunch& p, int sms, cudaStream_t stream) {
  cudaError_t e = row::launch(attention_delta_kernel, dim3(ctas_for(p.n * p.heads)), kThreads, 0, stream, p);
  if (e == cudaSuccess) e = row::launch(attention_dq_kernel, dim3(ctas_for(p.n * p.heads)), kThreads, 0, stream, p);
  if (e == cudaSuccess) e = row::launch(attention_dkv_kernel, dim3(ctas_for(p.n * p.kv_heads)), kThreads, 0, stream, p);
  return e;
}

}  // namespace dmuon
