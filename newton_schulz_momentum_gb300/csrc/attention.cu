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
//
// What bounds it is the way of a row's scores out of tensor memory, through 128 exponentials a thread and back, against
// products that take as long. Measured, 32 heads of 128 with 8 key heads, 8192 tokens, causal: 367 us, 1500 TFLOP/s, 0.77
// of a library product's rate (450 us with the scores read twice, 407 with products issued one by one).
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

// By one warp. Without offsets the sequences are equal; otherwise 128 of them at a time, four to a lane, since a look
// at memory takes a microsecond however little is read.
template <typename F>
__device__ __forceinline__ Place find_place(const AttentionLaunch& p, int64_t slot, F&& per) {
  constexpr int kEach = 4;
  const int lane = threadIdx.x & 31;
  Place at{0, 0, 0};
  if (!p.offsets) {
    const int64_t len = p.n / p.sequences, piece = slot / p.sequences, s = slot - piece * p.sequences;
    if (piece < per(len)) at = {s * len, len, piece};
    return at;
  }
  for (int64_t s0 = 0; s0 < p.sequences; s0 += 32 * kEach) {
    int64_t begin[kEach], len[kEach], sum = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      const int64_t s = s0 + lane * kEach + k;
      begin[k] = len[k] = 0;
      if (s < p.sequences) len[k] = sequence_length(p, s, &begin[k]);
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k) sum += len[k] > 0 ? per(len[k]) : 0;
    const int64_t mine = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t left = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += left;
    }
    const unsigned behind = __ballot_sync(0xffffffffu, slot < sum);
    if (behind) {
      int64_t piece = slot - (sum - mine);
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int64_t pieces = len[k] > 0 ? per(len[k]) : 0;
        if (at.length == 0 && piece < pieces) at = {begin[k], len[k], piece};
        piece -= pieces;
      }
      const int l = __ffs(behind) - 1;
      at.begin = __shfl_sync(0xffffffffu, at.begin, l);
      at.length = __shfl_sync(0xffffffffu, at.length, l);
      at.piece = __shfl_sync(0xffffffffu, at.piece, l);
      return at;
    }
    slot -= __shfl_sync(0xffffffffu, sum, 31);
  }
  return at;
}

// The same with the longest pieces first, for up to 128 sequences: of `blocks` tiles each, one piece a tile, the pieces of
// a causal sequence are 1 to `blocks` tiles long, of another `blocks` each. The place's length in tiles (its level) is
// found by halving, then the sequence among those that have such a piece. For dk and dv, whose pieces are few and go through
// all of a key head's query heads: 37 sequences of 16001 tokens in all take 124 us so and 147 in their own order, whose last
// pieces may be long. (dq's pieces are many and short: 122 us in the sequences' order, 128 so, for the time of the search.)
__device__ __forceinline__ Place find_tile(const AttentionLaunch& p, int64_t slot) {
  if (!p.offsets || p.sequences > 128)
    return find_place(p, slot, [](int64_t length) { return (length + kTile - 1) / kTile; });
  constexpr int kEach = 4;
  const int lane = threadIdx.x & 31;
  Place at{0, 0, 0};
  int64_t begin[kEach], len[kEach];
  unsigned blocks[kEach], most = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int64_t s = lane * kEach + k;
    begin[k] = len[k] = 0;
    if (s < p.sequences) len[k] = sequence_length(p, s, &begin[k]);
    blocks[k] = static_cast<unsigned>((len[k] + kTile - 1) / kTile);
    most = max(most, blocks[k]);
  }
  // Pieces of at least `level` tiles, of all sequences.
  auto count = [&](unsigned level) {
    unsigned mine = 0;
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (blocks[k] >= level) mine += p.causal ? blocks[k] - level + 1 : blocks[k];
    return __reduce_add_sync(0xffffffffu, mine);
  };
  const unsigned place = static_cast<unsigned>(slot);
  if (place >= count(1)) return at;
  unsigned low = 1, high = __reduce_max_sync(0xffffffffu, most);  // the largest level with more pieces than `place`
  while (low < high) {
    const unsigned mid = (low + high + 1) / 2;
    if (count(mid) > place) low = mid;
    else high = mid - 1;
  }
  const unsigned level = low, index = place - count(level + 1);  // among the pieces of this length
  unsigned mine = 0;
#pragma unroll
  for (int k = 0; k < kEach; ++k) mine += p.causal ? blocks[k] >= level : blocks[k] == level ? level : 0u;
  unsigned sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned left = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += left;
  }
  const int l = __ffs(__ballot_sync(0xffffffffu, index < sum)) - 1;
  int64_t rest = static_cast<int64_t>(index) - (sum - mine);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int64_t here = p.causal ? blocks[k] >= level : blocks[k] == level ? level : 0u;
    if (at.length == 0 && rest < here) at = {begin[k], len[k], p.causal ? static_cast<int64_t>(blocks[k] - level) : rest};
    rest -= here;
  }
  at.begin = __shfl_sync(0xffffffffu, at.begin, l);
  at.length = __shfl_sync(0xffffffffu, at.length, l);
  at.piece = __shfl_sync(0xffffffffu, at.piece, l);
  return at;
}

__device__ __forceinline__ const bf16* at(const HeadArray& a, int64_t token, int64_t head) {
  return static_cast<const bf16*>(a.data) + token * a.token + head * a.head;
}
__device__ __forceinline__ bf16* out_at(const HeadArray& a, int64_t token, int64_t head) {
  return static_cast<bf16*>(const_cast<void*>(a.data)) + token * a.token + head * a.head;
}

// Zeros in the rows of tokens that belong to no sequence, spread over the grid's CTAs; by a warp of each that has time.
__device__ __forceinline__ void zero_rows_outside(const AttentionLaunch& p, const HeadArray& a, int heads, float* lse) {
  if (!p.offsets || !p.zero_outside) return;
  const int64_t first = row::load_id(p.offsets, p.id_bytes, 0), last = row::load_id(p.offsets, p.id_bytes, p.sequences);
  const int64_t before = first < 0 ? 0 : first > p.n ? p.n : first, from = last < before ? before : last > p.n ? p.n : last;
  const int64_t rows = (before + p.n - from) * heads;
  const int64_t lane = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x & 31);
  for (int64_t r = lane; r < rows; r += static_cast<int64_t>(gridDim.x) * 32) {
    const int64_t k = r / heads, head = r - k * heads, token = k < before ? k : from + (k - before);
    bf16* x = out_at(a, token, head);
    for (int c = 0; c < p.dim; c += 8) *reinterpret_cast<uint4*>(x + c) = make_uint4(0, 0, 0, 0);
    if (lse) lse[head * p.n + token] = 0.f;
  }
}

// ---------------------------------------------------------------------------- tiles and products

// Columns of tensor memory: a CTA takes all 512 of them, from address 0 on.
constexpr uint32_t kCols = 512;

// A tile is 128 rows of kD columns (a head's, padded with zeros to 64 or 128), as boxes of 64 columns.
template <int kD>
struct Tile {
  static constexpr int kBytes = kTile * kD * 2, kBoxes = kD / 64, kBoxBytes = kTile * 128;
};

// One thread's copies of a tile: `row` is the first token's index in the arrays.
template <int kD>
__device__ __forceinline__ void load_tile(uint32_t dst, const CUtensorMap* map, int head, int64_t row, uint64_t* bar) {
#pragma unroll
  for (int b = 0; b < Tile<kD>::kBoxes; ++b)
    tma_load_3d(dst + b * Tile<kD>::kBoxBytes, map, b * 64, head, static_cast<int>(row), bar);
}

// The products of a tile are issued by one lane of a warp that is here as a whole, all of them in one statement: operands
// that are brought together for one product after another, under a branch, take longer than the products (eight of
// 128 x 128 x 16 from an idle start: 520 cycles of issue by lane 0, 340 under an elected lane's branch, 104 like this,
// 512 for the products themselves). Offsets are in 16-byte units of a descriptor's low word.
#define DM_SS(step, off, add)                                                                                          \
  "add.u32 l, %1, " off ";\n\tmov.b64 a, {l, %3};\n\tadd.u32 l, %2, " off ";\n\tmov.b64 b, {l, %3};\n\t"              \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, " add ";\n\t"
#define DM_TS(step, a_off, b_off)                                                                                      \
  "add.u32 t, %1, " a_off ";\n\tadd.u32 l, %2, " b_off ";\n\tmov.b64 b, {l, %3};\n\t"                                  \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [t], b, %4, " step ";\n\t"
#define DM_ELECT                                                                                                       \
  "{\n\t.reg .pred e, f, p, q;\n\t.reg .b64 a, b;\n\t.reg .b32 l, t;\n\telect.sync _|e, 0xffffffff;\n\t"              \
  "setp.ne.u32 f, 0, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"

// D = A B^T of two tiles.
template <int kD>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a, uint32_t b) {
  static_assert(Tile<kD>::kBoxBytes >> 4 == 1024, "offsets of the second box");
  const uint32_t desc = instr_desc_bf16<kTile, kTile>(false);
  const uint64_t da = smem_desc(a, 16, 1024), db = smem_desc(b, 16, 1024);
  const uint32_t al = static_cast<uint32_t>(da), bl = static_cast<uint32_t>(db), high = static_cast<uint32_t>(db >> 32);
  if constexpr (kD == 64) {
    asm volatile(DM_ELECT DM_SS(0, "0", "f") DM_SS(1, "2", "q") DM_SS(2, "4", "q") DM_SS(3, "6", "q") "}\n" ::"r"(d),
                 "r"(al), "r"(bl), "r"(high), "r"(desc)
                 : "memory");
  } else {
    asm volatile(DM_ELECT DM_SS(0, "0", "f") DM_SS(1, "2", "q") DM_SS(2, "4", "q") DM_SS(3, "6", "q")
                     DM_SS(4, "1024", "q") DM_SS(5, "1026", "q") DM_SS(6, "1028", "q") DM_SS(7, "1030", "q") "}\n" ::"r"(d),
                 "r"(al), "r"(bl), "r"(high), "r"(desc)
                 : "memory");
  }
}

// D (+)= A B, A being 128 x 128 bf16 in tensor memory, two of its columns in one: side by side from `a` on, or kParts:
// each 32 of them at the start of the 32 columns of the scores that they were made from.
template <int kD, bool kParts>
__device__ __forceinline__ void mma_columns(uint32_t d, uint32_t a, uint32_t b, bool add) {
  const uint32_t desc = instr_desc_bf16<kTile, kD>(true);
  const uint64_t db = smem_desc(b, Tile<kD>::kBoxBytes, 1024);
  const uint32_t bl = static_cast<uint32_t>(db), high = static_cast<uint32_t>(db >> 32);
  if constexpr (!kParts) {
    asm volatile(DM_ELECT "setp.ne.u32 p, %5, 0;\n\t" DM_TS("p", "0", "0") DM_TS("q", "8", "128") DM_TS("q", "16", "256")
                     DM_TS("q", "24", "384") DM_TS("q", "32", "512") DM_TS("q", "40", "640") DM_TS("q", "48", "768")
                         DM_TS("q", "56", "896") "}\n" ::"r"(d),
                 "r"(a), "r"(bl), "r"(high), "r"(desc), "r"(static_cast<uint32_t>(add))
                 : "memory");
  } else {
    asm volatile(DM_ELECT "setp.ne.u32 p, %5, 0;\n\t" DM_TS("p", "0", "0") DM_TS("q", "8", "128") DM_TS("q", "32", "256")
                     DM_TS("q", "40", "384") DM_TS("q", "64", "512") DM_TS("q", "72", "640") DM_TS("q", "96", "768")
                         DM_TS("q", "104", "896") "}\n" ::"r"(d),
                 "r"(a), "r"(bl), "r"(high), "r"(desc), "r"(static_cast<uint32_t>(add))
                 : "memory");
  }
}
#undef DM_SS
#undef DM_TS
#undef DM_ELECT

// D += A B^T of two strips, 128 rows of 16 columns: 8 rows of 16 bytes one after another, the second 8 columns of the same
// rows 128 bytes behind, the next 8 rows 256.
constexpr int kStripBytes = kTile * 32;
__device__ __forceinline__ void mma_strips(uint32_t d, uint32_t a, uint32_t b) {
  // No swizzle (layout 0), descriptor version 1.
  constexpr uint64_t form = (static_cast<uint64_t>(128 >> 4) << 16) | (static_cast<uint64_t>(256 >> 4) << 32) | (1ull << 46);
  asm volatile(
      "{\n\t.reg .pred e, q;\n\telect.sync _|e, 0xffffffff;\n\tsetp.eq.u32 q, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, q;\n\t}\n" ::"r"(d),
      "l"(form | ((a & 0x3FFFFu) >> 4)), "l"(form | ((b & 0x3FFFFu) >> 4)), "r"(instr_desc_bf16<kTile, kTile>(false))
      : "memory");
}

// x to 24 bits as three bf16 terms, in the first half of a strip's row.
__device__ __forceinline__ void store_strip(uint8_t* strip, int row, float x) {
  const float hi = __bfloat162float(__float2bfloat16_rn(x));
  const float rest = isinf(x) ? 0.f : x - hi, mid = __bfloat162float(__float2bfloat16_rn(rest));
  *reinterpret_cast<uint4*>(strip + (row >> 3) * 256 + (row & 7) * 16) =
      make_uint4(pack_bf16(hi, mid), pack_bf16(rest - mid, 0.f), 0u, 0u);
}

// ---------------------------------------------------------------------------- forward

template <int kD>
struct Fwd : Tile<kD> {
  static constexpr int kSlots = 4, kTileBytes = Tile<kD>::kBytes;
  static constexpr int kThreads = 320;  // warps 0-3 and 4-7: a unit's rows each; 8: copies; 9: products
  static constexpr int kSmem = (2 + kSlots) * kTileBytes + 1024 + 256;
  static constexpr uint32_t kScores = 0, kOut = 256;  // columns of the first unit; the second's are kTile behind
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

// A warp's 32 rows of kCols columns of an accumulator from taddr on, times each lane's f, to `out` as bf16: the first
// `rows` rows, `stride` elements apart, and `columns` columns. Through `stage` (64 kCols bytes of shared memory), so that
// neighbouring lanes store neighbouring 16 bytes: of a row each, a store would touch 32 rows.
template <int kCols>
__device__ __forceinline__ void store_block(uint8_t* stage, uint32_t taddr, float f, bf16* out, int64_t stride, int rows,
                                            int columns) {
  constexpr int kChunks = kCols / 8;  // of 16 bytes in a row
  constexpr int kTurn = kChunks < 8 ? kChunks - 1 : 7;
  const int lane = threadIdx.x & 31, turn = kChunks < 8 ? (lane >> 1) & kTurn : lane & kTurn;
#pragma unroll
  for (int c = 0; c < kCols; c += 32) {
    uint32_t r[32];
    tmem_ld32_issue(taddr + c, r);
    tmem_ld_wait(r);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r[8 * k + e]) * f;
      *reinterpret_cast<uint4*>(stage + (lane * kChunks + ((c / 8 + k) ^ turn)) * 16) = row::pack16(v);
    }
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < kChunks; ++k) {
    const int id = k * 32 + lane, row = id / kChunks, chunk = id % kChunks;
    const int at = chunk ^ (kChunks < 8 ? (row >> 1) & kTurn : row & kTurn);
    if (row < rows && chunk * 8 < columns)
      *reinterpret_cast<uint4*>(out + row * stride + chunk * 8) = *reinterpret_cast<uint4*>(stage + (row * kChunks + at) * 16);
  }
}

// A row of outputs times f; seldom run, so a few columns at a time beside the 128 scores that the thread holds.
template <int kD>
__device__ __forceinline__ void scale_outputs(uint32_t tmem_out, float f) {
#pragma unroll 1
  for (int c = 0; c < kD; c += 8) {
    uint32_t r[8];
    tmem_ld8_issue(tmem_out + c, r);
    tmem_ld_wait(r);
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * f);
    tmem_st8(tmem_out + c, r);
  }
  tmem_st_wait();
}

template <int kD>
__global__ void __launch_bounds__(Fwd<kD>::kThreads, 1) attention_kernel(const __grid_constant__ AttentionLaunch p) {
  using F = Fwd<kD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem + 2 * F::kTileBytes;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u, ring_at = base + 2 * F::kTileBytes;
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

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int kv = blockIdx.x % p.kv_heads;
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
    const Place found = find_place(p, blockIdx.x / p.kv_heads,
                                   [&](int64_t len) { return ((len + kTile - 1) / kTile * group + 1) / 2; });
    if (lane == 0) place = found;
    if (found.length > 0) tmem_alloc(tmem_slot, kCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int64_t begin = place.begin, length = place.length;
  if (length == 0) {
    if (warp == 0) zero_rows_outside(p, p.out, p.heads, p.lse);
    return;
  }
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
        load_tile<kD>(base + j * F::kTileBytes, &p.map_q, units[j].head, begin + units[j].row, q_full);
      for (int t = 0; ok && t < 2 * tiles; ++t) {  // keys and values of a tile in turn
        if (!wait_fast(&empty[slot], phase ^ 1u, abort_flag, p.status)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&full[slot], F::kTileBytes);
        load_tile<kD>(ring_at + slot * F::kTileBytes, t & 1 ? &p.map_v : &p.map_k, kv,
                      begin + static_cast<int64_t>(t >> 1) * kTile, &full[slot]);
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
    zero_rows_outside(p, p.out, p.heads, p.lse);
    if (lane == 0 && (!ok || *abort_flag)) {
      wait_bounded(q_full, 0, abort_flag, p.status, kDrainLimitNs, false);
      for (int s = 0; s < F::kSlots; ++s)
        if ((issued >> s) & 1u) wait_bounded(&full[s], (parity >> s) & 1u, abort_flag, p.status, kDrainLimitNs, false);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ products
    const int counts[2] = {__shfl_sync(0xffffffffu, units[0].tiles, 0), __shfl_sync(0xffffffffu, units[1].tiles, 0)};
    const int n = max(counts[0], counts[1]);
    const bool cut = __any_sync(0xffffffffu, patch);
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      return __all_sync(0xffffffffu, wait_fast(bar, ph, abort_flag, p.status)) != 0;
    };
    auto scores = [&](int j, int key_slot) {
      mma_rows<kD>(F::kScores + j * kTile, base + j * F::kTileBytes, ring_at + key_slot * F::kTileBytes);
      mma_commit_elected(&s_full[j]);
    };
    int slot = 0;
    uint32_t phase = 0;
    auto next = [&] {
      if (++slot == F::kSlots) slot = 0, phase ^= 1u;
    };
    bool ok = wait(q_full, 0) && wait(&full[0], 0);
    if (ok) {
      tc_fence_after();
#pragma unroll
      for (int j = 0; j < 2; ++j)
        if (counts[j] > 0) scores(j, 0);
      mma_commit_elected(&empty[0]);
      next();
    }
    for (int i = 0; ok && i < n; ++i) {
      const int v_slot = slot;
      ok = wait(&full[v_slot], phase) && (!cut || i + 1 < n || wait(patched, 0));
      next();
      const int k_slot = slot;
      const uint32_t k_phase = phase;
      if (ok && i + 1 < n) {
        ok = wait(&full[k_slot], k_phase);
        next();
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (ok && i < counts[j]) {
          ok = wait(&p_full[j], i & 1);
          tc_fence_after();
          if (ok) {
            mma_columns<kD, false>(F::kOut + j * kTile, F::kScores + j * kTile, ring_at + v_slot * F::kTileBytes, i > 0);
            if (i + 1 == counts[j]) mma_commit_elected(&o_full[j]);
          }
        }
        if (j == 1 && ok) mma_commit_elected(&empty[v_slot]);
        if (ok && i + 1 < counts[j]) scores(j, k_slot);
      }
      if (ok && i + 1 < n) mma_commit_elected(&empty[k_slot]);
    }
    if (elect_one()) {
      mma_commit(drain);
      wait_bounded(drain, 0, abort_flag, p.status, kDrainLimitNs, false);
    }
  } else {
    // ------------------------------------------------------------------ softmax: one row a thread
    const int j = warp >> 2, r = (warp & 3) * 32 + lane;
    const Unit u = units[j];
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = lanes + F::kScores + j * kTile, t_o = lanes + F::kOut + j * kTile;
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
      // All 128 scores in registers at once: a wait for tensor memory is one for all loads under way, so pieces of a row
      // would each take its latency.
      uint32_t x[kTile];
#pragma unroll
      for (int c = 0; c < kTile; c += 32) tmem_ld32_issue(t_s + c, x + c);
      tmem_ld_wait(x);
      if (negative) {
#pragma unroll
        for (int c = 0; c < kTile; ++c) x[c] ^= 0x80000000u;
      }
      if (masked) {
#pragma unroll
        for (int c = 0; c < kTile; ++c) x[c] = c < keys ? x[c] : 0xff800000u;
      }
      float m4[4] = {top, top, top, top};
#pragma unroll
      for (int c = 0; c < kTile; c += 8)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          m4[q] = fmaxf(m4[q], fmaxf(__uint_as_float(x[c + 2 * q]), __uint_as_float(x[c + 2 * q + 1])));
      const float m = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
      if (__any_sync(0xffffffffu, (m - top) * sl2 > kRaise)) {
        const float f = top == m ? 1.f : pow2((top - m) * sl2);
        top = m;
        sum = mul2(sum, make_float2(f, f));
        if (i > 0) scale_outputs<kD>(t_o, f);
      }
      const float shift = top == -INFINITY ? 0.f : -top * sl2;
#pragma unroll
      for (int c = 0; c < kTile; c += 16) {
        uint32_t half[8];
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          float2 y = fma2(make_float2(__uint_as_float(x[c + e]), __uint_as_float(x[c + e + 1])), make_float2(sl2, sl2),
                          make_float2(shift, shift));
          y = make_float2(pow2(y.x), pow2(y.y));
          sum = add2(sum, y);
          half[e / 2] = pack_bf16(y.x, y.y);
        }
        tmem_st8(t_s + c / 2, half);
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
        // Over the unit's queries, which no product reads any more.
        const int64_t left = length - u.row - (warp & 3) * 32;
        if (left > 0)
          store_block<kD>(smem + j * F::kTileBytes + (warp & 3) * 64 * kD, t_o, inverse,
                          out_at(p.out, begin + u.row + (warp & 3) * 32, u.head), p.out.token,
                          static_cast<int>(left < 32 ? left : 32), p.dim);
        if (live) p.lse[static_cast<int64_t>(u.head) * p.n + token] =
            kLn2 * ((top == -INFINITY ? 0.f : top * sl2) + log2f(total));
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(0, kCols);
}

// ---------------------------------------------------------------------------- backward
//
// Two kernels, each over its own rows, so that every sum has one owner and one order (a single pass would add dq or dk
// and dv across CTAs): scores and dout . v are formed in both, 7 products of a pair of tiles in place of 5.
//
// Queries (dq): a CTA has 128 queries of one head. Scores lie in one buffer of tensor memory, dout . v in two in turn,
// so that the products for the next tile of keys run while ds of this one is formed (over its dout . v, as bf16, the left
// operand of the product with the keys). D = dout . out is off by what out lost in its rounding, which counts where
// rows have few keys, whose ds cancel. So the sum of ds, which is 0 but for that, is added to D: for dk in all rows
// (delta), and for dq in rows whose keys lie in one tile.
//
// Keys (dk, dv): a CTA has 128 keys of a key head and meets the queries of all its query heads. Scores are formed
// transposed, so that a thread has a key's row and p and ds are again left operands from tensor memory: scores, dout . v,
// dv and dk fill its 512 columns. Products of one kind run while the warps work on the other:
// dv(i), scores(i + 1), dk(i), dout . v(i + 1).
//
// In both, 16 warps form p and ds, each thread a quarter of a row: four warps a scheduler, since a warp alone spends most
// of its time on latencies (8192 tokens with 8 warps of 64 columns a thread, and D by loads of whole rows: 1.42 ms).
//
// Measured, 32 heads of 128 with 8 key heads, 8192 tokens, causal: 1.31 ms, 1.05 PFLOP/s of the five products that the
// gradient is made of and 1.47 of the seven that are formed, 0.84 of what a library product sustains for as long on the
// same chip, whose power limit it then runs at. 37 sequences of 16001 tokens in all, 14 + 2 heads of 64: 242 us, 122 of
// them dq (2002 CTAs of some 4 tiles, 9 us each from the first copy to the last row), 124 dk and dv.

constexpr int kPart = 32;             // columns of a row that a thread has
constexpr int kRowWarps = 16;

template <int kD>
struct Bwd : Tile<kD> {
  static constexpr int kTileBytes = Tile<kD>::kBytes;
  static constexpr int kThreads = 608;  // warps 0-15: rows; 16: copies; 17: products; 18: the queries' lse and D
  static constexpr int kKeySlots = 3, kValueSlots = 2, kQuerySlots = 3;
  static constexpr int kSmemQueries = (2 + kKeySlots + kValueSlots) * kTileBytes + 256 + kTile * 4 + 1024;
  static constexpr int kSmemKeys = 6 * kTileBytes + 5 * kStripBytes + 256 + 1024;
};

// Zeros in the rows from `valid` on of a tile in shared memory, by a warp, visible to the products.
template <int kD>
__device__ __forceinline__ void clear_rows(uint8_t* tile, int valid) {
  for (int b = 0; b < Tile<kD>::kBoxes; ++b)
    for (int i = valid * 8 + (threadIdx.x & 31); i < kTile * 8; i += 32)
      *reinterpret_cast<uint4*>(tile + b * Tile<kD>::kBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
  fence_async_smem();
}

// 32 columns of this thread's lane.
__device__ __forceinline__ void load_part(uint32_t taddr, float (&v)[kPart]) {
  uint32_t r[kPart];
  tmem_ld32_issue(taddr, r);
  tmem_ld_wait(r);
#pragma unroll
  for (int k = 0; k < kPart; ++k) v[k] = __uint_as_float(r[k]);
}

template <int kD>
__global__ void __launch_bounds__(Bwd<kD>::kThreads, 1) attention_dq_kernel(const __grid_constant__ AttentionLaunch p) {
  using F = Bwd<kD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *keys = smem + 2 * F::kTileBytes, *values = keys + F::kKeySlots * F::kTileBytes;  // behind queries and dout
  const uint32_t q_at = (smem_u32(smem_raw) + 1023) & ~1023u, do_at = q_at + F::kTileBytes, keys_at = do_at + F::kTileBytes,
                 values_at = keys_at + F::kKeySlots * F::kTileBytes;
  float* exchange = reinterpret_cast<float*>(smem);  // 4 x 128, over the queries when they are no longer needed
  uint64_t* q_full = reinterpret_cast<uint64_t*>(values + F::kValueSlots * F::kTileBytes);
  uint64_t* k_full = q_full + 1;
  uint64_t* k_empty = k_full + F::kKeySlots;
  uint64_t* v_full = k_empty + F::kKeySlots;
  uint64_t* v_empty = v_full + F::kValueSlots;
  uint64_t* patched = v_empty + F::kValueSlots;
  uint64_t* s_full = patched + 1;
  uint64_t* s_read = s_full + 1;
  uint64_t* dp_full = s_read + 1;  // of either buffer
  uint64_t* ds_full = dp_full + 2;
  uint64_t* exchanged = ds_full + 2;
  uint64_t* done = exchanged + 1;
  uint64_t* drain = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* row_delta = reinterpret_cast<float*>(q_full + 32);
  __shared__ Place place;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int head = blockIdx.x % p.heads, kv = head / (p.heads / p.kv_heads);
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < F::kKeySlots; ++s) mbar_init(&k_full[s], 1), mbar_init(&k_empty[s], 1);
    for (int s = 0; s < F::kValueSlots; ++s) mbar_init(&v_full[s], 1), mbar_init(&v_empty[s], 1);
    mbar_init(patched, 1), mbar_init(s_full, 1), mbar_init(s_read, kRowWarps);
    for (int b = 0; b < 2; ++b) mbar_init(&dp_full[b], 1), mbar_init(&ds_full[b], kRowWarps);
    mbar_init(exchanged, kRowWarps), mbar_init(done, 1), mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  griddep_wait();
  if (warp == 17) {
    const Place found = find_place(p, blockIdx.x / p.heads, [](int64_t len) { return (len + kTile - 1) / kTile; });
    if (lane == 0) place = found;
    if (found.length > 0) tmem_alloc(tmem_slot, kCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int64_t begin = place.begin, length = place.length;
  if (length == 0) {
    if (warp == 0) zero_rows_outside(p, p.dq, p.heads, nullptr);
    return;
  }
  constexpr uint32_t t_s = 0, t_dp = kTile, t_dq = 3 * kTile;
  const int64_t blocks = (length + kTile - 1) / kTile, block = blocks - 1 - place.piece, row0 = block * kTile;  // long rows first
  const int tiles = static_cast<int>(p.causal ? block + 1 : blocks);
  const bool patch = static_cast<int64_t>(tiles) * kTile > length;
  auto wait = [&](uint64_t* bar, uint32_t phase) { return wait_fast(bar, phase & 1u, abort_flag, p.status); };

  if (warp == 16) {
    // ------------------------------------------------------------------ copies
    bool ok = true;
    int i = 0, loaded_v = 0;
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, 2 * F::kTileBytes);
      load_tile<kD>(q_at, &p.map_q, head, begin + row0, q_full);
      load_tile<kD>(do_at, &p.map_dout, head, begin + row0, q_full);
      for (; i < tiles; ++i) {
        const int64_t row = begin + static_cast<int64_t>(i) * kTile;
        const int ks = i % F::kKeySlots, vs = i % F::kValueSlots;
        if (!(ok = wait(&k_empty[ks], i / F::kKeySlots + 1))) break;
        mbar_arrive_expect_tx(&k_full[ks], F::kTileBytes);
        load_tile<kD>(keys_at + ks * F::kTileBytes, &p.map_k, kv, row, &k_full[ks]);
        if (!(ok = wait(&v_empty[vs], i / F::kValueSlots + 1))) {
          ++i;
          break;
        }
        mbar_arrive_expect_tx(&v_full[vs], F::kTileBytes);
        load_tile<kD>(values_at + vs * F::kTileBytes, &p.map_v, kv, row, &v_full[vs]);
        ++loaded_v;
      }
    }
    __syncwarp();
    if (patch) {  // the keys behind the sequence meet ds of 0, and must be 0 too
      const int last = (tiles - 1) % F::kKeySlots;
      ok = __all_sync(0xffffffffu, ok && wait(&k_full[last], (tiles - 1) / F::kKeySlots));
      if (ok) {
        clear_rows<kD>(keys + last * F::kTileBytes, static_cast<int>(length - static_cast<int64_t>(tiles - 1) * kTile));
        __syncwarp();
        if (lane == 0) mbar_arrive(patched);
      }
    }
    zero_rows_outside(p, p.dq, p.heads, nullptr);
    if (lane == 0 && (!ok || *abort_flag)) {
      wait_bounded(q_full, 0, abort_flag, p.status, kDrainLimitNs, false);
      for (int t = max(0, i - F::kKeySlots); t < i; ++t)
        wait_bounded(&k_full[t % F::kKeySlots], (t / F::kKeySlots) & 1, abort_flag, p.status, kDrainLimitNs, false);
      for (int t = max(0, loaded_v - F::kValueSlots); t < loaded_v; ++t)
        wait_bounded(&v_full[t % F::kValueSlots], (t / F::kValueSlots) & 1, abort_flag, p.status, kDrainLimitNs, false);
    }
  } else if (warp == 17) {
    // ------------------------------------------------------------------ products
    const int n = __shfl_sync(0xffffffffu, tiles, 0);
    const bool cut = __any_sync(0xffffffffu, patch);
    auto all_wait = [&](uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };
    int ks = 0, vs = 0, dqs = 0;  // slots of the next scores, dout . v and dq
    uint32_t k_phase = 0, v_phase = 0;
    auto scores = [&](int i) {
      if (!all_wait(&k_full[ks], k_phase) || (cut && i + 1 == n && !all_wait(patched, 0)) || (i > 0 && !all_wait(s_read, i - 1)))
        return false;
      tc_fence_after();
      mma_rows<kD>(t_s, q_at, keys_at + ks * F::kTileBytes);
      mma_commit_elected(s_full);
      if (++ks == F::kKeySlots) ks = 0, k_phase ^= 1u;
      return true;
    };
    auto along = [&](int i) {
      if (!all_wait(&v_full[vs], v_phase)) return false;
      tc_fence_after();
      mma_rows<kD>(t_dp + (i & 1) * kTile, do_at, values_at + vs * F::kTileBytes);
      mma_commit_elected(&dp_full[i & 1]);
      mma_commit_elected(&v_empty[vs]);
      if (++vs == F::kValueSlots) vs = 0, v_phase ^= 1u;
      return true;
    };
    bool ok = all_wait(q_full, 0) && scores(0) && along(0);
    for (int i = 0; ok && i < n; ++i) {
      if (i + 1 < n) ok = scores(i + 1) && along(i + 1);
      ok = ok && all_wait(&ds_full[i & 1], i >> 1);
      if (!ok) break;
      tc_fence_after();
      mma_columns<kD, true>(t_dq, t_dp + (i & 1) * kTile, keys_at + dqs * F::kTileBytes, i > 0);
      mma_commit_elected(&k_empty[dqs]);
      if (i + 1 == n) mma_commit_elected(done);
      if (++dqs == F::kKeySlots) dqs = 0;
    }
    if (elect_one()) {
      mma_commit(drain);
      wait_bounded(drain, 0, abort_flag, p.status, kDrainLimitNs, false);
    }
  } else if (warp < kRowWarps) {
    // ------------------------------------------------------------------ rows
    const int part = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const bool live = row0 + r < length;
    const int64_t token = begin + (live ? row0 + r : 0);
    const float sl2 = p.scale * kLog2e, lse2 = live ? p.lse[static_cast<int64_t>(head) * p.n + token] * kLog2e : INFINITY;
    // D of the rows, 16 lanes to one: read by a thread each, a load would touch 32 rows (16 warps: 16000 cycles).
    {
      uint4 o[4], g[4];
      const int c = (lane & 15) * 8;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int q = warp * 8 + 2 * k + (lane >> 4);
        const int64_t row = begin + (row0 + q < length ? row0 + q : 0);
        o[k] = g[k] = make_uint4(0, 0, 0, 0);
        if (c < p.dim) {
          o[k] = *reinterpret_cast<const uint4*>(at(p.out, row, head) + c);
          g[k] = *reinterpret_cast<const uint4*>(at(p.dout, row, head) + c);
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float a[8], b[8], d = 0.f;
        row::unpack16<bf16>(a, o[k]);
        row::unpack16<bf16>(b, g[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) d = fmaf(a[e], b[e], d);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        if ((lane & 15) == 0) row_delta[warp * 8 + 2 * k + (lane >> 4)] = d;
      }
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kRowWarps * 32) : "memory");  // nothing above waits: all of them come
    float delta = row_delta[r];
    float2 rest = make_float2(0.f, 0.f);  // sum of ds, in two parts
    bool ok = true;
    for (int i = 0; i < tiles; ++i) {
      ok = __all_sync(0xffffffffu, wait(s_full, i));
      if (!ok) break;
      tc_fence_after();
      float prob[kPart];
      load_part(t_s + lanes + part * kPart, prob);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_read);
      const int64_t key0 = static_cast<int64_t>(i) * kTile;
      const bool masked = (p.causal && key0 == row0) || key0 + kTile > length;
      const int here = masked ? static_cast<int>((p.causal && live ? row0 + r + 1 : length) - key0) - part * kPart : kPart;
#pragma unroll
      for (int k = 0; k < kPart; k += 2) {
        const float2 y = fma2(make_float2(prob[k], prob[k + 1]), make_float2(sl2, sl2), make_float2(-lse2, -lse2));
        prob[k] = pow2(y.x), prob[k + 1] = pow2(y.y);
      }
      if (masked) {
#pragma unroll
        for (int k = 0; k < kPart; ++k) prob[k] = k < here ? prob[k] : 0.f;
      }
      ok = __all_sync(0xffffffffu, wait(&dp_full[i & 1], i >> 1));
      if (!ok) break;
      tc_fence_after();
      const uint32_t t = t_dp + (i & 1) * kTile + lanes + part * kPart;
      float dp[kPart];
      load_part(t, dp);
      if (tiles == 1) {
        // All keys of these rows are at hand: the whole D before the first ds.
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kPart; ++k) sum += k < here ? prob[k] * (dp[k] - delta) : 0.f;
        exchange[part * kTile + r] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(exchanged);
        ok = __all_sync(0xffffffffu, wait(exchanged, 0));
        if (!ok) break;
        delta += (exchange[r] + exchange[kTile + r]) + (exchange[2 * kTile + r] + exchange[3 * kTile + r]);
      }
      if (masked) {  // ds = 0 whatever dout . v is there
#pragma unroll
        for (int k = 0; k < kPart; ++k) dp[k] = k < here ? dp[k] : delta;
      }
      uint32_t half[16];
#pragma unroll
      for (int k = 0; k < kPart; k += 2) {
        float2 ds = add2(make_float2(dp[k], dp[k + 1]), make_float2(-delta, -delta));
        ds = mul2(ds, make_float2(prob[k], prob[k + 1]));
        rest = add2(rest, ds);
        half[k / 2] = pack_bf16(ds.x, ds.y);
      }
      tmem_st16(t, half);  // over columns that have been read
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ds_full[i & 1]);
    }
    if (ok) ok = __all_sync(0xffffffffu, wait(done, 0));
    if (ok && tiles > 1) {
      exchange[part * kTile + r] = rest.x + rest.y;
      __syncwarp();
      if (lane == 0) mbar_arrive(exchanged);
      ok = __all_sync(0xffffffffu, wait(exchanged, 0));
      if (ok) delta += (exchange[r] + exchange[kTile + r]) + (exchange[2 * kTile + r] + exchange[3 * kTile + r]);
    }
    if (ok) {
      tc_fence_after();
      if (live && part == 0) p.delta[static_cast<int64_t>(head) * p.n + token] = delta;
      const int64_t first = row0 + (warp & 3) * 32, left = length - first;
      if (part * kPart < kD && left > 0)  // over keys, which no product reads any more
        store_block<kPart>(keys + warp * 64 * kPart, t_dq + lanes + part * kPart, p.scale,
                           out_at(p.dq, begin + first, head) + part * kPart, p.dq.token,
                           static_cast<int>(left < 32 ? left : 32), p.dim - part * kPart);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 17) tmem_dealloc(0, kCols);
}

template <int kD>
__global__ void __launch_bounds__(Bwd<kD>::kThreads, 1) attention_dkv_kernel(const __grid_constant__ AttentionLaunch p) {
  using F = Bwd<kD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *queries = smem + 2 * F::kTileBytes, *dout = queries + F::kQuerySlots * F::kTileBytes;  // behind keys and values
  const uint32_t k_at = (smem_u32(smem_raw) + 1023) & ~1023u, v_at = k_at + F::kTileBytes, queries_at = v_at + F::kTileBytes,
                 dout_at = queries_at + F::kQuerySlots * F::kTileBytes;
  uint8_t* strips = dout + F::kTileBytes;  // ones; two stages of -lse / scale and -D of the queries
  const uint32_t ones_at = dout_at + F::kTileBytes;
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(strips + 5 * kStripBytes);
  uint64_t* q_full = kv_full + 1;
  uint64_t* q_empty = q_full + F::kQuerySlots;
  uint64_t* do_full = q_empty + F::kQuerySlots;
  uint64_t* do_empty = do_full + 1;
  uint64_t* st_full = do_empty + 1;
  uint64_t* st_empty = st_full + 2;
  uint64_t* s_full = st_empty + 2;
  uint64_t* p_full = s_full + 1;
  uint64_t* dp_full = p_full + 1;
  uint64_t* ds_full = dp_full + 1;
  uint64_t* done = ds_full + 1;
  uint64_t* drain = done + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ Place place;

  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int kv = blockIdx.x % p.kv_heads, group = p.heads / p.kv_heads;
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    for (int s = 0; s < F::kQuerySlots; ++s) mbar_init(&q_full[s], 1), mbar_init(&q_empty[s], 1);
    for (int s = 0; s < 2; ++s) mbar_init(&st_full[s], 1), mbar_init(&st_empty[s], 1);
    mbar_init(do_full, 1), mbar_init(do_empty, 1);
    mbar_init(s_full, 1), mbar_init(p_full, kRowWarps), mbar_init(dp_full, 1), mbar_init(ds_full, kRowWarps);
    mbar_init(done, 1), mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  griddep_wait();
  if (warp == 17) {
    const Place found = find_tile(p, blockIdx.x / p.kv_heads);
    if (lane == 0) place = found;
    if (found.length > 0) tmem_alloc(tmem_slot, kCols);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const int64_t begin = place.begin, length = place.length;
  if (length == 0) {
    if (warp == 0) zero_rows_outside(p, p.dk, p.kv_heads, nullptr), zero_rows_outside(p, p.dv, p.kv_heads, nullptr);
    return;
  }
  constexpr uint32_t t_s = 0, t_dp = kTile, t_dv = 2 * kTile, t_dk = 3 * kTile;
  const int64_t blocks = (length + kTile - 1) / kTile, key0 = place.piece * kTile, first = p.causal ? place.piece : 0;
  const int per_head = static_cast<int>(blocks - first);  // tiles of queries
  const int64_t tiles = static_cast<int64_t>(per_head) * group;
  const bool ragged = length % kTile != 0;  // a head's last tile of queries has rows of other sequences
  auto wait = [&](uint64_t* bar, int64_t phase) { return wait_fast(bar, static_cast<uint32_t>(phase) & 1u, abort_flag, p.status); };

  if (warp == 16) {
    // ------------------------------------------------------------------ copies
    if (lane == 0) {
      mbar_arrive_expect_tx(kv_full, 2 * F::kTileBytes);
      load_tile<kD>(k_at, &p.map_k, kv, begin + key0, kv_full);
      load_tile<kD>(v_at, &p.map_v, kv, begin + key0, kv_full);
      // The queries of a tile are there a tile earlier than its dout, which the next one's replaces as soon as dv has it.
      int64_t i = 0, loaded = 0;
      bool ok = true;
      int h = 0, b = 0, slot = 0;
      uint32_t phase = 0;
      auto next_queries = [&] {
        if (loaded == tiles) return true;
        if (!wait(&q_empty[slot], phase ^ 1u)) return false;
        mbar_arrive_expect_tx(&q_full[slot], F::kTileBytes);
        load_tile<kD>(queries_at + slot * F::kTileBytes, &p.map_q, kv * group + h, begin + (first + b) * kTile, &q_full[slot]);
        if (++b == per_head) b = 0, ++h;
        if (++slot == F::kQuerySlots) slot = 0, phase ^= 1u;
        ++loaded;
        return true;
      };
      ok = next_queries();
      for (int ho = 0, bo = 0; ok && i < tiles; ++i) {
        if (!(ok = next_queries()) || !(ok = wait(do_empty, i + 1))) break;
        mbar_arrive_expect_tx(do_full, F::kTileBytes);
        load_tile<kD>(dout_at, &p.map_dout, kv * group + ho, begin + (first + bo) * kTile, do_full);
        if (++bo == per_head) bo = 0, ++ho;
      }
      if (!ok || *abort_flag) {
        wait_bounded(kv_full, 0, abort_flag, p.status, kDrainLimitNs, false);
        for (int64_t t = loaded > F::kQuerySlots ? loaded - F::kQuerySlots : 0; t < loaded; ++t)
          wait_bounded(&q_full[t % F::kQuerySlots], (t / F::kQuerySlots) & 1, abort_flag, p.status, kDrainLimitNs, false);
        if (i > 0) wait_bounded(do_full, (i - 1) & 1, abort_flag, p.status, kDrainLimitNs, false);
      }
    }
    __syncwarp();
    zero_rows_outside(p, p.dk, p.kv_heads, nullptr);
    zero_rows_outside(p, p.dv, p.kv_heads, nullptr);
  } else if (warp == 17) {
    // ------------------------------------------------------------------ products
    const int each = __shfl_sync(0xffffffffu, per_head, 0);
    const int64_t n = static_cast<int64_t>(each) * group;
    const bool cut = __any_sync(0xffffffffu, ragged);
    auto all_wait = [&](uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };
    int left = each, left_do = each;  // tiles to come of the head whose scores, whose dout . v are formed next
    // A head's last tile of queries may end in rows of other sequences: whatever they hold meets p and ds of 0, and must be
    // 0 too.
    const int valid = __shfl_sync(0xffffffffu, static_cast<int>(length - (blocks - 1) * kTile), 0);
    int qs = 0;  // slot of the next scores
    uint32_t q_phase = 0;
    auto scores = [&](uint32_t turn, int stage) {
      if (!all_wait(&q_full[qs], q_phase) || !all_wait(&st_full[stage], turn >> 1)) return false;
      if (--left == 0) {
        left = each;
        if (cut) clear_rows<kD>(queries + qs * F::kTileBytes, valid);
        __syncwarp();
      }
      tc_fence_after();
      mma_rows<kD>(t_s, k_at, queries_at + qs * F::kTileBytes);
      mma_strips(t_s, ones_at, ones_at + (1 + 2 * stage) * kStripBytes);
      mma_commit_elected(s_full);
      if (++qs == F::kQuerySlots) qs = 0, q_phase ^= 1u;
      return true;
    };
    auto along = [&](uint32_t turn, int stage) {
      if (!all_wait(do_full, turn)) return false;
      if (--left_do == 0) {
        left_do = each;
        if (cut) clear_rows<kD>(dout, valid);
        __syncwarp();
      }
      tc_fence_after();
      mma_rows<kD>(t_dp, v_at, dout_at);
      mma_strips(t_dp, ones_at, ones_at + (2 + 2 * stage) * kStripBytes);
      mma_commit_elected(dp_full);
      mma_commit_elected(&st_empty[stage]);
      return true;
    };
    bool ok = all_wait(kv_full, 0) && scores(0, 0) && along(0, 0);
    int slot = 0;  // of the queries that dk takes next
    uint32_t turn = 0;  // the tile, modulo 4
    for (int64_t i = 0; ok && i < n; ++i) {
      const uint32_t turn1 = (turn + 1) & 3;
      if (!(ok = all_wait(p_full, turn))) break;
      tc_fence_after();
      mma_columns<kD, true>(t_dv, t_s, dout_at, i > 0);
      mma_commit_elected(do_empty);
      if (i + 1 < n && !(ok = scores(turn1, turn1 & 1))) break;
      if (!(ok = all_wait(ds_full, turn))) break;
      tc_fence_after();
      mma_columns<kD, true>(t_dk, t_dp, queries_at + slot * F::kTileBytes, i > 0);
      mma_commit_elected(&q_empty[slot]);
      if (i + 1 == n) mma_commit_elected(done);
      if (i + 1 < n) ok = along(turn1, turn1 & 1);
      if (++slot == F::kQuerySlots) slot = 0;
      turn = turn1;
    }
    if (elect_one()) {
      mma_commit(drain);
      wait_bounded(drain, 0, abort_flag, p.status, kDrainLimitNs, false);
    }
  } else if (warp == 18) {
    // ------------------------------------------------------------------ the queries' lse and D
    // They enter the products as one more step of 16 columns, 1 for each key and the value in three bf16 terms for the
    // query: a thread has a key's row, so it would have to read every query's value from shared memory, whose time the
    // products need (1024 of 2800 cycles of a tile). The values are asked for a tile ahead.
    bool ok = true;
    float lse[4], delta[4];
    const float by = -1.f / p.scale;
    for (int k = lane; k < 5 * kStripBytes / 16; k += 32) {
      const bool one = k < kStripBytes / 16 && (k & 15) < 8;
      *reinterpret_cast<uint4*>(strips + k * 16) = make_uint4(one ? 0x3f803f80u : 0u, one ? 0x00003f80u : 0u, 0u, 0u);
    }
    int h1 = 0, b1 = 0;  // the next tile
    auto fetch = [&] {
      const int64_t row = (first + b1) * kTile, list = static_cast<int64_t>(kv * group + h1) * p.n + begin;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int64_t q = row + lane + 32 * k;
        const bool live = q < length;
        lse[k] = live ? p.lse[list + q] : 0.f;
        delta[k] = live ? p.delta[list + q] : 0.f;
      }
      if (++b1 == per_head) b1 = 0, ++h1;
    };
    fetch();
    for (int64_t i = 0, b = 0; i < tiles; ++i) {
      const int s = static_cast<int>(i & 1);
      ok = __all_sync(0xffffffffu, wait(&st_empty[s], (i >> 1) + 1));
      if (!ok) break;
      const bool last = ++b == per_head;
      const int valid = ragged && last ? static_cast<int>(length - (blocks - 1) * kTile) : kTile;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // A query behind the sequence has p = 2^(0 - infinity) = 0.
        const int q = lane + 32 * k;
        store_strip(strips + (1 + 2 * s) * kStripBytes, q, q < valid ? lse[k] * by : p.scale < 0.f ? INFINITY : -INFINITY);
        store_strip(strips + (2 + 2 * s) * kStripBytes, q, -delta[k]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&st_full[s]);
      if (i + 1 < tiles) fetch();
      if (last) b = 0;
    }
  } else {
    // ------------------------------------------------------------------ rows
    const int part = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float sl2 = p.scale * kLog2e;
    bool ok = true;
    int left = 0;
    for (int64_t i = 0; i < tiles; ++i) {
      const bool diagonal = p.causal && left == 0;  // a head's first tile of queries is that of the keys
      left = left == 0 ? per_head - 1 : left - 1;
      ok = __all_sync(0xffffffffu, wait(s_full, i));
      if (!ok) break;
      tc_fence_after();
      float prob[kPart];
      load_part(t_s + lanes + part * kPart, prob);
#pragma unroll
      for (int k = 0; k < kPart; k += 2) {
        const float2 y = mul2(make_float2(prob[k], prob[k + 1]), make_float2(sl2, sl2));  // (x - lse) log2(e)
        prob[k] = pow2(y.x), prob[k + 1] = pow2(y.y);
      }
      const int from = diagonal ? r - part * kPart : 0;  // the queries before the key do not meet it
      if (diagonal) {
#pragma unroll
        for (int k = 0; k < kPart; ++k) prob[k] = k < from ? 0.f : prob[k];
      }
      uint32_t half[16];
#pragma unroll
      for (int k = 0; k < kPart; k += 2) half[k / 2] = pack_bf16(prob[k], prob[k + 1]);
      tmem_st16(t_s + lanes + part * kPart, half);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
      ok = __all_sync(0xffffffffu, wait(dp_full, i));
      if (!ok) break;
      tc_fence_after();
      const uint32_t t = t_dp + lanes + part * kPart;
      float dp[kPart];
      load_part(t, dp);
      if (diagonal) {  // ds = 0 whatever dout . v is there
#pragma unroll
        for (int k = 0; k < kPart; ++k) dp[k] = k < from ? 0.f : dp[k];
      }
#pragma unroll
      for (int k = 0; k < kPart; k += 2) {
        const float2 ds = mul2(make_float2(dp[k], dp[k + 1]), make_float2(prob[k], prob[k + 1]));
        half[k / 2] = pack_bf16(ds.x, ds.y);
      }
      tmem_st16(t, half);  // over columns that have been read
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (ok) ok = __all_sync(0xffffffffu, wait(done, 0));
    if (ok) {
      tc_fence_after();
      // Two parts store dv, two dk, half of the columns each; over keys and values, which no product reads any more.
      constexpr int kCols = kD / 2;
      const bool is_key = part >= 2;
      const int c = (part & 1) * kCols;
      const int64_t first_key = key0 + (warp & 3) * 32, left_keys = length - first_key;
      if (left_keys > 0)
        store_block<kCols>(smem + warp * 64 * kCols, (is_key ? t_dk : t_dv) + lanes + c, is_key ? p.scale : 1.f,
                           out_at(is_key ? p.dk : p.dv, begin + first_key, kv) + c, is_key ? p.dk.token : p.dv.token,
                           static_cast<int>(left_keys < 32 ? left_keys : 32), p.dim - c);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 17) tmem_dealloc(0, kCols);
}

// ---------------------------------------------------------------------------- launches

// Pieces that the sequences have: of equal ones exactly; of others at most, each having one more than its tokens fill.
int64_t tiles_of(const AttentionLaunch& p) {
  if (!p.offsets) return p.sequences * ((p.n / p.sequences + kTile - 1) / kTile);
  return std::max<int64_t>(1, p.n / kTile + std::min(p.sequences, p.n));
}

constexpr int kMaxDevices = 64;

// Heads are neighbours in the grid: the longest rows of all of them start first. `known`: the devices on which the
// kernel's shared memory has been asked for (the caller holds the library's lock).
template <typename K>
cudaError_t launch_tiles(K* kernel, bool (&known)[kMaxDevices], AttentionLaunch& p, int64_t slots, int heads, int threads,
                         int smem, cudaStream_t stream) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kMaxDevices || !known[dev]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices) known[dev] = true;
  }
  return row::launch(kernel, dim3(static_cast<unsigned>(slots * heads)), threads, smem, stream, p);
}

template <int kD>
cudaError_t launch_forward(AttentionLaunch& p, cudaStream_t stream) {
  using F = Fwd<kD>;
  const int64_t group = p.heads / p.kv_heads;
  // Pairs of units; with offsets every sequence may leave half a pair.
  int64_t slots = 0;
  if (!p.offsets) slots = p.sequences * (((p.n / p.sequences + kTile - 1) / kTile * group + 1) / 2);
  else slots = (tiles_of(p) * group + std::min(p.sequences, p.n)) / 2 + 1;
  static bool known[kMaxDevices];
  return launch_tiles(attention_kernel<kD>, known, p, slots, p.kv_heads, F::kThreads, F::kSmem, stream);
}

template <int kD>
cudaError_t launch_backward(AttentionLaunch& p, cudaStream_t stream) {
  using F = Bwd<kD>;
  static bool known[2][kMaxDevices];
  const cudaError_t e =
      launch_tiles(attention_dq_kernel<kD>, known[0], p, tiles_of(p), p.heads, F::kThreads, F::kSmemQueries, stream);
  if (e != cudaSuccess) return e;
  return launch_tiles(attention_dkv_kernel<kD>, known[1], p, tiles_of(p), p.kv_heads, F::kThreads, F::kSmemKeys, stream);
}

cudaError_t set_maps(AttentionLaunch& p) {
  const char* why = nullptr;
  p.scale_log2 = fabsf(p.scale) * kLog2e;
  if (!encode_heads(&p.map_q, p.q, p.dim, p.heads, p.n, kTile, &why) ||
      !encode_heads(&p.map_k, p.k, p.dim, p.kv_heads, p.n, kTile, &why) ||
      !encode_heads(&p.map_v, p.v, p.dim, p.kv_heads, p.n, kTile, &why) ||
      (p.dout.data && !encode_heads(&p.map_dout, p.dout, p.dim, p.heads, p.n, kTile, &why)))
    return cudaErrorInvalidValue;
  return cudaSuccess;
}

}  // namespace

int64_t attention_workspace(AttentionLaunch& p, char* ws) {
  if (ws) p.delta = reinterpret_cast<float*>(ws);
  return static_cast<int64_t>(sizeof(float)) * p.n * p.heads;
}

cudaError_t launch_attention(AttentionLaunch& p, cudaStream_t stream) {
  const cudaError_t e = set_maps(p);
  if (e != cudaSuccess) return e;
  return p.dim <= 64 ? launch_forward<64>(p, stream) : launch_forward<128>(p, stream);
}

cudaError_t launch_attention_grad(AttentionLaunch& p, cudaStream_t stream) {
  const cudaError_t e = set_maps(p);
  if (e != cudaSuccess) return e;
  return p.dim <= 64 ? launch_backward<64>(p, stream) : launch_backward<128>(p, stream);
}

}  // namespace dmuon
