// Attention of several query tokens of each sequence over its paged rows (aircache_paged_attend).
//
//   x_j = scale q . k_j for the rows j that the token sees,  o = sum_j exp(x_j - m) v_j / l,  l = sum_j exp(x_j - m).
//
// 4 D operations for each (token, query head, row): bound by the matrix units where a sequence has many tokens, by HBM
// where it has few.  The query heads of a KV head are packed: 128 query rows are floor(128 / g) tokens with their g
// heads, so that one tile of keys and values serves them all.
//
// A unit of work is a KV head and up to two such query tiles ("streams") of one sequence, over the 128-row key tiles
// that any of its tokens sees.  With more tokens than a tile holds, the streams are two query tiles that take the same
// keys in turn (wide); with fewer, they are one query tile whose key tiles go to the streams alternately (narrow), and
// their results are joined at the end.  Either way one stream's softmax runs while the tensor cores work for the other.
// The units lie on a line, each with its key tiles and some places for its end, and every CTA takes an equal run of it
// (one CTA to an SM, persistent): ragged batches and long rows leave no SM idle.  Units that a run's border cuts leave
// their parts in the workspace, and a second kernel joins them in the order of the CTAs.
//
// In a CTA: two groups of four softmax warps, one to a stream; a warp to each stream's MMAs; one that copies keys and
// values (TMA, boxes of as many rows as divide a page and 128, into a ring of tiles); one that brings queries and clears
// the value rows behind the sequence's last (a weight of 0 times whatever a page holds there could be NaN).  S = Q K^T
// goes to a TMEM buffer per stream; a softmax thread owns a row of it (its TMEM lane), takes it to registers whole, and
// writes the weights as bf16 over the buffer's first half, from where the next MMA takes them as its A operand: O += P V
// accumulates in TMEM.  The product begins when half of the weights are there.  The reference of the exponentials moves
// only when a row's maximum passes it by 2^8; then O is rescaled in place, which nothing else touches in between because
// a thread's MMAs run in order.  The streams' bursts of MMAs take turns: side by side each would take twice as long, and
// both softmaxes would wait for both.
//
// What the loop is bound by, at 128-wide heads: 2,048 cycles of the tensor cores for a tile of keys and two streams, 1,190
// of the exponentials (4.6 cycles to a warp's), and the chain of a stream: its softmax (1,350 cycles alone, 2,100 beside
// the other's), half of P V, S and the waits between them.  A tile takes 3,000 cycles (tensor pipe 65 to 67 % active).
// Why it is built so (1,000 tokens over 130,000 rows, 28 to 4 heads, each beside what it replaced on one machine): MMA
// operands in a warp's uniform registers take a sixth less time than one lane's branch, a warp to each stream's MMAs and
// turns 5 % less, a run's description out of the softmax threads' registers 8 %; sixteen softmax warps with half a row
// each, which meet for every maximum, took a third more.
//
// int8 rows: eight more warps widen the codes, exactly, into the bf16 tiles.  The softmax threads multiply logits by the
// keys' scales and weights by the values', which takes 64 logits at a time, twice (3,900 cycles to a tile).  Neither issue
// slots (44 to 47 %), the tensor pipe (13 to 23 %) nor DRAM (7 to 12 %) are at a limit; the loop is 40 % of the time, and
// how starts, ends of units and waits share the rest is not measured.
//
// Weights that meet V are rounded once to bf16 (at most 2^-8 of each weight, independent of one another; the error of an
// output against 64 bits goes from 0.0017 of its norm, its own rounding to bf16, to 0.0023).  For the prefixes of a shared
// decode (FINE) they are a sum of two bf16, 16 bits, as in the decode step that it stands in for (error 0.0017): what the
// first leaves takes the rest of S's columns and a second product.  That is half as much again of P V for the tensor
// cores: 4 x 256 tokens over 12,544 rows would take 205 us instead of 161, a chunk of 1,000 tokens over 130,000 rows 1,895
// instead of 1,440.  Logits, maximum, sum, O, parts and the joins are fp32.
//
// A weight of 0 does not hide a NaN or an infinity in V from a matrix product.  A CTA that finds an output that is not
// finite while its sum is walks over its units a second time: values that are not finite are cleared before the product
// and added to the outputs of the rows that see them, and the weights are 2^-40 of what they were (sums of large values
// may have passed fp32's range; logits minus a reference near 40 are then rounded at 2^-19, weights under 2^-86 are 0).  A
// row that sees none of the run's keys wants no second walk: its part is zeros.  Ragged questions of which every sequence
// holds a NaN take 2.4 ms instead of 0.6; row by row, a warp to an output row, they took a thousand times that.
//
// Measured (28 query and 4 KV heads of 128, bf16, calls back to back, on several machines): 16 ragged questions of up to
// 1,024 tokens behind 576 to 9,000 rows 574 to 631 us (737 GFLOP, 1.2 to 1.3 PFLOP/s); 1,000 tokens over 130,000 rows 1,235
// to 1,472 us; 4 x 256 tokens over 12,544 rows 152 to 164 us; one token of each of 16 sequences over 16,384 rows 97 us (5.6
// TB/s; the decode kernel 87); four drafts of eight chats 14 to 15 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "attend.cuh"
#include "rowmma.cuh"
#include "tmap.cuh"
#include "umma.cuh"

namespace aircache {
namespace {

constexpr int kAtKeys = 128;                  // rows of a key tile
constexpr int kAtRows = 128;                  // query rows of a stream (TMEM lanes)
// Behind the eight softmax warps: the streams' MMA issue (8 and 9), keys and values, queries and tails; from 12 on
// eight that widen int8 codes
constexpr int kAtMma = 8, kAtLoad = 10, kAtAux = 11, kAtWiden = 12;
constexpr uint32_t kAtEnd = 2;                // places of the line for a unit's end
constexpr float kAtSlack = 8.f;               // base-2 powers that a maximum may pass its reference by
constexpr uint32_t kAtS = 0, kAtO = 256;      // TMEM columns: S of stream i at 128 i, O at 256 + 128 i
constexpr int kAtGroup = 16;                  // query heads of a KV head, at most
constexpr int kAtStaged = 4096;               // sequences whose lengths and offsets go through shared memory
constexpr int kAtHeader = 256;                // workspace: error word
constexpr long long kAtLong = 4 * kWaitCycles;  // waits that stand behind another warp's

template <int D, bool Q8>
struct AtCfg {
  static constexpr int kThreads = Q8 ? 640 : 384;
  // registers of a thread: what the other warps give, the softmax warps, which hold a row of 128 logits, take
  static constexpr int kRegs = Q8 ? 96 : 168, kRegsSoft = Q8 ? 144 : 208, kRegsOther = Q8 ? 64 : 88;
  static_assert(256 * kRegsSoft + (kThreads - 256) * kRegsOther <= kThreads * kRegs, "within the launch's own");
  static constexpr int kSlab = kAtKeys * 128;       // [128 rows][64 bf16]
  static constexpr int kTile = kSlab * (D / 64);
  static constexpr int kStages = (Q8 ? 3 : 5) * 128 / D;       // tiles of the ring
  static constexpr int kCodeTile = kAtKeys * D;                // int8 rows: tiles of codes before them,
  static constexpr int kCodeStages = Q8 ? (D == 128 ? 3 : 5) : 0;
  static constexpr int kScaleStages = Q8 ? 4 : 0;              // and the scales of a tile's keys and values: as they
                                                               // come, then as the softmax takes them
  // (a tile's values are widened before its stage of scales can be another's: five entries or more lie between)
  static_assert(kCodeStages <= 5);
  static constexpr int kOffQ = 0;                              // two query tiles
  static constexpr int kOffRing = 2 * kTile;
  static constexpr int kOffCodes = kOffRing + kStages * kTile;
  static constexpr int kOffScales = kOffCodes + kCodeStages * kCodeTile;
  static constexpr int kOffCtl = kOffScales + kScaleStages * 4 * kAtKeys * 4;
};

// A unit whose parts are to be joined (parts < 2: none): of CTAs c0 .. c0 + parts - 1.
struct alignas(16) AtCut {
  int parts, c0, h, ntok;
  int64_t token0;
  int slot, pad;
};

// x / d for 0 <= x < 2^31 and 1 <= d <= 2^30: with 2^(L-1) < d <= 2^L, M = ceil(2^(31 + L) / d) <= 2^32 - 1 and
// M d - 2^(31 + L) < d, so that x M / 2^(31 + L) passes x / d by less than 1 / d.
struct AtDivisor {
  uint32_t m;
  int shift;
  __host__ __device__ __forceinline__ int quotient(int x) const { return (int)(((uint64_t)(uint32_t)x * m) >> shift); }
};
inline AtDivisor divisor(int d) {
  int shift = 31;
  while ((1ll << (shift - 31)) < d) ++shift;
  return {(uint32_t)(((1ull << shift) + d - 1) / d), shift};
}

struct AtRun;
struct AtArgs {
  Pages pages;
  const int32_t* cu;
  const int32_t* row_begin;
  const int32_t* row_end;
  __nv_bfloat16* out;
  int64_t out_stride_tok, out_stride_head;
  float* lse;
  AttendPart part;
  int32_t* error;
  AtCut* cut;       // [CTAs]: the unit that begins in the CTA and ends in another
  AtRun* start;      // [CTAs]: where each begins
  int2* range;      // [slots]: the key tiles that a unit's tokens see (with row_begin or row_end)
  float2* part_ml;  // [2 CTAs][rows_cap]
  float* part_o;    // [2 CTAs][rows_cap][D]
  int64_t num_tokens;
  AtDivisor by_unit, by_page, by_group, by_cta;  // by 2 tok_tile, page_rows / 16, group, ctas
  int slots, group, tok_tile, h_q, causal, rows_cap, ctas;
  int box_shift;  // boxes of 2^box_shift rows
  int ranged;     // a kernel has filled `range`; otherwise every CTA does, with the same
  int few;        // every CTA's warps place the batch by themselves: at most 32 units to a KV head, fewer than 2^31 places
  float scale_log2;
};

// D[tmem] (+)= A[tmem] * B[smem]: A is M rows (lanes) of 16-bit elements, two to a column.
__device__ __forceinline__ void umma_bf16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int a, int b, int c, int d, int e,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
      "{%2, %3, %4, %5, %6}], [%7];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(smem_u32(bar))
      : "memory");
}
// Two fp32 multiply-adds and additions in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("add.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= FLT_MAX; }
// True for one lane of the warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("mul.rn.f32x2 %0, %1, %2;\n"
      : "=l"(reinterpret_cast<uint64_t&>(r))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return r;
}
// Logits of 32 keys from `at` on: those outside [from, from + wide) become -inf.  By a warp, each lane its own row's.
__device__ __forceinline__ void mask32(float v[32], int from, uint32_t wide, int at) {
  const int lo = min(max(from - at, 0), 32);
  const int hi = (int)min(max((int64_t)from + wide - at, (int64_t)0), (int64_t)32);
  const uint32_t in = (uint32_t)(((1ull << hi) - 1) & ~((1ull << lo) - 1));
  if (__all_sync(0xffffffffu, in == 0xffffffffu)) return;
#pragma unroll
  for (int c = 0; c < 32; ++c) v[c] = in >> c & 1 ? v[c] : -INFINITY;
}
// Arrives where `on` says so, without a branch: the lanes stay together.
__device__ __forceinline__ void mbar_arrive_if(bool on, uint64_t* bar) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %1, 0;\n @p mbarrier.arrive.shared::cta.b64 _, [%0];\n}\n" ::"r"(
                   smem_u32(bar)),
               "r"((uint32_t)on)
               : "memory");
}
// Arrives `n` times.
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
// Two int8 codes (the bytes that `sel` picks) as two bf16, exactly: the low seven bits in the mantissa of 128 are
// 128 + (c mod 128), and 128 is taken away again, or 256 where the sign bit is set.
__device__ __forceinline__ uint32_t widen2_bf16(uint32_t c4, uint32_t sel) {
  const uint32_t t = __byte_perm(c4, 0x43434343u, sel);
  const uint32_t x = t & 0xff7fff7fu, y = (t & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 r = __hsub2(reinterpret_cast<const __nv_bfloat162&>(x), reinterpret_cast<const __nv_bfloat162&>(y));
  return reinterpret_cast<const uint32_t&>(r);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What is left of two weights when the bf16 pair `w` has been taken away, as bf16 again.
__device__ __forceinline__ uint32_t rest2(float2 e, uint32_t w) {
  const float2 r = fma2(make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), make_float2(-1.f, -1.f), e);
  return pack2(r.x, r.y);
}

// ------------------------------------------------------------------ the line of units

// Tokens of a unit for one KV head, and the key tiles that any of them sees.
struct AtUnit {
  int s, tok0, ntok, n;  // sequence, first token of it, tokens, the sequence's tokens
  int rows, t0, c;       // its rows, first key tile, key tiles
  int token0;            // the batch's token of tok0
};
// Units of sequence s start at slot cu[s] / (2 tok_tile) + s: never less than the units before it, so that a slot's
// sequence is found without a sum over the batch, and at most num_seqs slots are empty.
struct AtSeqs {
  const int32_t* cu;
  const int32_t* lens;
};
__device__ __forceinline__ AtSeqs seqs_of(const AtArgs& a) { return {a.cu, a.pages.lens}; }
__device__ __forceinline__ int slot_base(const AtArgs& a, int c0, int s) {
  return a.by_unit.quotient(min(max(c0, 0), (int)a.num_tokens)) + s;
}
__device__ __forceinline__ int find_seq(const AtArgs& a, const AtSeqs& q, int slot) {
  int lo = 0, hi = a.pages.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (slot_base(a, q.cu[mid], mid) <= slot)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}
// Rows [lo, hi) that token i (of the sequence; `token` of the batch) sees.
__device__ __forceinline__ void token_rows(const AtArgs& a, int rows, int n, int i, int64_t token, int& lo, int& hi) {
  lo = 0;
  hi = a.causal ? max(rows - n + i + 1, 0) : rows;
  if (a.row_begin) lo = max(lo, a.row_begin[token]);
  if (a.row_end) hi = min(hi, a.row_end[token]);
  if (hi <= lo) lo = hi = 0;
}
// The unit of `slot` in sequence s, whose tokens are c0 .. c1 - 1 and whose rows len; ntok = 0 when there is none.
// range: where the units' key tiles are listed, if tokens have ranges of their own.
__device__ __forceinline__ AtUnit make_unit(const AtArgs& a, int s, int slot, int c0, int c1, int len, const int2* range) {
  AtUnit u;
  u.s = s;
  u.n = c0 >= 0 && c1 >= c0 && c1 <= a.num_tokens ? c1 - c0 : 0;
  u.rows = len >= 0 && len <= a.pages.max_rows ? len : 0;
  const int64_t first = (int64_t)(slot - slot_base(a, c0, s)) * (2 * a.tok_tile);
  const bool in = first >= 0 && first < u.n;
  u.tok0 = in ? (int)first : 0;
  u.ntok = in ? min(2 * a.tok_tile, u.n - u.tok0) : 0;
  u.token0 = in ? c0 + u.tok0 : 0;
  u.t0 = u.c = 0;
  if (in) {
    if (range) {
      const int2 r = range[slot];
      u.t0 = r.x;
      u.c = r.y - r.x;
    } else {
      const int hi = a.causal ? max(u.rows - u.n + u.tok0 + u.ntok, 0) : u.rows;
      u.c = (int)(((int64_t)hi + kAtKeys - 1) / kAtKeys);
    }
  }
  return u;
}
__device__ __forceinline__ AtUnit unit_of(const AtArgs& a, const AtSeqs& q, int s, int slot, const int2* range) {
  return make_unit(a, s, slot, q.cu[s], q.cu[s + 1], q.lens[s], range);
}

// A unit's key tiles by its tokens' own ranges, by a warp.
__device__ __forceinline__ void find_range(const AtArgs& a, const AtSeqs& q, int slot) {
  const AtUnit u = unit_of(a, q, find_seq(a, q, slot), slot, nullptr);
  int from = INT32_MAX, to = 0;
  for (int i = threadIdx.x & 31; i < u.ntok; i += 32) {
    int lo, hi;
    token_rows(a, u.rows, u.n, u.tok0 + i, u.token0 + i, lo, hi);
    if (hi > lo) from = min(from, lo), to = max(to, hi);
  }
  from = __reduce_min_sync(0xffffffffu, from);
  to = __reduce_max_sync(0xffffffffu, to);
  if ((threadIdx.x & 31) == 0) a.range[slot] = to > 0 ? make_int2(from / kAtKeys, (to - 1) / kAtKeys + 1) : make_int2(0, 0);
}

// A CTA's places of the line, and the walk over the units in them.
struct AtRun {
  uint64_t at;               // the unit's first place
  int slot, h;
  AtUnit u;
  int first, count;          // the CTA's key tiles of the unit, from u.t0 on
};
__device__ __forceinline__ void clip(AtRun& r, uint64_t per) {  // per: places of a CTA
  const uint64_t lo = per * blockIdx.x, from = max(r.at, lo), to = min(r.at + r.u.c, lo + per);
  r.first = (int)(min(from, r.at + r.u.c) - r.at);
  r.count = to > from ? (int)(to - from) : 0;
}
// (`r` is the warp's: every lane reads before any writes the same over it)
__device__ __forceinline__ bool next_unit(const AtArgs& a, AtRun& r, uint64_t per) {
  __syncwarp();
  const uint64_t at = r.at + r.u.c + kAtEnd;
  const int h = r.h + 1, s0 = r.u.s;
  int slot = r.slot;
  __syncwarp();
  if (at >= per * (blockIdx.x + 1)) return false;
  if (h == a.pages.h_kv) {
    AtUnit u;
    int s = s0;
    do {
      if (++slot >= a.slots) return false;
      while (s + 1 < a.pages.num_seqs && slot_base(a, a.cu[s + 1], s + 1) <= slot) ++s;
      u = unit_of(a, seqs_of(a), s, slot, a.range);
    } while (u.ntok == 0);
    r.u = u;
    r.slot = slot;
  }
  r.h = h == a.pages.h_kv ? 0 : h;
  r.at = at;
  clip(r, per);
  __syncwarp();
  return true;
}
// A unit that fits one query tile takes its key tiles alternately with both streams.
__device__ __forceinline__ bool narrow(const AtArgs& a, const AtUnit& u) { return u.ntok <= a.tok_tile; }
// Key tiles of stream i in a run.
__device__ __forceinline__ int stream_tiles(bool nar, int count, int i) { return nar ? (count + 1 - i) / 2 : count; }

// Ring entry pos of a run: whether it is a tile of values, and which of the run's tiles.  Wide: K0 V0 K1 V1 ..; narrow:
// K0 K1 V0 K2 V1 .. (the streams' first logits come before the first weights).
__device__ __forceinline__ bool entry_of(bool nar, int count, int pos, int& j) {
  bool val;
  if (!nar) {
    val = pos & 1;
    j = pos >> 1;
  } else if (pos == 2 * count - 1) {
    val = true;
    j = count - 1;
  } else {
    val = pos > 0 && !(pos & 1);
    j = val ? pos / 2 - 1 : (pos + 1) / 2;
  }
  return val;
}

struct AtScratch {
  uint64_t sum[24];
  AtRun run;
};
template <int D, bool Q8>
struct AtCtl {
  using C = AtCfg<D, Q8>;
  static constexpr int kCodes = Q8 ? C::kCodeStages : 1, kScales = Q8 ? C::kScaleStages : 1;
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t tail[C::kStages];  // of a stage that holds values to be cleared in part: its copies have landed
  uint64_t cfull[kCodes], cempty[kCodes], scfull[kScales], scready[kScales], scempty[kScales];
  uint64_t qfull, qempty, turn[2], sfull[2], phalf[2], pfull[2], ofull[2], mlfull, mlfree, done, again;
  uint32_t tmem;
  uint32_t odd[C::kStages];  // second walk: bit q: rows 4 q .. 4 q + 3 of a stage's values hold any that is not finite
  int bad, stop;             // a row wants the second walk; a warp has given up
  alignas(16) float2 ml[2][kAtRows];  // narrow units: the streams' references and sums of each row
  uint64_t per;        // places of a CTA
  AtRun run[C::kThreads / 32];  // each warp's place: read seldom, not worth registers
};
// (64-bit division takes many times a 32-bit one's time, and is seldom needed)
__device__ __forceinline__ uint64_t quotient(uint64_t x, uint64_t y) {
  return ((x | y) >> 32) == 0 ? (uint32_t)x / (uint32_t)y : x / y;
}
// Few units: every warp finds the CTA's place by itself, a slot to a lane.  Lane s has the offsets c0, c1 of sequence
// s and its length.
__device__ __forceinline__ bool make_run_small(const AtArgs& a, int c0, int c1, int len, uint64_t& share, AtRun& r) {
  const int lane = threadIdx.x & 31;
  const int base = lane < a.pages.num_seqs ? slot_base(a, c0, lane) : INT32_MAX;
  int s = 0;  // the last sequence that starts at the lane's slot or before
#pragma unroll
  for (int step = 16; step > 0; step >>= 1) {
    const int x = __shfl_sync(0xffffffffu, base, s + step);
    if (x <= lane) s += step;
  }
  const int u0 = __shfl_sync(0xffffffffu, c0, s), u1 = __shfl_sync(0xffffffffu, c1, s), ul = __shfl_sync(0xffffffffu, len, s);
  AtUnit u;
  u.ntok = 0;
  if (lane < a.slots) u = make_unit(a, s, lane, u0, u1, ul, a.range);
  const uint32_t wide = u.c + kAtEnd, mine = u.ntok ? wide * a.pages.h_kv : 0;
  uint32_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  const uint32_t total = __shfl_sync(0xffffffffu, incl, 31);
  const uint32_t per = max(2u, (uint32_t)a.by_cta.quotient(total + a.ctas - 1));  // (a narrow unit's streams take a tile each)
  const uint32_t lo = min(per * blockIdx.x, total), hi = min(lo + per, total);
  if (lane == 0) share = per;  // (every warp the same)
  if (lo < hi && lo >= incl - mine && lo < incl) {
    AtRun x;
    x.slot = lane;
    x.h = (int)((lo - (incl - mine)) / wide);
    x.at = incl - mine + x.h * wide;
    x.u = u;
    clip(x, per);
    r = x;
  }
  __syncwarp();
  return lo < hi;
}
// By all threads of the CTA; false if the CTA has no place.
template <int THREADS>
__device__ bool make_run(const AtArgs& a, const AtSeqs& q, AtScratch* sc, uint64_t& share, AtRun& r) {
  static_assert(THREADS <= 768, "warps' sums");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (a.slots + THREADS - 1) / THREADS;
  const int s0 = min(tid * each, a.slots), s1 = min(s0 + each, a.slots);
  uint64_t mine = 0;
  int seq0 = 0;
  if (s0 < s1) {
    int s = seq0 = find_seq(a, q, s0);
    for (int i = s0; i < s1; ++i) {
      while (s + 1 < a.pages.num_seqs && slot_base(a, q.cu[s + 1], s + 1) <= i) ++s;
      const AtUnit u = unit_of(a, q, s, i, a.range);
      if (u.ntok) mine += (uint64_t)(u.c + kAtEnd) * a.pages.h_kv;
    }
  }
  uint64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) sc->sum[warp] = incl;
  __syncthreads();
  uint64_t before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += sc->sum[w];
    total += sc->sum[w];
  }
  const uint64_t per = max((uint64_t)2, quotient(total + gridDim.x - 1, gridDim.x));
  const uint64_t lo = min(per * blockIdx.x, total), hi = min(lo + per, total);
  if (tid == 0) share = per;
  if (lo < hi && lo >= before && lo < before + mine) {
    uint64_t at = before;
    int s = seq0;
    for (int i = s0; i < s1; ++i) {
      while (s + 1 < a.pages.num_seqs && slot_base(a, q.cu[s + 1], s + 1) <= i) ++s;
      const AtUnit u = unit_of(a, q, s, i, a.range);
      if (!u.ntok) continue;
      const uint64_t wide = u.c + kAtEnd;
      if (lo < at + wide * a.pages.h_kv) {
        AtRun x;
        x.slot = i;
        x.h = (int)quotient(lo - at, wide);
        x.at = at + x.h * wide;
        x.u = u;
        clip(x, per);
        sc->run = x;
        break;
      }
      at += wide * a.pages.h_kv;
    }
  }
  __syncthreads();
  if (lo < hi) r = sc->run;
  __syncthreads();  // (what lies in `sc`'s place may come)
  return lo < hi;
}

// ------------------------------------------------------------------ results

// A CTA's part of a unit that began before it lies in slot 2 x CTA, of one that begins in it in the next.  A slot holds
// [D / 4][rows_cap] pieces of four columns, so that a warp's rows are next to one another.
__device__ __forceinline__ int64_t part_slot(int cta, bool begins) { return 2 * (int64_t)cta + (begins ? 1 : 0); }

// The log-sum-exp of a row.
__device__ __forceinline__ void write_lse(const AtArgs& a, int64_t token, int head, float m, float l) {
  const float x = l == 0.f ? -INFINITY : m + log2f(l);
  if (a.part.lse2) a.part.lse2[token * a.h_q + head] = x;
  if (a.lse) a.lse[token * a.h_q + head] = x * 0.69314718055994531f;
}
// E consecutive columns of a row.
template <int D, int E>
__device__ __forceinline__ void write_out(const AtArgs& a, int64_t token, int head, int col, const float* y) {
  if (a.part.out) {
    float* to = a.part.out + (token * a.h_q + head) * D + col;
#pragma unroll
    for (int e = 0; e < E; e += 4) *reinterpret_cast<float4*>(to + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
    return;
  }
  __nv_bfloat16* to = a.out + token * a.out_stride_tok + (int64_t)head * a.out_stride_head + col;
#pragma unroll
  for (int e = 0; e < E; e += 8)
    *reinterpret_cast<uint4*>(to + e) = make_uint4(pack2(y[e], y[e + 1]), pack2(y[e + 2], y[e + 3]),
                                                   pack2(y[e + 4], y[e + 5]), pack2(y[e + 6], y[e + 7]));
}

// ------------------------------------------------------------------ the attention

// Adds the values of row `at` that are not finite (int8: NaN, where the scale is not) to O in a warp's TMEM lanes, of the
// query rows that see it.
template <int D, bool Q8>
__device__ __forceinline__ void add_odd(const AtArgs& a, int s, int h, int at, bool sees, uint32_t o_cols) {
  const Pages& p = a.pages;
  const int at_page = a.by_page.quotient(at >> 4), in_page = at - at_page * p.page_rows;
  const int page = (p.table + (int64_t)s * p.table_stride)[at_page];
  if (!__all_sync(0xffffffffu, page_ok(p, page))) return;
  const float scale = Q8 ? p.v_scale[page_slot(p, page, h, in_page)] : 0.f;
  const __nv_bfloat16* v = reinterpret_cast<const __nv_bfloat16*>(p.v) + (Q8 ? 0 : page_elem(p, page, h, in_page));
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    float x[16], o[16];
    bool any = false;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      x[e] = Q8 ? (finite(scale) ? 0.f : NAN) : __bfloat162float(v[c + e]);
      any |= !finite(x[e]);
    }
    if (!__any_sync(0xffffffffu, any)) continue;
    tmem_ld16(o_cols + c, o);
    tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (sees && !finite(x[e])) o[e] += x[e];
    __syncwarp();
    tmem_st16(o_cols + c, o);
    tmem_wait_st();
  }
}

// FINE: weights meet V as a sum of two bf16, those of 64 keys in 32 columns each.
template <int D, bool Q8, bool FINE>
__global__ void __launch_bounds__(AtCfg<D, Q8>::kThreads, 1) paged_attend_kernel(const __grid_constant__ CUtensorMap qmap,
                                                                     const __grid_constant__ CUtensorMap kmap,
                                                                     const __grid_constant__ CUtensorMap vmap,
                                                                     const __grid_constant__ AtArgs a) {
  using C = AtCfg<D, Q8>;
  using Ctl = AtCtl<D, Q8>;
  extern __shared__ __align__(1024) uint8_t sm[];
  Ctl* ctl = reinterpret_cast<Ctl*>(sm + C::kOffCtl);
  const uint32_t base = smem_u32(sm);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Pages& p = a.pages;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&ctl->full[i], Q8 ? 8 : 1);
      mbar_init(&ctl->empty[i], 2);
      mbar_init(&ctl->tail[i], 1);
    }
    for (int i = 0; i < C::kCodeStages; ++i) {
      mbar_init(&ctl->cfull[i], 1);
      mbar_init(&ctl->cempty[i], 8);
    }
    for (int i = 0; i < C::kScaleStages; ++i) {
      mbar_init(&ctl->scfull[i], 1);
      mbar_init(&ctl->scready[i], 8);
      mbar_init(&ctl->scempty[i], 8);
    }
    mbar_init(&ctl->qfull, 1);
    mbar_init(&ctl->qempty, 2);
    mbar_init(&ctl->mlfull, 8);
    mbar_init(&ctl->mlfree, 8);
    mbar_init(&ctl->done, 2);
    mbar_init(&ctl->again, C::kThreads / 32);
    ctl->bad = ctl->stop = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->sfull[i], 1);
      mbar_init(&ctl->turn[i], 1);
      mbar_init(&ctl->phalf[i], 4);
      mbar_init(&ctl->pfull[i], 4);
      mbar_init(&ctl->ofull[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == kAtMma) {
    __syncwarp();
    tmem_alloc(&ctl->tmem, 512);
    tmem_relinquish();
  }
  if (warp == kAtLoad && lane == 0) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&qmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
  }
  pdl_wait();
  pdl_trigger();
  AtRun& r = ctl->run[warp];
  bool any;
  auto wrong = [&](int c0, int c1, int len) {  // what a batch's description says that cannot be
    return c0 < 0 || c1 < c0 || c1 > a.num_tokens || len < 0 || len > p.max_rows || (a.causal && len < c1 - c0);
  };
  tc_fence_before();
  if (a.few) {
    const bool in = lane < p.num_seqs;
    const int c0 = in ? a.cu[lane] : 0, c1 = in ? a.cu[lane + 1] : 0, len = in ? p.lens[lane] : 0;
    if (blockIdx.x == 0 && warp == 0 && in && wrong(c0, c1, len)) set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
    if (a.range && !a.ranged)
      for (int slot = warp; slot < a.slots; slot += C::kThreads / 32) find_range(a, seqs_of(a), slot);
    __syncthreads();  // (publishes the mbarriers and TMEM too)
    any = make_run_small(a, c0, c1, len, ctl->per, r);
  } else {
    // lengths and token offsets lie where the tiles will until the CTA has found its place: searches go to shared memory
    AtSeqs seqs = seqs_of(a);
    if (p.num_seqs <= kAtStaged) {
      int32_t* lens = reinterpret_cast<int32_t*>(sm);
      int32_t* cu = lens + kAtStaged;
      for (int s = tid; s <= p.num_seqs; s += C::kThreads) {
        cu[s] = a.cu[s];
        if (s < p.num_seqs) lens[s] = p.lens[s];
      }
      seqs = {cu, lens};
      __syncthreads();
    }
    if (blockIdx.x == 0) {
      bool bad = false;
      for (int s = tid; s < p.num_seqs; s += C::kThreads) bad |= wrong(seqs.cu[s], seqs.cu[s + 1], seqs.lens[s]);
      if (bad) set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
    }
    // (its barriers publish the mbarriers and TMEM too)
    any = make_run<C::kThreads>(a, seqs, reinterpret_cast<AtScratch*>(ctl->ml), ctl->per, r);
  }
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  if (any && tid == 0) a.start[blockIdx.x] = r;
  __syncwarp();
  // A warp's next unit.  Behind the last one all warps meet, and walk over the units a second time, with `clean` set, if
  // any row of the first walk wants it
  auto onward = [&](bool& clean) {
    if (next_unit(a, r, ctl->per)) return true;
    if (clean) return false;
    if (lane == 0) mbar_arrive(&ctl->again);
    if (!mbar_wait_warp(&ctl->again, 0, kAtLong)) {
      set_error(a.error, AIRCACHE_ERR_DEVICE_TIMEOUT);
      return false;
    }
    if (!ctl->bad || ctl->stop) return false;
    r = a.start[blockIdx.x];
    __syncwarp();
    return clean = true;
  };
  auto give_up = [&](bool clean) {
    set_error(a.error, AIRCACHE_ERR_DEVICE_TIMEOUT);
    if (lane == 0 && !clean) {
      ctl->stop = 1;
      mbar_arrive(&ctl->again);
    }
    __syncwarp();
  };
  if (warp >= kAtMma) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::kRegsOther));
    if (warp == kAtLoad) {
      // ---- keys and values.  Lane b holds the page of the b-th box of a chunk of 32 boxes (4 to 32 tiles), of the even
      // and the odd chunks: the next chunk's are looked up while this one is copied.  The copies are issued in turn by one
      // lane (issued by a lane each they took four times as long, as their operands are the warp's)
      const int box_shift = a.box_shift, box = 1 << box_shift;
      const int boxes_shift = 7 - box_shift, per_shift = 5 - boxes_shift;  // boxes of a tile, tiles of a chunk
      static_assert(kAtKeys == 128);
      const bool one = elect_one();
      uint32_t n = 0, tiles = 0;  // entries and key tiles so far
      bool ok = true, clean = false;
      for (bool more = any; more && ok; more = ok && onward(clean)) {
        const int count = r.count;
        if (count == 0) continue;
        const bool nar = narrow(a, r.u);
        const int32_t* table = p.table + (int64_t)r.u.s * p.table_stride;
        const int tile0 = r.u.t0 + r.first, rows = r.u.rows, h = r.h;
        struct Place {
          int page, row;  // of a box; -1: none
        };
        auto look = [&](int chunk) -> Place {
          const int64_t row = ((int64_t)tile0 + ((int64_t)chunk << per_shift)) * kAtKeys + ((int64_t)lane << box_shift);
          if (row >= rows || row >= (int64_t)(tile0 + count) * kAtKeys) return {-1, 0};
          const int at = a.by_page.quotient((int)row >> 4);
          const int page = table[at];
          if (page_ok(p, page)) return {page, (int)row - at * p.page_rows};
          set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
          return {(int)p.num_pages, 0};  // (behind the tensor: its rows arrive as zeros)
        };
        Place even = look(0), odd = look(1);
        for (int pos = 0; pos < 2 * count; ++pos, ++n) {
          int j;  // the key tile within the run
          const bool val = entry_of(nar, count, pos, j);
          const int chunk = j >> per_shift, in_chunk = j - (chunk << per_shift);
          if (val && in_chunk == 0 && chunk > 0) {  // keys are at most two tiles ahead of values, a chunk four or more
            if (chunk & 1)
              even = look(chunk + 1);
            else
              odd = look(chunk + 1);
          }
          const int left = rows - (tile0 + j) * kAtKeys;                     // rows from the tile's first on
          const int boxes = (min(left, kAtKeys) + box - 1) >> box_shift;     // that hold any
          const Place mine = chunk & 1 ? odd : even;
          const int lane0 = in_chunk << boxes_shift;
          const CUtensorMap* map = val ? &vmap : &kmap;
          if constexpr (Q8) {
            // codes to their own ring, from where they are widened into the tiles' one; with a tile's keys its scales
            const uint32_t st = n % C::kCodeStages;
            if (n >= C::kCodeStages) ok = mbar_wait_warp(&ctl->cempty[st], (n / C::kCodeStages + 1) & 1, kAtLong);
            const uint32_t sc = (tiles + j) % C::kScaleStages, turn = (tiles + j) / C::kScaleStages;
            if (ok && !val && turn > 0) ok = mbar_wait_warp(&ctl->scempty[sc], (turn + 1) & 1, kAtLong);
            if (!ok) break;
            // a lane to each box of codes, and of the keys' and of the values' scales
            const int b = lane & ((1 << boxes_shift) - 1);
            const int page = __shfl_sync(0xffffffffu, mine.page, lane0 + b);
            const int row = __shfl_sync(0xffffffffu, mine.row, lane0 + b);
            const bool codes = lane < (1 << boxes_shift) && b < boxes;
            const bool scale = !val && lane < (2 << boxes_shift) && b < boxes, there = scale && page < p.num_pages;
            const uint32_t scales = __popc(__ballot_sync(0xffffffffu, there));
            float* to =
                  reinterpret_cast<float*>(sm + C::kOffScales) + (sc * 4 + (lane >> boxes_shift)) * kAtKeys + (b << box_shift);
            if (scale && !there)  // (of a page out of bounds)
              for (int e = 0; e < box; ++e) to[e] = 0.f;
            __syncwarp();
            if (one) {
              mbar_arrive_expect_tx(&ctl->cfull[st], (uint32_t)((boxes << box_shift) * D));
              if (!val) mbar_arrive_expect_tx(&ctl->scfull[sc], scales << (box_shift + 2));
            }
            __syncwarp();
            fence_proxy_async_smem();
            if (codes)
              tma_load_4d(base + C::kOffCodes + st * C::kCodeTile + ((b * D) << box_shift), map, 0, row, h, page,
                          &ctl->cfull[st]);
            if (there)
              bulk_g2s(to, (codes ? p.k_scale : p.v_scale) + page_slot(p, page, h, row), 4 << box_shift, &ctl->scfull[sc]);
          } else {
            const uint32_t st = n % C::kStages;
            if (n >= C::kStages) ok = mbar_wait_warp(&ctl->empty[st], (n / C::kStages + 1) & 1, kAtLong);
            if (!ok) break;
            // values behind the last row (in a second walk all that are not finite) are cleared by another warp, which
            // then says that the tile is there
            uint64_t* bar = val && (clean || left < kAtKeys) ? &ctl->tail[st] : &ctl->full[st];
            if (one) {
              mbar_arrive_expect_tx(bar, (uint32_t)((boxes << box_shift) * 2 * D));
              fence_proxy_async_smem();
            }
            const uint32_t dst = base + C::kOffRing + st * C::kTile;
            for (int b = 0; b < boxes; ++b) {
              const int page = __shfl_sync(0xffffffffu, mine.page, lane0 + b);
              const int row = __shfl_sync(0xffffffffu, mine.row, lane0 + b);
              if (one) {
#pragma unroll
                for (int slab = 0; slab < D / 64; ++slab)
                  tma_load_5d(dst + slab * C::kSlab + ((b * 128) << box_shift), map, 0, row, slab, h, page, bar);
              }
            }
            __syncwarp();
          }
        }
        tiles += count;
      }
      if (!ok) {
        // the copies in flight land before the CTA's shared memory is another's
        give_up(clean);
        constexpr uint32_t kRing = Q8 ? C::kCodeStages : C::kStages;
        uint64_t* bars = Q8 ? ctl->cfull : ctl->full;
        for (uint32_t f = n > kRing ? n - kRing : 0; f < n; ++f) (void)mbar_wait_warp(&bars[f % kRing], (f / kRing) & 1);
        for (uint32_t f = 0; Q8 && f < C::kScaleStages && f <= tiles; ++f) (void)mbar_wait_warp(&ctl->scfull[f], 0);
      }
    } else if (warp == kAtAux) {
      // ---- queries, and the values behind a sequence's last row
      uint32_t units = 0, tails = 0, n = 0;  // tails: bit st is the parity of tail[st]
      bool ok = true, clean = false;
      for (bool more = any; more && ok; more = ok && onward(clean)) {
        if (r.count == 0) continue;
        const bool nar = narrow(a, r.u);
        if (units > 0) ok = mbar_wait_warp(&ctl->qempty, (units - 1) & 1, kAtLong);
        if (!ok) break;
        if (lane == 0) {
          const int streams = nar ? 1 : 2;
          fence_proxy_async_smem();
          mbar_arrive_expect_tx(&ctl->qfull, (uint32_t)(streams * (D / 64) * a.tok_tile * a.group * 128));
          for (int i = 0; i < streams; ++i)
            for (int sl = 0; sl < D / 64; ++sl)
              tma_load_4d(base + C::kOffQ + i * C::kTile + sl * C::kSlab, &qmap, 0, sl, r.h * a.group,
                          r.u.token0 + i * a.tok_tile, &ctl->qfull);
        }
        __syncwarp();
        ++units;
        const int64_t last = (int64_t)(r.u.t0 + r.first + r.count) * kAtKeys;
        for (int pos = 0; !Q8 && clean && pos < 2 * r.count; ++pos) {
          int j;
          if (!entry_of(nar, r.count, pos, j)) continue;
          const uint32_t st = (n + pos) % C::kStages;
          ok = mbar_wait_warp(&ctl->tail[st], (tails >> st) & 1, kAtLong);
          if (!ok) break;
          tails ^= 1u << st;
          uint8_t* tile = sm + C::kOffRing + st * C::kTile;
          const int valid = min(r.u.rows - (r.u.t0 + r.first + j) * kAtKeys, kAtKeys);
          uint32_t odd = 0;
          for (int i = lane; i < kAtKeys * (D / 8); i += 32) {
            const int row = i / (D / 8), rest = i % (D / 8);
            uint4* at = reinterpret_cast<uint4*>(tile + (rest >> 3) * C::kSlab + row * 128 + (rest & 7) * 16);
            uint4 x = *at;
            uint32_t w[4] = {x.x, x.y, x.z, x.w};
            bool any_odd = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // (all ones in the exponent)
              const uint32_t lo = (w[e] & 0x7f80u) == 0x7f80u ? 0xffffu : 0u;
              const uint32_t hi = (w[e] & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u;
              any_odd |= (lo | hi) != 0;
              w[e] &= ~(lo | hi);
            }
            const bool behind = row >= valid;
            if (behind || any_odd) *at = behind ? make_uint4(0, 0, 0, 0) : make_uint4(w[0], w[1], w[2], w[3]);
            if (any_odd && !behind) odd |= 1u << (row >> 2);
          }
          odd = __reduce_or_sync(0xffffffffu, odd);
          if (lane == 0) ctl->odd[st] = odd;
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->full[st]);
        }
        if (!ok) break;
        if (!Q8 && !clean && last > r.u.rows) {
          const uint32_t st = (n + 2 * r.count - 1) % C::kStages;  // a run's last entry
          ok = mbar_wait_warp(&ctl->tail[st], (tails >> st) & 1, kAtLong);
          if (!ok) break;
          tails ^= 1u << st;
          uint8_t* tile = sm + C::kOffRing + st * C::kTile;
          const int valid = r.u.rows - (int)(last - kAtKeys);
          for (int i = valid * (D / 8) + lane; i < kAtKeys * (D / 8); i += 32) {
            const int row = i / (D / 8), rest = i % (D / 8);
            *reinterpret_cast<uint4*>(tile + (rest >> 3) * C::kSlab + row * 128 + (rest & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->full[st]);
        }
        n += 2 * r.count;
      }
      if (!ok) give_up(clean);
      if (units > 0) (void)mbar_wait_warp(&ctl->qfull, (units - 1) & 1);  // (landed)
    } else if (warp == kAtMma || warp == kAtMma + 1) {
      // ---- the MMAs of stream i: S of its first tile; then, tile by tile, O += P V and S of the next.  The whole warp
      // walks along, with values that the compiler knows to be one for all lanes, and one lane issues: MMAs take their
      // operands from uniform registers (a chunk of a 130,000-row prompt took a fifth longer with one lane alone in a
      // branch).  Each stream has a warp of its own, which hides the waits between one's MMAs behind the other's
      constexpr uint32_t id_s = umma_idesc_bf16(kAtRows, kAtKeys);
      constexpr uint32_t id_o = umma_idesc_bf16_bmn(kAtRows, D);
      const int i = __shfl_sync(0xffffffffu, warp - kAtMma, 0);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const uint32_t ts = tm + kAtS + 128 * i, to = tm + kAtO + 128 * i, tp = ts;
      const bool one = elect_one();
      uint32_t units = 0, n = 0, p_it = 0, turns = 0;
      bool ok = true, clean = false;
      // the streams issue in turns: one's burst of MMAs would otherwise slow the other's, and both softmaxes wait for both
      auto my_turn = [&] { return (i == 0 && turns == 0) || mbar_wait_warp(&ctl->turn[i], (turns - (i == 0)) & 1, kAtLong); };
      auto pass = [&] {
        if (one) mbar_arrive(&ctl->turn[1 - i]);
      };
      for (bool more = any; more && ok; more = ok && onward(clean)) {
        const int count = __shfl_sync(0xffffffffu, r.count, 0);
        if (count == 0) continue;
        const bool nar = __shfl_sync(0xffffffffu, (int)narrow(a, r.u), 0);
        const int tiles = stream_tiles(nar, count, i);
        ok = mbar_wait_warp(&ctl->qfull, units & 1, kAtLong);
        if (!ok) break;
        ++units;
        const uint64_t qd = umma_desc_sw128(base + C::kOffQ + (nar ? 0 : i * C::kTile));
        auto entry = [&](uint32_t pos, uint32_t& st) {  // waits for a tile
          const uint32_t e = n + pos;
          st = e % C::kStages;
          return mbar_wait_warp(&ctl->full[st], (e / C::kStages) & 1, kAtLong);
        };
        auto release = [&](uint32_t st) {  // (by both streams, or by the one that has it)
          umma_commit(&ctl->empty[st]);
          if (nar) umma_commit(&ctl->empty[st]);
        };
        auto key_entry = [&](int it) { return nar ? max(2 * (2 * it + i) - 1, 0) : 2 * it; };
        auto logits = [&](int it, uint32_t st) {
          const uint64_t kd = umma_desc_sw128(base + C::kOffRing + st * C::kTile);
          if (one) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = ((kk >> 2) * C::kSlab + (kk & 3) * 32) >> 4;  // (of the address field)
              umma_bf16(ts, qd + off, kd + off, id_s, kk > 0);
              if (kk == D / 16 - 3) mbar_arrive(&ctl->turn[1 - i]);  // (what is left covers the other's waking up)
            }
            umma_commit(&ctl->sfull[i]);
            release(st);
            if (it == tiles - 1) umma_commit(&ctl->qempty);
          }
          __syncwarp();
        };
        uint32_t ks = 0, vs = 0;
        if (tiles > 0) {
          ok = entry(key_entry(0), ks);
          if (!ok) break;
          tc_fence_after();
          ok = my_turn();
          if (!ok) break;
          ++turns;
          logits(0, ks);
        } else {
          ok = my_turn();
          if (!ok) break;
          ++turns;
          pass();
          if (one) mbar_arrive(&ctl->qempty);
        }
        for (int it = 0; it < tiles; ++it) {
          // (what the tiles' waits cost is over before the weights come)
          ok = entry(nar ? min(2 * (2 * it + i) + 2, 2 * count - 1) : 2 * it + 1, vs) &&
               (it + 1 == tiles || entry(key_entry(it + 1), ks)) &&
               mbar_wait_warp(&ctl->phalf[i], p_it & 1, kAtLong) && my_turn();
          if (!ok) break;
          ++turns;
          tc_fence_after();
          const uint64_t vd = umma_desc_sw128_mn(base + C::kOffRing + vs * C::kTile, C::kSlab, 1024);
          auto weigh = [&](int half, bool first) {
#pragma unroll
            for (int kk = 0; kk < kAtKeys / 32; ++kk) {
              const int at = half * (kAtKeys / 32) + kk;
              umma_bf16_ts(to, tp + (FINE ? 64 * half + 8 * kk : 8 * at), vd + (at * 16 * 128 >> 4), id_o,
                           !first || it > 0 || kk > 0 || clean);
              if constexpr (FINE) umma_bf16_ts(to, tp + 64 * half + 32 + 8 * kk, vd + (at * 16 * 128 >> 4), id_o, 1);
            }
          };
          if (one) weigh(0, true);
          __syncwarp();
          ok = mbar_wait_warp(&ctl->pfull[i], p_it & 1, kAtLong);
          if (!ok) break;
          ++p_it;
          tc_fence_after();
          if (one) {
            weigh(1, false);
            release(vs);
            if (it + 1 == tiles) umma_commit(&ctl->ofull[i]);
          }
          __syncwarp();
          if (it + 1 < tiles)
            logits(it + 1, ks);
          else
            pass();
        }
        if (ok && nar && i == 1 && tiles < stream_tiles(nar, count, 0)) {  // (a turn for each of the first stream's)
          ok = my_turn();
          ++turns;
          pass();
        }
        n += 2 * count;
      }
      if (!ok) give_up(clean);
      if (one) umma_commit(&ctl->done);  // nothing of the tensor cores' is left behind
      (void)mbar_wait_warp(&ctl->done, 0);
    } else if (Q8 && warp >= kAtWiden) {
      // ---- int8 codes become bf16 tiles, half a row to a thread; value rows behind the sequence's last are zeros
      uint32_t n = 0, tiles = 0;
      bool ok = true, clean = false;
      const int row = (tid - kAtWiden * 32) & 127;
      const int half = (tid - kAtWiden * 32) >> 7;
      for (bool more = any; more && ok; more = ok && onward(clean)) {
        if (r.count == 0) continue;
        const bool nar = narrow(a, r.u);
        for (int pos = 0; pos < 2 * r.count; ++pos, ++n) {
          int j;
          const bool val = entry_of(nar, r.count, pos, j);
          const uint32_t cs = n % (Q8 ? C::kCodeStages : 1), st = n % C::kStages;
          const uint32_t sc = (tiles + j) % (Q8 ? C::kScaleStages : 1);
          const bool behind = (int64_t)(r.u.t0 + r.first + j) * kAtKeys + row >= r.u.rows;
          float* scales = reinterpret_cast<float*>(sm + C::kOffScales) + sc * 4 * kAtKeys + row;
          if (!val) {
            // A key's scale takes the logits' factor along.  A value's that is not finite makes its row one of NaN: what a
            // weight of 0 makes of that is mended as bf16 rows' is, by a second walk
            ok = mbar_wait_warp(&ctl->scfull[sc], ((tiles + j) / (Q8 ? C::kScaleStages : 1)) & 1, kAtLong);
            if (!ok) break;
            const float x = scales[half * kAtKeys];
            scales[(2 + half) * kAtKeys] = half == 0 ? x * a.scale_log2 : behind ? 0.f : finite(x) ? x : 1.f;
          }
          const bool zero = val && behind, bad = val && !behind && !finite(scales[kAtKeys]);
          ok = mbar_wait_warp(&ctl->cfull[cs], (n / (Q8 ? C::kCodeStages : 1)) & 1, kAtLong);
          if (!ok) break;
          const uint8_t* from = sm + C::kOffCodes + cs * C::kCodeTile;
          uint8_t* to = sm + C::kOffRing + st * C::kTile + row * 128;
          uint4 x[D / 32];
#pragma unroll
          for (int q = 0; q < D / 32; ++q)
            x[q] = *reinterpret_cast<const uint4*>(from + swz8<D>(row * D + 16 * (half * (D / 32) + q)));
          __syncwarp();
          if (lane == 0) mbar_arrive(&ctl->cempty[cs]);
          if (n >= C::kStages) ok = mbar_wait_warp(&ctl->empty[st], (n / C::kStages + 1) & 1, kAtLong);
          if (!ok) break;
          if (clean && val) {
            uint32_t quads = __ballot_sync(0xffffffffu, bad), byte = 0;
            for (int q = 0; q < 8; ++q) byte |= (quads >> (4 * q) & 15) ? 1u << q : 0u;
            if (half == 0 && lane == 0) reinterpret_cast<uint8_t*>(&ctl->odd[st])[row >> 5] = (uint8_t)byte;
          }
#pragma unroll
          for (int q = 0; q < D / 32; ++q) {
            const int c = half * (D / 32) + q;
            uint4 lo = make_uint4(widen2_bf16(x[q].x, 0x4140u), widen2_bf16(x[q].x, 0x4342u), widen2_bf16(x[q].y, 0x4140u),
                                  widen2_bf16(x[q].y, 0x4342u));
            uint4 hi = make_uint4(widen2_bf16(x[q].z, 0x4140u), widen2_bf16(x[q].z, 0x4342u), widen2_bf16(x[q].w, 0x4140u),
                                  widen2_bf16(x[q].w, 0x4342u));
            if (zero || bad) {
              const uint32_t u = zero || clean ? 0u : 0x7fc07fc0u;
              lo = hi = make_uint4(u, u, u, u);
            }
            uint8_t* slab = to + (c >> 2) * C::kSlab;
            *reinterpret_cast<uint4*>(slab + (((2 * c) & 7) ^ (row & 7)) * 16) = lo;
            *reinterpret_cast<uint4*>(slab + (((2 * c + 1) & 7) ^ (row & 7)) * 16) = hi;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (!val) mbar_arrive(&ctl->scready[sc]);
            mbar_arrive(&ctl->full[st]);
          }
        }
        tiles += r.count;
      }
      if (!ok) give_up(clean);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::kRegsSoft));
    // ---- softmax: stream i, query row `row` (its TMEM lane)
    const int i = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = tl + kAtS + 128 * i, tp = ts;  // logits; the weights over them
    if (tid == 0) a.cut[blockIdx.x].parts = 0;  // (until a run says otherwise)
    const int tok = a.by_group.quotient(row), hh = row - tok * a.group;
    uint32_t it_s = 0, it_o = 0, joins = 0, tiles0 = 0;
    bool ok = true, clean = false;
    for (bool more = any; more && ok; more = ok && onward(clean)) {
      const bool nar = narrow(a, r.u);
      const int my_tok = nar ? tok : tok + i * a.tok_tile;  // of the unit
      const bool valid = tok < a.tok_tile && my_tok < r.u.ntok;
      const int64_t token = (int64_t)r.u.token0 + my_tok;
      const int head = r.h * a.group + hh;
      if (r.count == 0) {
        if (r.u.c == 0 && r.at >= ctl->per * blockIdx.x && valid && (!nar || i == 0)) {  // nothing to see
          const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          for (int c = 0; c < D; c += 8) write_out<D, 8>(a, token, head, c, zero);
          write_lse(a, token, head, 0.f, 0.f);
        }
        continue;
      }
      // rows without a query see every key, so that they mask nothing; what they get is not read
      int lo = 0, hi = INT32_MAX;
      if (valid) token_rows(a, r.u.rows, r.u.n, r.u.tok0 + my_tok, token, lo, hi);
      const bool idle = !__any_sync(0xffffffffu, valid);
      const int tiles = stream_tiles(nar, r.count, i);
      float m = -FLT_MAX;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      for (int it = 0; it < tiles; ++it) {
        if (!mbar_wait_warp(&ctl->sfull[i], it_s & 1, kAtLong)) {
          ok = false;
          break;
        }
        ++it_s;
        tc_fence_after();
        const int j = nar ? 2 * it + i : it;
        const int k0 = (r.u.t0 + r.first + j) * kAtKeys;
        const uint32_t sc = Q8 ? (tiles0 + j) % (Q8 ? C::kScaleStages : 1) : 0;
        if constexpr (Q8) {
          ok = mbar_wait_warp(&ctl->scready[sc], ((tiles0 + j) / C::kScaleStages) & 1, kAtLong);
          if (!ok) break;
        }
        if (clean) {
          // second walk: the tile's values that are not finite are zeros by now, and go to O here, to the rows that see them
          const uint32_t e = 2 * tiles0 + (nar ? min(2 * j + 2, 2 * r.count - 1) : 2 * j + 1), st = e % C::kStages;
          ok = mbar_wait_warp(&ctl->full[st], (e / C::kStages) & 1, kAtLong);
          if (!ok) break;
          if (it == 0) {
            const float zero[16] = {};
            for (int c = 0; c < D; c += 16) tmem_st16(tl + kAtO + 128 * i + c, zero);
            tmem_wait_st();  // (add_odd reads these columns)
          }
          for (uint32_t odd = ctl->odd[st]; odd; odd &= odd - 1)
            for (int f = 0; f < 4; ++f) {
              const int at = k0 + 4 * (__ffs(odd) - 1) + f;
              const bool sees = valid && at >= lo && at < hi;
              if (__any_sync(0xffffffffu, sees)) add_odd<D, Q8>(a, r.u.s, r.h, at, sees, tl + kAtO + 128 * i);
            }
          tmem_wait_st();
          __syncwarp();
        }
        if (!idle) {
          const bool masked = !__all_sync(0xffffffffu, lo <= k0 && hi - k0 >= kAtKeys);
          const int from = lo - k0;
          const uint32_t wide = (uint32_t)(hi - lo);
          const float* ks = reinterpret_cast<const float*>(sm + C::kOffScales) + (sc * 4 + 2) * kAtKeys;
          // moves the reference to a maximum that passes it by more than the slack
          auto refer = [&](float top) {
            // (a second walk's weights are 2^-40 of what they were)
            const float mx = (Q8 ? top : top * a.scale_log2) + (clean ? 40.f : 0.f);
            if (__any_sync(0xffffffffu, valid && mx > m + kAtSlack)) {  // (what lies in rows without a query has no say)
              const float to = fmaxf(m, mx), f = fast_exp2(m - to);
              m = to;
              sum[0].x *= f, sum[0].y *= f, sum[1].x *= f, sum[1].y *= f;
              if (it > 0) {
#pragma unroll
                for (int c = 0; c < D; c += 16) {
                  float o[16];
                  tmem_ld16(tl + kAtO + 128 * i + c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] *= f;
                  tmem_st16(tl + kAtO + 128 * i + c, o);
                }
              }
            }
          };
          const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
          auto half_done = [&] {  // the first half of the weights is in place: its product can begin
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            mbar_arrive_if(lane == 0, &ctl->phalf[i]);
          };
          if constexpr (!Q8) {
            float v[kAtKeys];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, v + 32 * c);
            tmem_wait_ld();
            if (masked) {
#pragma unroll
              for (int h = 0; h < kAtKeys; h += 32) mask32(v + h, from, wide, h);
            }
            float top[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) top[e] = fmaxf(v[e], v[4 + e]);
#pragma unroll
            for (int c = 8; c < kAtKeys; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) top[e] = fmaxf(fmaxf(top[e], v[c + e]), v[c + 4 + e]);
            refer(fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])));
            const float2 ref2 = make_float2(-m, -m);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t w[32], z[FINE ? 32 : 1];
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                const float2 x = fma2(make_float2(v[64 * half + 2 * c], v[64 * half + 2 * c + 1]), scale2, ref2);
                const float2 e = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                sum[c & 1] = add2(sum[c & 1], e);
                w[c] = pack2(e.x, e.y);
                if constexpr (FINE) z[c] = rest2(e, w[c]);
              }
              tmem_st32(tp + (FINE ? 64 : 32) * half, reinterpret_cast<const float*>(w));
              if constexpr (FINE) tmem_st32(tp + 64 * half + 32, reinterpret_cast<const float*>(z));
              if (half == 0) half_done();
            }
          } else {
            // 64 at a time (144 registers a thread): the logits get the key's scale and their mask and go back to where
            // they were, then come again as weights, which get the value's scale
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
            for (int h = 0; h < kAtKeys; h += 64) {
              float v[64];
              tmem_ld32(ts + h, v);
              tmem_ld32(ts + h + 32, v + 32);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 64; e += 4) {
                const float4 k4 = *reinterpret_cast<const float4*>(ks + h + e);
                const float2 x = mul2(make_float2(v[e], v[e + 1]), make_float2(k4.x, k4.y));
                const float2 y = mul2(make_float2(v[e + 2], v[e + 3]), make_float2(k4.z, k4.w));
                v[e] = x.x, v[e + 1] = x.y, v[e + 2] = y.x, v[e + 3] = y.y;
              }
              if (masked) {
                mask32(v, from, wide, h);
                mask32(v + 32, from, wide, h + 32);
              }
#pragma unroll
              for (int e = 0; e < 64; e += 4) {
                top[0] = fmaxf(fmaxf(top[0], v[e]), v[e + 1]);
                top[1] = fmaxf(fmaxf(top[1], v[e + 2]), v[e + 3]);
              }
              tmem_st32(ts + h, v);
              tmem_st32(ts + h + 32, v + 32);
            }
            refer(fmaxf(top[0], top[1]));
            tmem_wait_st();
            const float2 ref2 = make_float2(-m, -m);
#pragma unroll 1
            for (int h = 0; h < kAtKeys; h += 64) {
              float v[64];
              tmem_ld32(ts + h, v);
              tmem_ld32(ts + h + 32, v + 32);
              tmem_wait_ld();
              uint32_t w[32], z[FINE ? 32 : 1];
#pragma unroll
              for (int e = 0; e < 64; e += 4) {
                const float4 v4 = *reinterpret_cast<const float4*>(ks + kAtKeys + h + e);
                float2 x = add2(make_float2(v[e], v[e + 1]), ref2), y = add2(make_float2(v[e + 2], v[e + 3]), ref2);
                x = make_float2(fast_exp2(x.x), fast_exp2(x.y));
                y = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                sum[0] = add2(sum[0], x);
                sum[1] = add2(sum[1], y);
                x = mul2(x, make_float2(v4.x, v4.y));
                y = mul2(y, make_float2(v4.z, v4.w));
                w[e / 2] = pack2(x.x, x.y);
                w[e / 2 + 1] = pack2(y.x, y.y);
                if constexpr (FINE) z[e / 2] = rest2(x, w[e / 2]), z[e / 2 + 1] = rest2(y, w[e / 2 + 1]);
              }
              tmem_st32(tp + (FINE ? h : h / 2), reinterpret_cast<const float*>(w));
              if constexpr (FINE) tmem_st32(tp + h + 32, reinterpret_cast<const float*>(z));
              if (h == 0) half_done();
            }
          }
          tmem_wait_st();
          tc_fence_before();
        } else if (lane == 0) {
          mbar_arrive(&ctl->phalf[i]);
        }
        if constexpr (Q8) {
          __syncwarp();
          if (lane == 0) mbar_arrive_n(&ctl->scempty[sc], nar ? 2 : 1);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->pfull[i]);
      }
      if (!ok) break;
      tiles0 += r.count;
      float l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      if (tiles > 0) {
        if (!mbar_wait_warp(&ctl->ofull[i], it_o & 1, kAtLong)) {
          ok = false;
          break;
        }
        ++it_o;
        tc_fence_after();
      }
      // ---- the run's result: O of stream 0 times f0 and that of stream 1 times f1, over columns c0 .. c1 - 1.  A narrow
      // unit's streams join theirs, each half the columns
      const bool other = nar && r.count > 1;  // the second stream has any
      float f0 = i == 0 || nar ? 1.f : 0.f, f1 = 1.f - f0;
      const int c0 = nar ? i * (D / 2) : 0, c1 = nar ? c0 + D / 2 : D;
      if (nar) {
        ctl->ml[i][row] = make_float2(m, l);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->mlfull);
        ok = mbar_wait_warp(&ctl->mlfull, joins & 1, kAtLong);
        if (!ok) break;
        tc_fence_after();
        const float2 x = ctl->ml[0][row], y = ctl->ml[1][row];
        m = fmaxf(x.x, y.x);
        f0 = fast_exp2(x.x - m);
        f1 = fast_exp2(y.x - m);
        l = x.y * f0 + y.y * f1;
      }
      if (!idle) {
        const bool cut = r.count < r.u.c;
        // A row that sees none of the run's keys has the result 0 whatever their values are: a weight of 0 times one that is
        // not finite has made its O NaN, which a join would take along
        const int row0 = (r.u.t0 + r.first) * kAtKeys;
        const bool blind = hi <= row0 || lo - row0 >= r.count * kAtKeys;
        const int64_t slot = part_slot(blockIdx.x, r.first == 0) * a.rows_cap;
        const int rho = my_tok * a.group + hh;
        if (!cut) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          f0 *= inv;
          f1 *= inv;
        }
        const float2 f02 = make_float2(f0, f0), f12 = make_float2(f1, f1), zero2 = make_float2(0.f, 0.f);
        float4* to = reinterpret_cast<float4*>(a.part_o + slot * D) + (int64_t)(c0 / 4) * a.rows_cap + rho;
        float2 not_finite[2] = {zero2, zero2};  // (0 times what is not finite is NaN)
#pragma unroll 1
        for (int c = c0; c < c1; c += 16) {
          float2 o[8];
          tmem_ld16(tl + kAtO + (nar ? 0 : 128 * i) + c, reinterpret_cast<float*>(o));
          if (other) {
            float2 x[8];
            tmem_ld16(tl + kAtO + 128 + c, reinterpret_cast<float*>(x));
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fma2(x[e], f12, mul2(o[e], f02));
          } else {
            const float2 f = nar || i == 0 ? f02 : f12;
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = mul2(o[e], f);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) not_finite[e & 1] = fma2(o[e], zero2, not_finite[e & 1]);
          if (blind || (!cut && l == 0.f)) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = zero2;
          }
          if (valid && cut) {
#pragma unroll
            for (int e = 0; e < 8; e += 2, to += a.rows_cap) *to = make_float4(o[e].x, o[e].y, o[e + 1].x, o[e + 1].y);
          } else if (valid) {
            write_out<D, 16>(a, token, head, c, reinterpret_cast<const float*>(o));
          }
          __syncwarp();  // (tcgen05.ld and .st want the warp's lanes together)
        }
        not_finite[0] = add2(not_finite[0], not_finite[1]);
        // (a part without a sum, whose logits are all minus infinity, is of a row that others may have given one)
        const bool bad = not_finite[0].x + not_finite[0].y != 0.f && !blind && (cut || l != 0.f);
        if (valid && c0 == 0) {
          if (cut)
            a.part_ml[slot + rho] = make_float2(m, l);
          else
            write_lse(a, token, head, m, l);
        }
        if (valid && bad && finite(l)) ctl->bad = 1;
      }
      if (tid == 0 && r.first == 0) {
        const uint64_t per = ctl->per;
        // (offsets out of order, an error, give every CTA a line of its own: no part of a unit lies behind the last CTA)
        const int cta = (int)quotient(r.at, per);
        const int parts = (int)min(quotient(r.at + r.u.c - 1, per), (uint64_t)a.ctas - 1) - cta + 1;
        if (parts > 1) a.cut[blockIdx.x] = AtCut{parts, cta, r.h, r.u.ntok, r.u.token0, r.slot, 0};
      }
      tc_fence_before();
      if (nar) {  // (either stream's O is both's to read)
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->mlfree);
        ok = mbar_wait_warp(&ctl->mlfree, joins & 1, kAtLong);
        if (!ok) break;
        ++joins;
        tc_fence_after();
      }
    }
    if (!ok) give_up(clean);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kAtMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The key tiles that each unit's tokens see, where tokens have ranges of their own.
constexpr int kArThreads = 128;
__global__ void __launch_bounds__(kArThreads) attend_range_kernel(const __grid_constant__ AtArgs a) {
  pdl_wait();
  pdl_trigger();
  const int slot = blockIdx.x * (kArThreads / 32) + (threadIdx.x >> 5);
  if (slot < a.slots) find_range(a, seqs_of(a), slot);
}

// Joins the parts of the units that several CTAs shared, in their order: a warp to 32 rows and E columns of them, a row
// to a lane, N parts in flight.
constexpr int kAfThreads = 256;
// As many CTAs as an SM holds at once (four of them: four drafts of eight chats took 14 % more), or one, where the next
// kernel is to start beside them.
constexpr int kAfCtas = 2;
template <int D, int E, int N>
__global__ void __launch_bounds__(kAfThreads) attend_finish_kernel(const __grid_constant__ AtArgs a) {
  // (results that are a part of another call's: its next kernel is the call's own, and waits for them where it needs them)
  if (a.part.out) pdl_trigger();
  pdl_wait();
  if (!a.part.out) pdl_trigger();
  // the cut units' items, a unit to a thread; ends[c]: those up to the unit that begins in CTA c
  __shared__ int ends[kAfThreads], sums[kAfThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const AtCut* mine = a.cut + tid;
  int incl = tid < a.ctas && mine->parts > 1 ? (mine->ntok * a.group + 31) / 32 * (D / E) : 0;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) sums[tid >> 5] = incl;
  __syncthreads();
  for (int w = 0; w < (tid >> 5); ++w) incl += sums[w];
  ends[tid] = incl;
  __syncthreads();
  for (int all = ends[kAfThreads - 1], i = blockIdx.x + gridDim.x * (tid >> 5); i < all; i += gridDim.x * (kAfThreads / 32)) {
    int unit = 0;  // the first whose end is past i
#pragma unroll
    for (int step = kAfThreads / 2; step > 0; step >>= 1)
      if (ends[unit + step - 1] <= i) unit += step;
    const AtCut cut = a.cut[unit];
    const int item = i - (unit ? ends[unit - 1] : 0), rows = cut.ntok * a.group;
    const int col = item % (D / E) * E, rho = min(item / (D / E) * 32 + lane, rows - 1);
    const bool valid = item / (D / E) * 32 + lane < rows;
    float m = -FLT_MAX, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int j0 = 0; j0 < cut.parts; j0 += N) {
      float2 ml[N];
      float4 x[N][E / 4];
#pragma unroll
      for (int f = 0; f < N; ++f) {
        const int j = min(j0 + f, cut.parts - 1);
        const int64_t slot = part_slot(cut.c0 + j, j == 0) * a.rows_cap;
        ml[f] = a.part_ml[slot + rho];
        const float4* from = reinterpret_cast<const float4*>(a.part_o + slot * D) + (int64_t)(col / 4) * a.rows_cap + rho;
#pragma unroll
        for (int e = 0; e < E / 4; ++e) x[f][e] = from[(int64_t)e * a.rows_cap];
      }
      float up = m;
#pragma unroll
      for (int f = 0; f < N; ++f) up = fmaxf(up, ml[f].x);
      const float f0 = fast_exp2(m - up);
      m = up;
      l *= f0;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] *= f0;
#pragma unroll
      for (int f = 0; f < N; ++f) {
        if (j0 + f >= cut.parts) continue;
        const float w = fast_exp2(ml[f].x - m);
        l = fmaf(ml[f].y, w, l);
        const float* y = reinterpret_cast<const float*>(x[f]);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(y[e], w, o[e]);
      }
    }
    const int my_tok = rho / a.group, head = cut.h * a.group + rho % a.group;
    const int64_t token = cut.token0 + my_tok;
    const float inv = 1.f / l;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] = l == 0.f ? 0.f : o[e] * inv;
      bad |= !finite(o[e]);
    }
    if (bad && finite(l)) {  // sums of finite parts may pass fp32's range before they are divided
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = 0.f;
      for (int j = 0; j < cut.parts; ++j) {
        const int64_t slot = part_slot(cut.c0 + j, j == 0) * a.rows_cap;
        const float w = fast_exp2(a.part_ml[slot + rho].x - m) * inv;
        const float4* from = reinterpret_cast<const float4*>(a.part_o + slot * D) + (int64_t)(col / 4) * a.rows_cap + rho;
#pragma unroll
        for (int e = 0; e < E / 4; ++e) {
          const float4 x = from[(int64_t)e * a.rows_cap];
          o[4 * e] = fmaf(x.x, w, o[4 * e]);
          o[4 * e + 1] = fmaf(x.y, w, o[4 * e + 1]);
          o[4 * e + 2] = fmaf(x.z, w, o[4 * e + 2]);
          o[4 * e + 3] = fmaf(x.w, w, o[4 * e + 3]);
        }
      }
    }
    if (valid) write_out<D, E>(a, token, head, col, o);
    if (valid && col == 0) write_lse(a, token, head, m, l);
  }
}

// ------------------------------------------------------------------ host

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
inline bool al16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; }
inline bool al4(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 3) == 0; }

int box_rows(int page_rows) {  // the largest power of two up to 128 that divides a page
  int b = kAtKeys;
  while (page_rows % b) b /= 2;
  return b;
}

// Boxes of as many rows of one page and KV head, one 128-byte slab of them (int8 rows: whole).
bool encode_kv(CUtensorMap* m, const void* base, const AttendPlan& pl) {
  auto enc = tma_encoder();
  if (!enc) return false;
  const Pages& p = pl.pages;
  if (pl.q8) {
    cuuint64_t dims[4] = {(cuuint64_t)pl.d, (cuuint64_t)p.page_rows, (cuuint64_t)p.h_kv, (cuuint64_t)p.num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)p.stride_row, (cuuint64_t)p.stride_head, (cuuint64_t)p.stride_page};
    cuuint32_t box[4] = {(cuuint32_t)pl.d, (cuuint32_t)box_rows(p.page_rows), 1, 1}, es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, pl.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               pl.d == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  cuuint64_t dims[5] = {64, (cuuint64_t)p.page_rows, (cuuint64_t)pl.d / 64, (cuuint64_t)p.h_kv, (cuuint64_t)p.num_pages};
  cuuint64_t strides[4] = {(cuuint64_t)p.stride_row * 2, 128, (cuuint64_t)p.stride_head * 2, (cuuint64_t)p.stride_page * 2};
  cuuint32_t box[5] = {64, (cuuint32_t)box_rows(p.page_rows), 1, 1, 1}, es[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             pl.d == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Boxes of a KV head's query heads of tok_tile tokens, one 128-byte slab of them: packed rows, head by head.
bool encode_q(CUtensorMap* m, const aircache_paged_attend_problem* p, const AttendPlan& pl) {
  auto enc = tma_encoder();
  if (!enc) return false;
  cuuint64_t dims[4] = {64, (cuuint64_t)pl.d / 64, (cuuint64_t)p->h_q, (cuuint64_t)p->num_tokens};
  cuuint64_t strides[3] = {128, (cuuint64_t)(p->h_q > 1 ? p->q_stride_head : pl.d) * 2,
                           (cuuint64_t)(p->num_tokens > 1 ? p->q_stride_tok : (int64_t)p->h_q * pl.d) * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)pl.g, (cuuint32_t)pl.tok_tile}, es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p->q), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool Q8, bool FINE>
int launch_at(const aircache_paged_attend_problem* p, const AttendPlan& pl, const AtArgs& a, cudaStream_t s) {
  using C = AtCfg<D, Q8>;
  CUtensorMap qm, km, vm;
  if (!encode_q(&qm, p, pl) || !encode_kv(&km, pl.pages.k, pl) || !encode_kv(&vm, pl.pages.v, pl))
    return AIRCACHE_ERR_UNSUPPORTED;
  constexpr int smem = C::kOffCtl + (int)sizeof(AtCtl<D, Q8>);
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  if (allow_smem(reinterpret_cast<const void*>(&paged_attend_kernel<D, Q8, FINE>), smem) != cudaSuccess) return AIRCACHE_ERR_CUDA;
  if (a.range && a.ranged && launch_pdl(attend_range_kernel, dim3((a.slots + kArThreads / 32 - 1) / (kArThreads / 32)),
                            dim3(kArThreads), 0, s, a) != cudaSuccess)
    return AIRCACHE_ERR_CUDA;
  static std::atomic<int> known{0};  // registers that the built kernel has; what a failed query says is not kept
  int regs = known.load(std::memory_order_relaxed);
  if (regs == 0) {
    cudaFuncAttributes f;
    if (cudaFuncGetAttributes(&f, reinterpret_cast<const void*>(&paged_attend_kernel<D, Q8, FINE>)) != cudaSuccess)
      return AIRCACHE_ERR_CUDA;
    known.store(regs = f.numRegs, std::memory_order_relaxed);
  }
  // (what the warps share out between them is what the launch brings)
  if (regs < C::kRegs) return AIRCACHE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.grid);
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, paged_attend_kernel<D, Q8, FINE>, qm, km, vm, a) != cudaSuccess) return AIRCACHE_ERR_CUDA;
  // Few units (at most half as many as CTAs) have many parts each, of which many are in flight; with more, few parts, it is
  // the pieces of work that are many, and larger.  (4 x 256 tokens over 12,544 rows, 128 units: 8 columns and 8 parts take 3 %
  // more than 16 and 3; four drafts of eight chats, 32 units: 6 % less; 24 chats behind a prefix of 131,072, 4 units: 5 %
  // less)
  const bool many = 2 * (int64_t)pl.slots * pl.pages.h_kv > pl.grid;
  const auto join = many ? &attend_finish_kernel<D, 16, 3> : &attend_finish_kernel<D, 8, 8>;
  return launch_pdl(join, dim3(a.part.out ? pl.grid : pl.grid * kAfCtas), dim3(kAfThreads), 0, s, a) == cudaSuccess
             ? AIRCACHE_OK
             : AIRCACHE_ERR_CUDA;
}

template <bool FINE>
int launch_at(const aircache_paged_attend_problem* p, const AttendPlan& pl, const AtArgs& a, cudaStream_t s) {
  if (pl.q8) return pl.d == 128 ? launch_at<128, true, FINE>(p, pl, a, s) : launch_at<64, true, FINE>(p, pl, a, s);
  return pl.d == 128 ? launch_at<128, false, FINE>(p, pl, a, s) : launch_at<64, false, FINE>(p, pl, a, s);
}

}  // namespace

int attend_plan(const aircache_paged_attend_problem* p, bool part, AttendPlan& pl) {
  if (!p) return AIRCACHE_ERR_INVALID_ARG;
  const int rc = check_pages(p->pages, pl.pages);
  if (rc != AIRCACHE_OK) return rc;
  const int d = p->pages->head_dim;
  if (p->num_tokens < 0 || p->num_tokens > 0x7fff0000LL || p->h_q <= 0 || p->h_q % p->pages->h_kv != 0 ||
      p->dtype != AIRCACHE_BF16 || (p->causal != 0 && p->causal != 1) || p->reserved0 != 0 || p->reserved1 != 0.f ||
      !(p->scale > 0.f) || !std::isfinite(1.4427f * p->scale) ||
      !p->q || !al16(p->q) || p->q_stride_tok % 8 != 0 || p->q_stride_head % 8 != 0 ||
      (p->num_tokens > 1 && p->q_stride_tok <= 0) || (p->h_q > 1 && p->q_stride_head <= 0) || !p->cu_tokens ||
      !al4(p->cu_tokens) || !al4(p->row_begin) || !al4(p->row_end) || !al4(p->lse))
    return AIRCACHE_ERR_INVALID_ARG;
  if (!part) {
    // outputs: rows apart from one another and from the queries
    const int64_t st = p->out_stride_tok, sh = p->out_stride_head;
    if (!p->out || !al16(p->out) || st % 8 != 0 || sh % 8 != 0) return AIRCACHE_ERR_INVALID_ARG;
    const bool many_t = p->num_tokens > 1, many_h = p->h_q > 1;
    if ((many_t && st < d) || (many_h && sh < d)) return AIRCACHE_ERR_INVALID_ARG;
    if (many_t && many_h) {
      const __int128 heads = (__int128)(p->h_q - 1) * sh + d, toks = (__int128)(p->num_tokens - 1) * st + d;
      if (st < heads && sh < toks) return AIRCACHE_ERR_INVALID_ARG;
    }
    // (without a token nothing is written)
    const int64_t T = p->num_tokens, H = p->h_q;
    const size_t nq = span_bytes(p->q, {{T, p->q_stride_tok}, {H, p->q_stride_head}}, d, 2);
    const size_t no = span_bytes(p->out, {{T, st}, {H, sh}}, d, 2), nl = p->lse ? span_bytes(p->lse, {{T, H}}, H, 4) : 0;
    auto meets = [&](const void* x, size_t n) {
      return arrays_meet(x, n, p->q, nq) || meets_cache(p->pages, pl.pages, x, n) ||
             arrays_meet(x, n, p->cu_tokens, 4 * ((size_t)p->pages->num_seqs + 1)) ||
             arrays_meet(x, n, p->row_begin, 4 * (size_t)T) || arrays_meet(x, n, p->row_end, 4 * (size_t)T);
    };
    if (T > 0 && (meets(p->out, no) || meets(p->lse, nl) || arrays_meet(p->lse, nl, p->out, no)))
      return AIRCACHE_ERR_INVALID_ARG;
  }
  pl.d = d;
  pl.h_q = p->h_q;
  pl.g = p->h_q / p->pages->h_kv;
  pl.q8 = p->pages->kv_dtype == AIRCACHE_INT8;
  if (pl.g > kAtGroup) return AIRCACHE_ERR_UNSUPPORTED;
  pl.tok_tile = kAtRows / pl.g;
  pl.slots = (int)(p->num_tokens / (2 * pl.tok_tile)) + p->pages->num_seqs;
  pl.grid = std::min(device_sms(), kAfThreads);
  pl.rows_cap = (int)std::min<int64_t>(2 * pl.tok_tile, std::max<int64_t>(p->num_tokens, 1)) * pl.g;
  pl.cut_off = kAtHeader;
  pl.start_off = pl.cut_off + up256(sizeof(AtCut) * (size_t)pl.grid);
  pl.range_off = pl.start_off + up256(sizeof(AtRun) * (size_t)pl.grid);
  pl.ml_off = pl.range_off + (p->row_begin || p->row_end ? up256(sizeof(int2) * (size_t)pl.slots) : 0);
  pl.o_off = pl.ml_off + up256(sizeof(float2) * 2 * (size_t)pl.grid * pl.rows_cap);
  pl.total = pl.o_off + up256(sizeof(float) * 2 * (size_t)pl.grid * pl.rows_cap * pl.d);
  return AIRCACHE_OK;
}

int attend_launch(const aircache_paged_attend_problem* p, const AttendPlan& pl, const AttendPart& part, uint8_t* ws,
                  int32_t* error, cudaStream_t s) {
  AtArgs a;
  a.pages = pl.pages;
  a.cu = p->cu_tokens;
  a.row_begin = p->row_begin;
  a.row_end = p->row_end;
  a.out = static_cast<__nv_bfloat16*>(p->out);
  a.out_stride_tok = p->out_stride_tok;
  a.out_stride_head = p->out_stride_head;
  a.lse = p->lse;
  a.part = part;
  a.error = error;
  a.cut = reinterpret_cast<AtCut*>(ws + pl.cut_off);
  a.start = reinterpret_cast<AtRun*>(ws + pl.start_off);
  a.range = p->row_begin || p->row_end ? reinterpret_cast<int2*>(ws + pl.range_off) : nullptr;
  a.part_ml = reinterpret_cast<float2*>(ws + pl.ml_off);
  a.part_o = reinterpret_cast<float*>(ws + pl.o_off);
  a.num_tokens = p->num_tokens;
  a.slots = pl.slots;
  a.group = pl.g;
  a.tok_tile = pl.tok_tile;
  a.h_q = p->h_q;
  a.causal = p->causal;
  // (places: tiles of a unit and its end, for each of 32 slots and every KV head)
  a.few = pl.slots <= 32 && (int64_t)32 * pl.pages.h_kv * (pl.pages.max_rows / kAtKeys + 1 + kAtEnd) < (1ll << 31) - pl.grid;
  a.ranged = !a.few;
  a.by_unit = divisor(2 * pl.tok_tile);
  a.by_page = divisor(pl.pages.page_rows / 16);
  a.by_group = divisor(pl.g);
  a.by_cta = divisor(pl.grid);
  a.ctas = pl.grid;
  a.rows_cap = pl.rows_cap;
  a.box_shift = 0;
  while ((1 << a.box_shift) < box_rows(pl.pages.page_rows)) ++a.box_shift;
  a.scale_log2 = (float)(1.4426950408889634 * (double)p->scale);
  if (part.out) return launch_at<true>(p, pl, a, s);
  return launch_at<false>(p, pl, a, s);
}

}  // namespace aircache

using namespace aircache;

extern "C" {

size_t aircache_paged_attend_workspace_size(const aircache_paged_attend_problem* p) {
  AttendPlan pl;
  return attend_plan(p, false, pl) == AIRCACHE_OK ? pl.total : 0;
}

int aircache_paged_attend(const aircache_paged_attend_problem* p, void* ws, size_t ws_bytes, void* stream) {
  AttendPlan pl;
  const int rc = attend_plan(p, false, pl);
  if (rc != AIRCACHE_OK) return rc;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) return AIRCACHE_ERR_INVALID_ARG;
  if (ws_bytes < pl.total) return AIRCACHE_ERR_WORKSPACE;
  if (p->pages->num_seqs == 0 || p->num_tokens == 0) return AIRCACHE_OK;
  return attend_launch(p, pl, AttendPart{nullptr, nullptr}, static_cast<uint8_t*>(ws), static_cast<int32_t*>(ws),
                       static_cast<cudaStream_t>(stream));
}

}  // extern "C"
