// One decode step of attention over a paged cache (aircache_paged_decode).
//
//   x_j = scale q . k_j,  o = sum_j exp(x_j - m) v_j / l,  l = sum_j exp(x_j - m),
//   mass_j += sum over the KV head's query heads of exp(x_j - m) / l.
//
// 4 g D operations for the 4 D bytes of a row's key and value (g query heads to a
// KV head): bound by HBM.  The batch's rows form one list of 64-row tiles,
// sequence by sequence and KV head by KV head, and every CTA takes an equal run
// of it, so ragged lengths leave no CTA idle.  A producer warp looks the pages
// up and copies each tile as four 16-row pieces (TMA; a page is a multiple of 16
// rows, so a piece never crosses one) into a ring of stages; four consumer warps
// take one piece each: S = Q K^T (16 query heads by 16 rows) and
// O^T += V^T P^T (16 columns by 8 heads, so up to 8 query heads pad nothing
// there) with mma.sync; tcgen05's 128-row operand would be seven eighths padding
// or more.  S's accumulators are P^T's operand as they are.  Between them an
// online softmax in base 2 whose reference moves only when a logit passes it by
// more than a few powers of two (a vote of the warp): the weights are then at
// most 2^8 (2 in f16), O is rarely rescaled, and no row maximum is formed
// otherwise.
//
// A (sequence, KV head) that several CTAs share is joined by a second kernel, in
// the order of the CTAs; it also turns the logits, which the first one stores
// when the rows' mass is wanted, into weights.  (Joined by the last CTA to
// arrive, a fence and an atomic after the partial results and a reload in the
// last one cost 8 us at the end of a 16 x 16k step, more than the launch, which
// starts while the first kernel runs.)
//
// Short sequences need neither the list nor the second kernel: a cluster of one to
// eight CTAs takes a (sequence, KV head), an equal part of its tiles each, and they
// join their parts, form the log-sum-exps and add to the mass themselves, through
// each other's shared memory (one of 701 rows: 7.3 us, a quarter longer by the list).
//
// int8 rows carry a scale each.  The key's multiplies the logit.  The value's
// joins the weight before it is rounded to f16: the weights of O are
// exp2(x_j + log2 s_j) against their own reference, and the sum l keeps its own.
// These rows are bound by the instructions that widen their codes and by the
// latency between them, not by bytes.
//
// The product with V takes 16-bit weights: bf16 ones as a sum of two (what
// rounding takes away goes through a second product, which costs no time beside
// the bytes), f16 ones (int8 rows) rounded once, to 2^-12, because these rows are
// bound by instructions and a second product is more of them.  Maximum, sum, O and the joins are fp32, and out is rounded
// once, to bf16.
//
// Measured (28 query and 4 KV heads of 128, calls back to back): 16 x 16,384
// bf16 rows 87 us (537 MB, 6.2 TB/s), with mass 102 to 105 us; 8 x 32,768 int8 rows
// 65 us (277 MB), with mass 75; 32 heads of 64 over 55,113 rows 74 to 88 us (452 MB,
// 5.1 to 6.1 TB/s, by the machine); one sequence of
// 8,192 rows 11 us, of 131,072 49 us; of 701, in one launch, 7.3 us; 16 x 16,384 of
// one KV head to 16 query heads 33 us, int8 30.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "attend.cuh"
#include "pages.cuh"
#include "rowmma.cuh"
#include "tmap.cuh"

namespace aircache {
namespace {

constexpr int kPdRows = 64;   // rows of a tile
constexpr int kPdWarps = 4;   // consumer warps, 16 rows each
constexpr int kPdThreads = (kPdWarps + 1) * 32;
constexpr int kPdGroup = 16;  // query heads of a KV head, at most
constexpr int kPdRanks = 8;     // CTAs of a cluster, at most
constexpr int kPdHeader = 256;  // workspace: error word, then the tile count of the last call

// HB: blocks of eight query heads.
template <int D, bool Q8, int HB>
struct PdCfg {
  static constexpr int kPiece = 16 * D * (Q8 ? 1 : 2);  // 16 rows of K or of V
  static constexpr int kTile = kPdWarps * kPiece;
  static constexpr int kStageBytes = 2 * kTile;
  static constexpr int kStages = (Q8 ? 65536 : 98304) / kStageBytes;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kCtas = HB == 1 ? 3 : 2;               // to an SM, for the registers
  static constexpr int kScratch = 8 * HB * D * 4;             // the warps' joined O
  static constexpr int kScales = Q8 ? kStages * 2 * kPdRows * 4 : 0;
  static constexpr int kMl = (kPdWarps + 1) * kPdGroup * 3 * 4 + kPdGroup * 4;  // (m, l, n) of each warp and
                                                              // head, of the CTA, and the heads' log-sum-exps
  static constexpr int kSmem = 1024 + kRing + kScratch + kScales + kMl + kStages * (8 + 8 + 4) + 448;
  static_assert(kSmem <= (Q8 && HB == 1 ? 75 : 113) * 1024, "CTAs per SM, as ctas_per_sm() says");
};
// CTAs to an SM: two rings of 96 KB keep enough bytes in flight for bf16 rows.  int8 rows are bound
// by the instructions that widen them: a third CTA gives them more warps to issue from.
constexpr int ctas_per_sm(bool q8, int group) { return q8 && group <= 8 ? 3 : 2; }

// A query head's result under the reference m and the sum l next to what it joins: factors of the two, and the
// log-sum-exp in base 2 (-inf: no rows).  prior < 0: there is no prior result.  (One whose factor is 0 takes part: 0
// times what is not finite is NaN, as for a row whose weight is 0.)
struct Joint {
  float own, prior, lse2;
};

// What the mass kernel needs of a tile: its place, and its pieces' pages (-1: not there).
struct TileInfo {
  int s, h, i, pad;
  int page[4];
};

struct PdArgs {
  Pages pages;
  const __nv_bfloat16* q;
  int64_t q_stride_seq, q_stride_head;
  __nv_bfloat16* out;
  float* lse;
  float* mass_out;
  int32_t* error;
  int32_t* tiles;    // tile count, for the mass kernel
  int2* cut;         // [CTAs]: the unit that begins in the CTA and ends in another (-1: none), and its parts
  int2* unit;        // [S * h_kv]: the first CTA that has a part of it, and how many have one
  float* lse2;       // [S * h_q] base 2, of units that one CTA has whole
  DecodePrior prior; // a result over other rows that each sequence's joins
  float4* part_ml;   // [2 CTAs][g]: m, l, n of O
  float* part_o;     // [2 CTAs][g][D]
  TileInfo* info;    // [tiles]
  float* logits;     // [tiles][g][64], base 2
  int64_t total_rows;
  int h_q, group, ctas, ranks;  // ranks: CTAs to a unit (kernels of short sequences)
  float scale_log2;
};

// Keys and values pass through L2 once: they are to go first, so that the stored logits stay for the
// mass (without the policy 16 x 16k with mass takes 3 % longer, 64-wide heads 5 %).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, int a, int b, int c, int d, int e,
                                            uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, "
      "{%2, %3, %4, %5, %6}], [%7], %8;\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// Rows of sequence s that count: 0 when its length is out of bounds.
__device__ __forceinline__ int rows_of(const Pages& p, int s) {
  const int n = p.lens[s];
  return n >= 0 && n <= p.max_rows ? n : 0;
}

// `head` of the batch's S * h_q.  Without a prior result there is nothing to form (own = 1).
__device__ __forceinline__ Joint joint(const PdArgs& a, int64_t head, float m, float l) {
  prior_wait();
  Joint j = {1.f, -1.f, l == 0.f ? -INFINITY : m + log2f(l)};
  if (head >= (int64_t)*a.prior.from * a.h_q && head < (int64_t)*a.prior.num * a.h_q) {
    const float p = a.prior.lse2[head];
    if (p != -INFINITY) {
      const float top = fmaxf(j.lse2, p);  // (a NaN stays one in the factor of its own)
      const float x = fast_exp2(j.lse2 - top), y = fast_exp2(p - top), z = x + y;
      j.own = x / z;
      j.prior = y / z;
      j.lse2 = top + log2f(z);
    }
  }
  return j;
}
// Four columns of a head's output: y times f is the result over its own rows.
template <int D>
__device__ __forceinline__ float4 join_prior(const PdArgs& a, const Joint& j, int64_t head, int d, float4 y) {
  y.x *= j.own, y.y *= j.own, y.z *= j.own, y.w *= j.own;
  if (!(j.prior < 0.f)) {
    const float4 p = *reinterpret_cast<const float4*>(a.prior.out + head * D + d);
    y.x = fmaf(p.x, j.prior, y.x);
    y.y = fmaf(p.y, j.prior, y.y);
    y.z = fmaf(p.z, j.prior, y.z);
    y.w = fmaf(p.w, j.prior, y.w);
  }
  return y;
}
// Writes four columns, and with the first of them the log-sum-exp.  f: what makes y the result over the own rows.
template <int D, bool PRIOR>
__device__ __forceinline__ void write_columns(const PdArgs& a, int64_t head, int d, float4 y, float f, float m, float l,
                                              bool lse2 = false) {
  y.x *= f, y.y *= f, y.z *= f, y.w *= f;
  float top = 0.f;
  if (PRIOR) {
    const Joint j = joint(a, head, m, l);
    y = join_prior<D>(a, j, head, d, y);
    top = j.lse2;
  } else if (d == 0) {
    top = l == 0.f ? -INFINITY : m + log2f(l);
  }
  const __nv_bfloat162 x[2] = {__floats2bfloat162_rn(y.x, y.y), __floats2bfloat162_rn(y.z, y.w)};
  *reinterpret_cast<uint2*>(a.out + head * D + d) = *reinterpret_cast<const uint2*>(x);
  if (d == 0 && a.lse) a.lse[head] = top * 0.69314718055994531f;
  if (d == 0 && lse2) a.lse2[head] = top == -INFINITY ? INFINITY : top;
}
// The log-sum-exp that turns a head's logits into weights (inf: none has one).
template <bool PRIOR>
__device__ __forceinline__ float mass_lse2(const PdArgs& a, int64_t head, float m, float l) {
  const float x = PRIOR ? joint(a, head, m, l).lse2 : l == 0.f ? -INFINITY : m + log2f(l);
  return x == -INFINITY ? INFINITY : x;
}

// How the batch's tiles are dealt out: the units (the sequences' KV heads) lie
// one after the other on a line, each with its tiles and then `kPdEnd` places
// without work, which stand for the time that a unit's end costs the CTAs it
// falls to (merging the warps, writing, joining, the next queries).  CTA c
// takes the places c * per .. c * per + per - 1, so the parts of a unit go to
// consecutive CTAs and only its first and its last run can be a part.  (48 ragged
// sequences with mass: 7 % longer than with 4 places with none, 2 % with 2 or 16.)
constexpr uint32_t kPdEnd = 4;

// A run of tiles of one unit: what a CTA does at a time.
struct Run {
  int s, h, len;         // the unit: its sequence, KV head and rows,
  uint32_t tiles, unit;  // tiles and its first place on the line;
  uint32_t first, count; // the CTA's tiles of it,
  uint32_t at;           // the batch's tiles before `first`
};

// The part of unit (s, h) at place `unit` that lies in the CTA's places lo .. hi-1.
__device__ __forceinline__ void clip_run(Run& r, uint32_t lo, uint32_t hi) {
  const uint32_t from = max(r.unit, lo), to = min(r.unit + r.tiles, hi);
  r.first = from - r.unit;
  r.count = to > from ? to - from : 0;
}

// Moves to the next unit that has tiles in the CTA's places; false if there is none.
__device__ __forceinline__ bool next_run(const Pages& p, Run& r, uint32_t lo, uint32_t hi) {
  r.at += r.tiles - r.first;
  r.unit += r.tiles + kPdEnd;
  if (r.unit >= hi) return false;
  if (++r.h == p.h_kv) {
    r.h = 0;
    do {
      if (++r.s >= p.num_seqs) return false;
      r.len = rows_of(p, r.s);
    } while (r.len == 0);
    r.tiles = (r.len + kPdRows - 1) / kPdRows;
  }
  clip_run(r, lo, hi);
  return true;
}

struct Share {
  int32_t tiles;  // of the batch; negative: too many, and nothing is computed
  uint32_t per, lo, hi;
  Run run;        // the CTA's first (count may be 0: the places behind a unit)
};
struct ShareScratch {
  uint32_t places[8], tiles[8];
  int64_t rows[8];
  Run run;
};
// By all threads of the CTA: lengths are summed by runs of consecutive sequences, one to a thread.
__device__ __forceinline__ Share make_share(const PdArgs& a, ShareScratch* sc) {
  const Pages& p = a.pages;
  constexpr int kWarps = kPdThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (p.num_seqs + kPdThreads - 1) / kPdThreads;
  const int s0 = min(tid * each, p.num_seqs), s1 = min(s0 + each, p.num_seqs);
  uint32_t tiles = 0, places = 0;
  int64_t rows = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = rows_of(p, s);
    if (n != p.lens[s] && blockIdx.x == 0) set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
    const uint32_t t = (n + kPdRows - 1) / kPdRows;
    tiles += t;
    places += t ? t + kPdEnd : 0;
    rows += n;
  }
  uint32_t incl_p = places, incl_t = tiles;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl_p, off), y = __shfl_up_sync(0xffffffffu, incl_t, off);
    if (lane >= off) incl_p += x, incl_t += y;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, off);
  if (lane == 31) sc->places[warp] = incl_p, sc->tiles[warp] = incl_t;
  if (lane == 0) sc->rows[warp] = rows;
  __syncthreads();
  uint32_t before = incl_p - places, tiles_before = incl_t - tiles, total = 0, all_tiles = 0;
  int64_t all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sc->places[w], tiles_before += sc->tiles[w];
    total += sc->places[w];
    all_tiles += sc->tiles[w];
    all += sc->rows[w];
  }
  Share sh;
  if (all > a.total_rows) {  // (only then could the counts above have passed 32 bits)
    if (blockIdx.x == 0 && tid == 0) set_error(a.error, AIRCACHE_ERR_CAPACITY);
    sh.tiles = -1;
    sh.per = sh.lo = sh.hi = 0;
    return sh;
  }
  const uint32_t h_kv = p.h_kv;
  total *= h_kv;
  sh.tiles = (int32_t)(all_tiles * h_kv);
  sh.per = max(1u, (total + gridDim.x - 1) / gridDim.x);
  sh.lo = min(sh.per * blockIdx.x, total);
  sh.hi = min(sh.lo + sh.per, total);
  if (sh.lo < sh.hi && sh.lo >= before * h_kv && sh.lo < (before + places) * h_kv) {
    uint32_t at = before * h_kv, t_at = tiles_before * h_kv;
    for (int s = s0; s < s1; ++s) {
      const int n = rows_of(p, s);
      const uint32_t t = (n + kPdRows - 1) / kPdRows, wide = t ? t + kPdEnd : 0;
      if (sh.lo < at + wide * h_kv) {
        Run r;
        r.s = s;
        r.h = (int)((sh.lo - at) / wide);
        r.len = n;
        r.tiles = t;
        r.unit = at + r.h * wide;
        clip_run(r, sh.lo, sh.hi);
        if (r.count == 0) r.first = t;
        r.at = t_at + r.h * t + r.first;
        sc->run = r;
        break;
      }
      at += wide * h_kv;
      t_at += t * h_kv;
    }
  }
  __syncthreads();
  sh.run = sc->run;
  return sh;
}

// Short sequences: `ranks` CTAs (a cluster) to a unit, with an equal part of its tiles each.
__device__ __forceinline__ Share make_unit(const PdArgs& a, ShareScratch* sc) {
  const Pages& p = a.pages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / a.ranks, rank = blockIdx.x % a.ranks;
  Share sh;
  Run& r = sh.run;
  r.s = unit / p.h_kv;
  r.h = unit % p.h_kv;
  r.len = rows_of(p, r.s);
  r.tiles = (r.len + kPdRows - 1) / kPdRows;
  r.unit = 0;
  sh.per = (r.tiles + a.ranks - 1) / a.ranks;
  r.first = min(rank * sh.per, r.tiles);
  r.count = min(sh.per, r.tiles - r.first);
  uint32_t tiles = 0;  // of the sequences before
  int64_t rows = 0;
  for (int s = tid; s < p.num_seqs; s += kPdThreads) {
    const int n = rows_of(p, s);
    if (n != p.lens[s] && blockIdx.x == 0) set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
    rows += n;
    if (s < r.s) tiles += (n + kPdRows - 1) / kPdRows;
  }
  tiles = __reduce_add_sync(0xffffffffu, tiles);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, off);
  if (lane == 0) sc->tiles[warp] = tiles, sc->rows[warp] = rows;
  __syncthreads();
  int64_t all = 0;
  tiles = 0;
#pragma unroll
  for (int w = 0; w < kPdThreads / 32; ++w) all += sc->rows[w], tiles += sc->tiles[w];
  r.at = tiles * p.h_kv + r.h * r.tiles + r.first;
  sh.lo = 0;
  sh.hi = r.tiles > 0;
  sh.tiles = 0;
  if (all > a.total_rows) {
    if (blockIdx.x == 0 && tid == 0) set_error(a.error, AIRCACHE_ERR_CAPACITY);
    sh.tiles = -1;
    sh.hi = 0;
  }
  return sh;
}

// SHORT: a cluster to a unit, and no second kernel.  PRIOR: the results are joined with those over other rows.
template <int D, bool Q8, int HB, bool SHORT, bool PRIOR>
__global__ void __launch_bounds__(kPdThreads, PdCfg<D, Q8, HB>::kCtas) paged_decode_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                  const __grid_constant__ CUtensorMap vmap,
                                                                  const __grid_constant__ PdArgs a) {
  using C = PdCfg<D, Q8, HB>;
  extern __shared__ uint8_t pd_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(pd_raw) + 1023) & ~uintptr_t(1023));
  float* scratch = reinterpret_cast<float*>(ring + C::kRing);               // [8 HB][D], swizzled
  float* scales = reinterpret_cast<float*>(ring + C::kRing + C::kScratch);  // [stages][K, V][64]
  float* mlw = reinterpret_cast<float*>(ring + C::kRing + C::kScratch + C::kScales);  // [4][16][3]
  float* part = mlw + kPdWarps * kPdGroup * 3;  // [16][3]
  float* lse2 = part + kPdGroup * 3;            // [16]
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(mlw) + C::kMl);
  uint64_t* empty = full + C::kStages;
  ShareScratch* share = reinterpret_cast<ShareScratch*>(empty + C::kStages);
  uint32_t* pieces = reinterpret_cast<uint32_t*>(share + 1);  // [stages] which pieces of a tile are there

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = a.group;
  const Pages& p = a.pages;
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kPdWarps);
    }
    fence_mbar_init();
  }
  if (warp == kPdWarps && lane == 0) {
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
  }
  // With a prior result the kernel before is the one that makes it, and writes nothing else that is read here: the rows
  // are read while it runs, and what joins waits for it (prior_wait), as the kernel's end does.  The kernel behind may
  // start early only if it is this call's own, the join of the list's parts
  constexpr bool late = PRIOR;
  if (!late) pdl_wait();
  if (!late || !SHORT) pdl_trigger();
  const Share sh = SHORT ? make_unit(a, share) : make_share(a, share);  // (its barriers publish the mbarriers too)
  if (!SHORT && blockIdx.x == 0 && tid == 0) *a.tiles = max(sh.tiles, 0);
  Run r = sh.run;

  if (warp == kPdWarps) {
    // ---- producer warp: lane j of 32 holds the page of the j-th 16-row piece
    // ahead (8 tiles); 0-3 copy keys, 4-7 values, 8-15 the scales of int8 rows
    const uint64_t policy = l2_evict_first_policy();
    int st = 0;
    uint32_t phase = 0, filled = 0;
    bool alive = true;
    for (bool more = sh.lo < sh.hi; more && alive; more = !SHORT && next_run(p, r, sh.lo, sh.hi)) {
      const int32_t* table = p.table + (int64_t)r.s * p.table_stride;
      int page = -1;
      for (uint32_t i = 0; i < r.count; ++i) {
        if ((i & 7) == 0) {
          const int row = (int)((r.first + i) * 4 + lane) * 16;
          page = -1;
          if (row < r.len && row < (int)((r.first + r.count) * kPdRows)) {
            page = table[row / p.page_rows];
            if (!page_ok(p, page)) {
              set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
              page = -1;
            }
          }
        }
        const int piece = lane & 3;
        const int pg = __shfl_sync(0xffffffffu, page, (i & 7) * 4 + piece);
        const uint32_t mask = __ballot_sync(0xffffffffu, pg >= 0) & 15u;
        if (filled >= C::kStages) {
          if (!mbar_wait_warp(&empty[st], phase ^ 1)) {
            set_error(a.error, AIRCACHE_ERR_DEVICE_TIMEOUT);
            alive = false;
            if (!SHORT && a.mass_out) {
              // the tiles from here on are not there: the mass kernel would find another call's pages in their place
              do {
                for (; i < r.count; ++i) {
                  if (lane < 4) a.info[r.at + i].page[lane] = -1;
                  if (lane == 4) *reinterpret_cast<int4*>(&a.info[r.at + i]) = make_int4(r.s, r.h, r.first + i, 0);
                }
                i = 0;
              } while (next_run(p, r, sh.lo, sh.hi));
            }
            break;
          }
        }
        uint8_t* dst = ring + st * C::kStageBytes + piece * C::kPiece;
        if (lane == 0) {
          pieces[st] = mask;
          fence_proxy_async_smem();  // the consumers' generic accesses of this stage come first
          mbar_arrive_expect_tx(&full[st], __popc(mask) * (2 * C::kPiece + (Q8 ? 128 : 0)));
        }
        __syncwarp();
        const int row = (int)(((r.first + i) * 4 + piece) * 16) % p.page_rows;
        if (pg >= 0 && lane < 8) {
          fence_proxy_async_smem();
          const uint32_t to = smem_u32(dst) + (lane >= 4 ? C::kTile : 0);
          const CUtensorMap* map = lane >= 4 ? &vmap : &kmap;
          if constexpr (Q8)
            tma_load_4d_hint(to, map, 0, row, r.h, pg, &full[st], policy);
          else
            tma_load_5d(to, map, 0, row, 0, r.h, pg, &full[st], policy);
        }
        if constexpr (Q8) {
          if (pg >= 0 && lane >= 8 && lane < 16) {
            fence_proxy_async_smem();
            const int64_t slot = page_slot(p, pg, r.h, row);
            bulk_g2s(scales + (st * 2 + (lane >= 12)) * kPdRows + piece * 16,
                     (lane >= 12 ? p.v_scale : p.k_scale) + slot, 64, &full[st]);
          }
        }
        if (!SHORT && a.mass_out) {
          const uint32_t t = r.at + i;
          if (lane < 4) a.info[t].page[lane] = pg;
          if (lane == 4) *reinterpret_cast<int4*>(&a.info[t]) = make_int4(r.s, r.h, r.first + i, 0);
        }
        ++filled;
        if (++st == C::kStages) st = 0, phase ^= 1;
      }
    }
    // every copy has landed before the CTA's shared memory is another's (consumers whose wait ran out left some behind)
    for (uint32_t f = filled > C::kStages ? filled - C::kStages : 0; f < filled; ++f)
      (void)mbar_wait_warp(&full[f % C::kStages], (f / C::kStages) & 1);
    if (SHORT && sh.lo < sh.hi) {  // (the consumers' barriers are the whole cluster's)
      cluster_sync_all();
      cluster_sync_all();
    }
    if (late) prior_wait();
    return;
  }

  // ---- consumers
  const int hA = lane >> 2, cq = lane & 3;  // S: heads hA and hA + 8, rows 2cq, 2cq + 1 of each eight
  if (!SHORT && tid == 0) a.cut[blockIdx.x] = make_int2(-1, 0);  // (until a run says otherwise)
  // sequences without rows: out = 0, lse = -inf
  for (int s = blockIdx.x; s < p.num_seqs && sh.tiles >= 0; s += gridDim.x) {
    if (rows_of(p, s) != 0) continue;
    for (int i = tid; i < a.h_q * (D / 4); i += kPdWarps * 32)
      write_columns<D, PRIOR>(a, (int64_t)s * a.h_q + i / (D / 4), i % (D / 4) * 4, make_float4(0.f, 0.f, 0.f, 0.f), 0.f, 0.f, 0.f);
    for (int i = tid; i < p.h_kv && !SHORT; i += kPdWarps * 32) a.unit[s * p.h_kv + i] = make_int2(0, 0);
  }
  int st = 0;
  uint32_t phase = 0;
  bool alive = true;
  for (bool more = sh.lo < sh.hi; more; more = !SHORT && next_run(p, r, sh.lo, sh.hi)) {
    if (!SHORT && r.count == 0) continue;
    // ---- the group's queries as A fragments (heads at or past g: zeros)
    uint32_t qa[D / 16][2 * HB];
#pragma unroll
    for (int b = 0; b < HB; ++b) {
      const bool in = hA + 8 * b < g;
      const __nv_bfloat16* q = a.q + (int64_t)r.s * a.q_stride_seq + (int64_t)(r.h * g + hA + 8 * b) * a.q_stride_head;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        uint2 x = make_uint2(0u, 0u);
        if (in) {
          if constexpr (Q8) {
            // k-step kk of quad lane cq covers d = cq*D/4 + 4kk + 0..3, as the key codes are read below
            x = *reinterpret_cast<const uint2*>(q + cq * (D / 4) + 4 * kk);
          } else {
            x.x = *reinterpret_cast<const uint32_t*>(q + 16 * kk + 2 * cq);
            x.y = *reinterpret_cast<const uint32_t*>(q + 16 * kk + 2 * cq + 8);
          }
        }
        qa[kk][b] = x.x;
        qa[kk][HB + b] = x.y;
      }
    }
    float kmult[HB];  // of head hA + 8b
#pragma unroll
    for (int b = 0; b < HB; ++b) {
      kmult[b] = a.scale_log2;
      if constexpr (Q8) {
        // Q enters the f16 product times the power of two that puts its head's largest |q| in
        // [2^14, 2^15): exact, and undone in the logit's multiplier.  Each head by its own, so that none
        // pushes another's values out of f16's range
        float mx = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int j = b; j < 2 * HB; j += HB) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qa[kk][j]));
            mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        float qscale = 1.f;
        if (mx > 0.f && mx < INFINITY) {
          int ex;
          (void)frexpf(mx, &ex);
          qscale = ldexpf(1.f, min(15 - ex, 120));
        }
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int j = b; j < 2 * HB; j += HB) {
            const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&qa[kk][j]));
            const __half2 hq = __floats2half2_rn(f.x * qscale, f.y * qscale);
            qa[kk][j] = *reinterpret_cast<const uint32_t*>(&hq);
          }
        kmult[b] /= qscale;
      }
    }
    // o[t][b]: columns 16t + hA and + 8 (rows of the product), heads 8b + 2cq and + 1
    float o[D / 16][HB][4];
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
      for (int b = 0; b < HB; ++b) o[t][b][0] = o[t][b][1] = o[t][b][2] = o[t][b][3] = 0.f;
    // of head hA + 8b: the sum's reference and this lane's part of the sum; O's reference (the
    // same, but for int8 rows).  Before any row: fp32's lowest, not -inf, against which a
    // logit under fp32's range would weigh NaN where it weighs nothing
    float m[HB], l[HB], n[HB];
#pragma unroll
    for (int b = 0; b < HB; ++b) m[b] = n[b] = -FLT_MAX, l[b] = 0.f;
    static_assert(kP16 == 16384.f, "2^14, as the weights' exponent takes it");
    constexpr float kSlack = 8.f, kSlack16 = 1.f;  // (f16 weights carry 2^14: 2^15 is the most they may reach)

    for (uint32_t i = 0; i < r.count && alive; ++i) {
      if (!mbar_wait_warp(&full[st], phase)) {
        if (lane == 0) set_error(a.error, AIRCACHE_ERR_DEVICE_TIMEOUT);
        alive = false;
        break;
      }
      const int valid = (pieces[st] >> warp) & 1 ? min(16, r.len - (int)(r.first + i) * kPdRows - 16 * warp) : 0;
      if (valid > 0) {
        uint8_t* kt = ring + st * C::kStageBytes + warp * C::kPiece;
        uint8_t* vt = kt + C::kTile;
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        float ks[HB][4], lv[4] = {0.f, 0.f, 0.f, 0.f};  // rows 2cq, 2cq+1, 2cq+8, 2cq+9
        auto qk = [&](int t, int kk, uint32_t b0, uint32_t b1) {
          const uint32_t af[4] = {qa[kk][0], HB == 2 ? qa[kk][1] : 0u, qa[kk][HB], HB == 2 ? qa[kk][3] : 0u};
          mma16816<Q8>(sc[t], af, b0, b1);
        };
        if constexpr (Q8) {
          const float* sk = scales + st * 2 * kPdRows + 16 * warp;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = 2 * cq + (j & 1) + 8 * (j >> 1);
#pragma unroll
            for (int b = 0; b < HB; ++b) ks[b][j] = kmult[b] * sk[row];
            lv[j] = row < valid ? __log2f(sk[kPdRows + row]) : 0.f;  // (past the end a scale may be anything)
          }
#pragma unroll
          for (int t = 0; t < 2; ++t) {  // (one eight of rows after the other: fewer registers at a time)
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
              const uint4 x =
                  *reinterpret_cast<const uint4*>(kt + swz8<D>((8 * t + hA) * D + cq * (D / 4) + 16 * w));
              const uint32_t k4[4] = {x.x ^ 0x80808080u, x.y ^ 0x80808080u, x.z ^ 0x80808080u, x.w ^ 0x80808080u};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                qk(t, 4 * w + e, widen2_f16(k4[e], 0x4140u), widen2_f16(k4[e], 0x4342u));
            }
          }
        } else {
          if (valid < 16) {
            // rows past the end may hold anything: zero their V so that weights of 0 add exactly 0
            for (int c = lane; c < 16 * (D / 8); c += 32) {
              const int rr = c / (D / 8), rest = c % (D / 8);
              if (rr >= valid)
                *reinterpret_cast<uint4*>(vt + (rest >> 3) * 2048 + rr * 128 + (rest & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
            }
            __syncwarp();
          }
          const uint32_t kb = smem_u32(kt);
          const int mi = lane >> 3, row = (lane & 7) + 8 * (mi >> 1);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t kf[4];
            ldsm_x4(kf, swz(kb + (kk >> 2) * 2048, row, 2 * (kk & 3) + (mi & 1)));
            qk(0, kk, kf[0], kf[1]);
            qk(1, kk, kf[2], kf[3]);
          }
        }
        // base-2 logits; rows at or past `valid` get weight 0
        bool over = false;
        float top[HB], ytop[HB];
#pragma unroll
        for (int b = 0; b < HB; ++b) {
          top[b] = ytop[b] = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float& x = sc[j >> 1][2 * b + (j & 1)];
            const bool in = 8 * (j >> 1) + 2 * cq + (j & 1) < valid;
            x = in ? x * (Q8 ? ks[b][j] : kmult[b]) : -INFINITY;
            top[b] = fmaxf(top[b], x);
            if (Q8) ytop[b] = fmaxf(ytop[b], x + lv[j]);
          }
          over |= top[b] > m[b] + kSlack;
          if (Q8) over |= ytop[b] > n[b] + kSlack16;
        }
        if (a.mass_out) {
          float* lg = a.logits + (int64_t)(r.at + i) * g * kPdRows + 16 * warp + 2 * cq;
#pragma unroll
          for (int b = 0; b < HB; ++b)
            if (hA + 8 * b < g)
#pragma unroll
              for (int t = 0; t < 2; ++t)
                *reinterpret_cast<float2*>(lg + (hA + 8 * b) * kPdRows + 8 * t) =
                    make_float2(sc[t][2 * b], sc[t][2 * b + 1]);
        }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int b = 0; b < HB; ++b) {
            float x = fmaxf(top[b], __shfl_xor_sync(0xffffffffu, top[b], 1));
            x = fmaxf(m[b], fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2)));
            float f = fast_exp2(m[b] - x);
            l[b] *= f;
            m[b] = x;
            if (Q8) {
              float y = fmaxf(ytop[b], __shfl_xor_sync(0xffffffffu, ytop[b], 1));
              y = fmaxf(n[b], fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2)));
              f = fast_exp2(n[b] - y);
              n[b] = y;
            }
            const float f0 = __shfl_sync(0xffffffffu, f, 8 * cq), f1 = __shfl_sync(0xffffffffu, f, 8 * cq + 4);
#pragma unroll
            for (int t = 0; t < D / 16; ++t) {
              o[t][b][0] *= f0;
              o[t][b][1] *= f1;
              o[t][b][2] *= f0;
              o[t][b][3] *= f1;
            }
          }
        }
        // the sum takes the weights before they are rounded: lse and mass need it
        uint32_t pb[HB][2], pl[HB][2];  // (pl: what rounding to bf16 takes from them)
#pragma unroll
        for (int b = 0; b < HB; ++b)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float x0 = sc[t][2 * b], x1 = sc[t][2 * b + 1];
            const float w0 = fast_exp2(x0 - m[b]), w1 = fast_exp2(x1 - m[b]);
            l[b] += w0 + w1;
            if constexpr (Q8) {
              // (2^14 enters the exponent: kP16 exp2(y - n) = exp2(y - (n - 14)))
              const __half2 h = __floats2half2_rn(fast_exp2(x0 + lv[2 * t] - (n[b] - 14.f)),
                                                  fast_exp2(x1 + lv[2 * t + 1] - (n[b] - 14.f)));
              pb[b][t] = *reinterpret_cast<const uint32_t*>(&h);
            } else {
              const __nv_bfloat162 h = __floats2bfloat162_rn(w0, w1);
              pb[b][t] = *reinterpret_cast<const uint32_t*>(&h);
              const __nv_bfloat162 r = __floats2bfloat162_rn(w0 - __low2float(h), w1 - __high2float(h));
              pl[b][t] = *reinterpret_cast<const uint32_t*>(&r);
            }
          }
        if constexpr (Q8) {
          // lane (hA, cq) takes rows 2cq, 2cq+1, 2cq+8, 2cq+9, value columns hA*(D/8) .. +D/8-1:
          // product row hA of m-tile t is the value column hA*(D/8) + 2t, row hA + 8 the next one
#pragma unroll
          for (int half = 0; half < D / 64; ++half) {  // eight columns of each row at a time
            uint2 v8[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              v8[j] = *reinterpret_cast<const uint2*>(
                  vt + swz8<D>((2 * cq + (j & 1) + 8 * (j >> 1)) * D + hA * (D / 8)) + 8 * half);
              v8[j].x ^= 0x80808080u;
              v8[j].y ^= 0x80808080u;
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {  // four columns: two rows' bytes interleaved, two columns to a word
              const uint32_t r0 = w ? v8[0].y : v8[0].x, r1 = w ? v8[1].y : v8[1].x;
              const uint32_t r2 = w ? v8[2].y : v8[2].x, r3 = w ? v8[3].y : v8[3].x;
              const uint32_t x0 = __byte_perm(r0, r1, 0x5140), x1 = __byte_perm(r0, r1, 0x7362);
              const uint32_t y0 = __byte_perm(r2, r3, 0x5140), y1 = __byte_perm(r2, r3, 0x7362);
              const uint32_t va[4] = {widen2_f16(x0, 0x4140u), widen2_f16(x0, 0x4342u), widen2_f16(y0, 0x4140u),
                                      widen2_f16(y0, 0x4342u)};
              const uint32_t vb[4] = {widen2_f16(x1, 0x4140u), widen2_f16(x1, 0x4342u), widen2_f16(y1, 0x4140u),
                                      widen2_f16(y1, 0x4342u)};
#pragma unroll
              for (int b = 0; b < HB; ++b) {
                mma16816<true>(o[4 * half + 2 * w][b], va, pb[b][0], pb[b][1]);
                mma16816<true>(o[4 * half + 2 * w + 1][b], vb, pb[b][0], pb[b][1]);
              }
            }
          }
        } else {
          const uint32_t vb = smem_u32(vt);
          const int mi = lane >> 3, row = (lane & 7) + 8 * (mi >> 1);
#pragma unroll
          for (int t = 0; t < D / 16; ++t) {
            uint32_t vf[4];
            ldsm_x4_trans(vf, swz(vb + (t >> 2) * 2048, row, 2 * (t & 3) + (mi & 1)));
#pragma unroll
            for (int b = 0; b < HB; ++b) {
              mma16816<false>(o[t][b], vf, pb[b][0], pb[b][1]);
              mma16816<false>(o[t][b], vf, pl[b][0], pl[b][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
      if (++st == C::kStages) st = 0, phase ^= 1;
    }

    // ---- join the four warps: (m, l, n) by all, then O in turns, each warp another quarter of the columns
    named_bar_sync(1, kPdWarps * 32);  // the last run's scratch and mlw are read
    // (addresses from here on are formed at each run's end, not held in registers through its tiles)
    int hA = lane >> 2, cq = lane & 3;
    asm volatile("" : "+r"(hA), "+r"(cq));
#pragma unroll
    for (int b = 0; b < HB; ++b) {
      float x = l[b] + __shfl_xor_sync(0xffffffffu, l[b], 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      if (cq == 0) {
        float* w = mlw + (warp * kPdGroup + hA + 8 * b) * 3;
        w[0] = m[b], w[1] = x, w[2] = Q8 ? n[b] : m[b];
      }
    }
    named_bar_sync(1, kPdWarps * 32);
    auto joined = [&](int hh, float& m, float& l, float& n) {
      m = n = -INFINITY;
      l = 0.f;
#pragma unroll
      for (int w = 0; w < kPdWarps; ++w) {
        m = fmaxf(m, mlw[(w * kPdGroup + hh) * 3]);
        n = fmaxf(n, mlw[(w * kPdGroup + hh) * 3 + 2]);
      }
#pragma unroll
      for (int w = 0; w < kPdWarps; ++w)
        l += mlw[(w * kPdGroup + hh) * 3 + 1] * fast_exp2(mlw[(w * kPdGroup + hh) * 3] - m);
    };
    // head hh's column d lies at d ^ 8 (hh / 2 mod 4): a warp's stores then fall into 32 banks
    auto place = [](int hh, int d) { return hh * D + (d ^ ((hh >> 1 & 3) << 3)); };
    {
      float c[HB][2];
#pragma unroll
      for (int b = 0; b < HB; ++b)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int hh = 8 * b + 2 * cq + e;
          float mm, ll, nn;
          joined(hh, mm, ll, nn);
          c[b][e] = fast_exp2(mlw[(warp * kPdGroup + hh) * 3 + 2] - nn);
        }
      auto put = [&](auto q, bool first) {
        constexpr int quarter = decltype(q)::value;
#pragma unroll
        for (int t = quarter * (D / 64); t < (quarter + 1) * (D / 64); ++t)
#pragma unroll
          for (int b = 0; b < HB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float* to = scratch + place(8 * b + 2 * cq + (j & 1), 16 * t + hA + 8 * (j >> 1));
              const float x = o[t][b][j] * c[b][j & 1];
              *to = first ? x : *to + x;
            }
      };
#pragma unroll 1
      for (int turn = 0; turn < 4; ++turn) {
        switch ((turn + warp) & 3) {
          case 0: put(std::integral_constant<int, 0>(), turn == 0); break;
          case 1: put(std::integral_constant<int, 1>(), turn == 0); break;
          case 2: put(std::integral_constant<int, 2>(), turn == 0); break;
          default: put(std::integral_constant<int, 3>(), turn == 0); break;
        }
        named_bar_sync(1, kPdWarps * 32);
      }
    }
    // int8 values: where the value column d went
    auto joined_o = [&](int hh, int d) {
      const int rem = d % (D / 8);
      return scratch[place(hh, Q8 ? 16 * (rem >> 1) + d / (D / 8) + 8 * (rem & 1) : d)];
    };
    const int64_t head0 = (int64_t)r.s * a.h_q + (int64_t)r.h * g;
    constexpr float kUndo = Q8 ? 1.f / kP16 : 1.f;
    if constexpr (SHORT) {
      if (tid < g) {
        float m, l, n;
        joined(tid, m, l, n);
        part[tid * 3] = m, part[tid * 3 + 1] = l, part[tid * 3 + 2] = n;
      }
      cluster_sync_all();
      const int rank = blockIdx.x % a.ranks;
      constexpr int kRanks = kPdRanks;
      // the ranks' references and sums of head hh: the common ones
      auto heads = [&](int hh, float m[kRanks], float l[kRanks], float n[kRanks], float& mm, float& ll, float& nn) {
#pragma unroll
        for (int j = 0; j < kRanks; ++j) {
          const uint32_t at = cluster_map(smem_u32(part + hh * 3), min(j, a.ranks - 1));
          m[j] = ld_cluster_f32(at);
          l[j] = ld_cluster_f32(at + 4);
          n[j] = ld_cluster_f32(at + 8);
        }
        mm = nn = -FLT_MAX;
        ll = 0.f;
#pragma unroll
        for (int j = 0; j < kRanks; ++j) mm = fmaxf(mm, m[j]), nn = fmaxf(nn, n[j]);
#pragma unroll
        for (int j = 0; j < kRanks; ++j)
          if (j < a.ranks) ll += l[j] * fast_exp2(m[j] - mm);
      };
      // four columns to a thread, the ranks in turn
      for (int c = rank + a.ranks * tid; c < g * (D / 4); c += a.ranks * kPdWarps * 32) {
        const int hh = c / (D / 4), d = c % (D / 4) * 4;
        float m[kRanks], l[kRanks], n[kRanks], mm, ll, nn, x[kRanks][4];
#pragma unroll
        for (int j = 0; j < kRanks; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rem = (d + e) % (D / 8);
            const int at = place(hh, Q8 ? 16 * (rem >> 1) + (d + e) / (D / 8) + 8 * (rem & 1) : d + e);
            x[j][e] = j < a.ranks ? ld_cluster_f32(cluster_map(smem_u32(scratch + at), j)) : 0.f;
          }
        heads(hh, m, l, n, mm, ll, nn);
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kRanks; ++j) {
          const float f = fast_exp2(n[j] - nn);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] += j < a.ranks ? f * x[j][e] : 0.f;
        }
        const float f = ll == 0.f ? 0.f : kUndo * fast_exp2(nn - mm) / ll;
        write_columns<D, PRIOR>(a, head0 + hh, d, make_float4(y[0], y[1], y[2], y[3]), f, mm, ll);
      }
      if (a.mass_out) {
        const int hh = tid - 3 * 32;
        if (hh >= 0 && hh < g) {
          float m[kRanks], l[kRanks], n[kRanks], mm, ll, nn;
          heads(hh, m, l, n, mm, ll, nn);
          lse2[hh] = mass_lse2<PRIOR>(a, head0 + hh, mm, ll);
        }
        named_bar_sync(1, kPdWarps * 32);  // (and the CTA's logits are written)
        for (int i = tid; i < (int)r.count * kPdRows; i += kPdWarps * 32) {
          const int row = r.first * kPdRows + i;
          if (row >= r.len) break;
          const int page = p.table[(int64_t)r.s * p.table_stride + row / p.page_rows];
          if (!page_ok(p, page)) continue;
          const int64_t slot = page_slot(p, page, r.h, row % p.page_rows);
          const float* lg = a.logits + (int64_t)(r.at + i / kPdRows) * g * kPdRows + i % kPdRows;
          float sum = 0.f, x[8];
          const float old = p.mass[slot];
          for (int q0 = 0; q0 < g; q0 += 8) {
#pragma unroll
            for (int q = 0; q < 8; ++q) x[q] = q0 + q < g ? lg[(q0 + q) * kPdRows] : -INFINITY;
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q0 + q < g) sum += fast_exp2(x[q] - lse2[q0 + q]);
          }
          a.mass_out[slot] = old + sum;
        }
      }
      cluster_sync_all();  // shared memory stays readable until every rank is done
      if (late) prior_wait();
      return;
    }
    if (tid == 0 && r.first == 0) {
      const int c0 = (int)(r.unit / sh.per);
      const int parts = (int)((r.unit + r.tiles - 1) / sh.per) - c0 + 1;
      a.unit[r.s * p.h_kv + r.h] = make_int2(c0, parts);
      if (parts > 1) a.cut[blockIdx.x] = make_int2(r.s * p.h_kv + r.h, parts);
    }
    if (r.count == r.tiles) {
      for (int c = tid; c < g * (D / 4); c += kPdWarps * 32) {
        const int hh = c / (D / 4), d = c % (D / 4) * 4;
        float m, l, n;
        joined(hh, m, l, n);
        const float f = l == 0.f ? 0.f : kUndo * fast_exp2(n - m) / l;
        write_columns<D, PRIOR>(a, head0 + hh, d,
                         make_float4(joined_o(hh, d), joined_o(hh, d + 1), joined_o(hh, d + 2), joined_o(hh, d + 3)), f, m,
                         l, a.mass_out != nullptr);
      }
      continue;
    }
    // ---- a part of a unit: the join kernel adds it to the others.  CTA c's part goes
    // to slot 2c when the unit began before c, to 2c + 1 when it began in c
    const int64_t slot = 2 * (int64_t)blockIdx.x + (r.first == 0 ? 1 : 0);
    for (int c = tid; c < g * (D / 4); c += kPdWarps * 32) {
      const int hh = c / (D / 4), d = c % (D / 4) * 4;
      *reinterpret_cast<float4*>(a.part_o + (slot * g + hh) * D + d) =
          make_float4(joined_o(hh, d), joined_o(hh, d + 1), joined_o(hh, d + 2), joined_o(hh, d + 3));
      if (d == 0) {
        float m, l, n;
        joined(hh, m, l, n);
        a.part_ml[slot * g + hh] = make_float4(m, l, n, 0.f);
      }
    }
  }
  if (late) prior_wait();
}

// The parts j0, j0 + step, .. of one unit, head hh and four columns, N of them in flight.
struct Joined {
  float m, l, n;
  float4 o;
  __device__ __forceinline__ void rescale(float m1, float n1) {
    l *= m == -INFINITY ? 0.f : fast_exp2(m - m1);
    const float f = m == -INFINITY ? 0.f : fast_exp2(n - n1);
    o.x *= f, o.y *= f, o.z *= f, o.w *= f;
    m = m1;
    n = n1;
  }
  __device__ __forceinline__ void add(const float4& x, const float4& y) {  // (m, l, n) and O, under the references
    if (x.x == -INFINITY) return;  // (a place without a part)
    l += x.y * fast_exp2(x.x - m);
    const float f = fast_exp2(x.z - n);
    o.x += f * y.x;
    o.y += f * y.y;
    o.z += f * y.z;
    o.w += f * y.w;
  }
};
// CTA c's part of a unit lies in slot 2c when the unit began before c, in 2c + 1 when it began in c.
__device__ __forceinline__ int64_t part_slot(int c0, int j) { return 2 * (int64_t)(c0 + j) + (j == 0); }
template <int D, int N>
__device__ __forceinline__ Joined join_parts(const PdArgs& a, int c0, int parts, int hh, int d, int first, int step) {
  Joined r = {-INFINITY, 0.f, -INFINITY, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int j0 = first; j0 < parts; j0 += step * N) {
    float4 x[N], y[N];
#pragma unroll
    for (int f = 0; f < N; ++f) {
      const int64_t j = part_slot(c0, min(j0 + f * step, parts - 1)) * a.group + hh;
      x[f] = a.part_ml[j];
      y[f] = *reinterpret_cast<const float4*>(a.part_o + j * D + d);
    }
    float m1 = r.m, n1 = r.n;
#pragma unroll
    for (int f = 0; f < N; ++f) {
      if (j0 + f * step >= parts) x[f].x = x[f].z = -INFINITY;
      m1 = fmaxf(m1, x[f].x);
      n1 = fmaxf(n1, x[f].z);
    }
    r.rescale(m1, n1);
#pragma unroll
    for (int f = 0; f < N; ++f) r.add(x[f], y[f]);
  }
  return r;
}
template <int D, bool PRIOR>
__device__ __forceinline__ void write_joined(const PdArgs& a, const Joined& r, int unit, int hh, int d, float undo) {
  const float f = r.l == 0.f ? 0.f : undo * fast_exp2(r.n - r.m) / r.l;
  write_columns<D, PRIOR>(a, (int64_t)unit * a.group + hh, d, r.o, f, r.m, r.l);  // (s h_kv + h) g + hh = s h_q + h g + hh
}

// After the attention.  Joins the parts of the units that several CTAs shared.
// Of up to kPfMany parts: a unit to a CTA, a thread to all parts of its four
// columns, one round trip or two.  Of more (few units, then): a query head to a
// CTA, whose threads also share the parts (one sequence of 8,192 rows, 76 parts
// to a KV head: 11 us for the step, 18 with a thread to all parts; 48
// sequences of 2,000: 30 us, 35 with a head to a CTA).
// MASS: also turns the stored logits into weights and adds them to the rows'
// mass: a warp takes a run of tiles, a lane two rows of each; it forms its unit's
// log-sum-exps from the parts itself, which costs less than a third launch that
// waits for the join (16 x 16k: 4 % longer with that launch).
constexpr int kPfThreads = 256;
constexpr int kPfMany = 16;
constexpr int kPfHeads = 16;  // heads of units in many parts that one CTA looks at
template <int D, bool MASS, bool PRIOR>
__global__ void __launch_bounds__(kPfThreads, MASS ? 4 : 3) paged_finish_kernel(const __grid_constant__ PdArgs a,
                                                                                float undo) {
  constexpr int kCols = D / 4, kGroups = kPfThreads / kCols;
  __shared__ float4 part_o[kGroups][kCols];
  __shared__ float3 part_ml[kGroups];
  pdl_wait();
  pdl_trigger();
  const Pages& p = a.pages;
  const int tid = threadIdx.x, lane = tid & 31, g = a.group;
  // this warp's tiles of the mass: the first one's logits and place come to L1 while the join is dealt out
  int t0 = 0, t1 = 0;
  if (MASS) {
    const int total = *a.tiles, warps = gridDim.x * (kPfThreads / 32), each = (total + warps - 1) / warps;
    t0 = min((int)(blockIdx.x * (kPfThreads / 32) + (tid >> 5)) * each, total);
    t1 = min(t0 + each, total);
    const char* lg = reinterpret_cast<const char*>(a.logits + (int64_t)t0 * g * kPdRows);
    if (t0 < t1 && lane < 2 * g) asm volatile("prefetch.global.L1 [%0];\n" ::"l"(lg + 128 * lane));
    if (t0 < t1 && lane == 0) asm volatile("prefetch.global.L1 [%0];\n" ::"l"(a.info + t0));
  }
  // the unit that begins in CTA c = blockIdx.x, if it is cut; and heads of units in many parts, dealt out apart
  // (every warp finds out by itself: nothing to wait for but the loads)
  const int2 cut = blockIdx.x < (unsigned)a.ctas ? a.cut[blockIdx.x] : make_int2(-1, 0);
  const uint32_t my_head = blockIdx.x + (uint32_t)lane * gridDim.x;
  const bool heavy = lane < kPfHeads && my_head < (uint32_t)(a.ctas * g) && a.cut[my_head / g].y > kPfMany;
  uint32_t heads = __ballot_sync(0xffffffffu, heavy);
  if (cut.y > 1 && cut.y <= kPfMany) {
    for (int c = tid; c < g * kCols; c += kPfThreads) {
      const int hh = c / kCols, d = c % kCols * 4;
      write_joined<D, PRIOR>(a, join_parts<D, MASS ? 4 : 8>(a, blockIdx.x, cut.y, hh, d, 0, 1), cut.x, hh, d, undo);
    }
  }
  const int col = tid % kCols, grp = tid / kCols;
  for (; heads; heads &= heads - 1) {
    const uint32_t i = blockIdx.x + (uint32_t)(__ffs(heads) - 1) * gridDim.x;
    const int c0 = (int)(i / g), hh = (int)(i % g);
    const int2 t = a.cut[c0];
    const Joined r = join_parts<D, 4>(a, c0, t.y, hh, 4 * col, grp, kGroups);
    __syncthreads();  // the last head's parts are read
    part_o[grp][col] = r.o;
    if (col == 0) part_ml[grp] = make_float3(r.m, r.l, r.n);
    __syncthreads();
    if (grp == 0) {
      Joined all = {-INFINITY, 0.f, -INFINITY, make_float4(0.f, 0.f, 0.f, 0.f)};
#pragma unroll
      for (int q = 0; q < kGroups; ++q) {
        all.m = fmaxf(all.m, part_ml[q].x);
        all.n = fmaxf(all.n, part_ml[q].z);
      }
#pragma unroll
      for (int q = 0; q < kGroups; ++q)
        all.add(make_float4(part_ml[q].x, part_ml[q].y, part_ml[q].z, 0.f), part_o[q][col]);
      write_joined<D, PRIOR>(a, all, t.x, hh, 4 * col, undo);
    }
  }
  if (!MASS) return;
  int now = -1;
  float lse = INFINITY;  // lane hh: of query head hh of unit `now`
  for (int t = t0; t < t1; ++t) {
    // (the logits' place goes by the tile alone: they load while the rest is looked up)
    const float* lg = a.logits + (int64_t)t * g * kPdRows + 2 * lane;
    float2 v[8];
#pragma unroll
    for (int hh = 0; hh < 8; ++hh)
      v[hh] = hh < g ? *reinterpret_cast<const float2*>(lg + hh * kPdRows) : make_float2(-INFINITY, -INFINITY);
    const int4 x = *reinterpret_cast<const int4*>(&a.info[t]);
    const int page = a.info[t].page[lane >> 3];
    const int u = x.x * p.h_kv + x.y, row = x.z * kPdRows + 2 * lane, len = p.lens[x.x];
    const bool in = page >= 0 && row < len;
    const int64_t slot = in ? page_slot(p, page, x.y, row % p.page_rows) : 0;
    float2 old = in ? *reinterpret_cast<const float2*>(p.mass + slot) : make_float2(0.f, 0.f);
    if (u != now) {
      now = u;
      const int2 un = a.unit[u];
      if (un.y < 2) {
        if (lane < g) lse = a.lse2[(int64_t)u * g + lane];
      } else {
        // the heads side by side, 32 / width lanes to each, four parts of a lane in flight
        const int width = g <= 8 ? 8 : 16, subs = 32 / width, hh = min(lane & (width - 1), g - 1);
        float m = -INFINITY, l = 0.f;
        for (int j0 = lane / width; j0 < un.y; j0 += 4 * subs) {
          float2 ml[4];
#pragma unroll
          for (int f = 0; f < 4; ++f)
            ml[f] = *reinterpret_cast<const float2*>(a.part_ml + part_slot(un.x, min(j0 + f * subs, un.y - 1)) * g + hh);
#pragma unroll
          for (int f = 0; f < 4; ++f) {
            if (j0 + f * subs >= un.y) continue;
            const float m1 = fmaxf(m, ml[f].x);
            l = l * fast_exp2(m - m1) + ml[f].y * fast_exp2(ml[f].x - m1);
            m = m1;
          }
        }
        float m1 = m;
        for (int off = width; off < 32; off <<= 1) m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, off));
        l = m == -INFINITY ? 0.f : l * fast_exp2(m - m1);
        for (int off = width; off < 32; off <<= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
        lse = mass_lse2<PRIOR>(a, (int64_t)u * g + hh, m1, l);
      }
    }
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int hh = 0; hh < 8; ++hh) {
      const float z = __shfl_sync(0xffffffffu, lse, hh);
      if (hh < g) {
        sum.x += fast_exp2(v[hh].x - z);
        sum.y += fast_exp2(v[hh].y - z);
      }
    }
    for (int hh = 8; hh < g; ++hh) {
      const float z = __shfl_sync(0xffffffffu, lse, hh);
      const float2 y = *reinterpret_cast<const float2*>(lg + hh * kPdRows);
      sum.x += fast_exp2(y.x - z);
      sum.y += fast_exp2(y.y - z);
    }
    if (!in) continue;
    if (row + 1 < len)
      *reinterpret_cast<float2*>(a.mass_out + slot) = make_float2(old.x + sum.x, old.y + sum.y);
    else
      a.mass_out[slot] = old.x + sum.x;
  }
}

// ------------------------------------------------------------------ host

struct PdPlan {
  Pages pages;
  bool q8;
  int d, g, grid, sms, ranks;  // ranks: CTAs to a unit of short sequences (0: the list)
  int64_t tiles;  // bound of the tile list
  size_t unit_off, lse_off, ml_off, o_off, info_off, lg_off, total;
};

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

int pd_plan(const aircache_paged_decode_problem* p, PdPlan& pl) {
  if (!p) return AIRCACHE_ERR_INVALID_ARG;
  const int rc = check_pages(p->pages, pl.pages);
  if (rc != AIRCACHE_OK) return rc;
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  if (p->h_q <= 0 || p->h_q % p->pages->h_kv != 0 || p->reserved0 != 0 || p->dtype != AIRCACHE_BF16 ||
      !(p->scale > 0.f) || !std::isfinite(1.4427f * p->scale) || p->total_rows < 1 || p->total_rows > 0x7fff0000LL || !p->q ||
      !p->out || !al16(p->q) || !al16(p->out) || p->q_stride_seq < 0 || p->q_stride_head < 0 ||
      p->q_stride_seq % 8 != 0 || p->q_stride_head % 8 != 0 || (p->mass_out && !p->pages->mass) ||
      (p->mass_out != p->pages->mass &&
       arrays_meet(p->mass_out, slot_bytes(pl.pages), p->pages->mass, slot_bytes(pl.pages))) ||
      (reinterpret_cast<uintptr_t>(p->lse) & 3) != 0 || !al16(p->mass_out))
    return AIRCACHE_ERR_INVALID_ARG;
  pl.g = p->h_q / p->pages->h_kv;
  if (pl.g > kPdGroup) return AIRCACHE_ERR_UNSUPPORTED;
  pl.q8 = p->pages->kv_dtype == AIRCACHE_INT8;
  pl.d = p->pages->head_dim;
  pl.sms = device_sms();
  const int64_t units = (int64_t)p->pages->num_seqs * p->pages->h_kv;
  pl.tiles = (p->total_rows / kPdRows + p->pages->num_seqs) * p->pages->h_kv;
  if (pl.tiles + (int64_t)kPdEnd * units > 0x7fffffffLL) return AIRCACHE_ERR_UNSUPPORTED;
  pl.grid = (int)std::max<int64_t>(1, std::min<int64_t>((int64_t)ctas_per_sm(pl.q8, pl.g) * pl.sms, pl.tiles));
  // Short sequences: the number of CTAs to a unit by the time of a call, in seventieths of a tile's
  // (0.57 us; int8 rows and mass cost twice that): its CTAs' tiles, what clusters of 4 and 8 add, and one for each
  // CTA.  Up to ten tiles' worth that beats the list and its second kernel (701 rows of 4 KV heads: 7.0 us
  // with 4 CTAs to each, 7.7 with 8, 8.2 with 2, 11.6 with 1, 8.9 by the list; 24 x 600: 11.1 and 13.2; but 4,000
  // rows: 11.3 and 9.8)
  pl.ranks = 0;
  const int64_t longest = (std::min<int64_t>(pl.pages.max_rows, p->total_rows) + kPdRows - 1) / kPdRows;  // tiles
  int64_t least = 701;
  for (int r = 1; r <= kPdRanks && units * r <= (int64_t)ctas_per_sm(pl.q8, pl.g) * pl.sms; r *= 2) {
    const int64_t cost = (pl.q8 || p->mass_out ? 140 : 70) * ((longest + r - 1) / r) + (r == 8 ? 224 : r == 4 ? 56 : 0) + units * r;
    if (cost < least) least = cost, pl.ranks = r;
  }
  pl.unit_off = kPdHeader + up256(sizeof(int2) * (size_t)pl.grid);
  pl.lse_off = pl.unit_off + up256(sizeof(int2) * (size_t)units);
  pl.ml_off = pl.lse_off + up256(sizeof(float) * (size_t)p->pages->num_seqs * p->h_q);
  pl.o_off = pl.ml_off + up256(sizeof(float4) * 2 * (size_t)pl.grid * pl.g);
  pl.info_off = pl.o_off + up256(sizeof(float) * 2 * (size_t)pl.grid * pl.g * pl.d);
  pl.lg_off = pl.info_off + (p->mass_out ? up256(sizeof(TileInfo) * (size_t)pl.tiles) : 0);
  pl.total = pl.lg_off + (p->mass_out ? up256(sizeof(float) * (size_t)pl.tiles * pl.g * kPdRows) : 0);
  return AIRCACHE_OK;
}

// One box: 16 rows of one page and KV head, every 128-byte column slab of them.
bool encode_pages(CUtensorMap* m, const void* base, const PdPlan& pl) {
  auto enc = tma_encoder();
  if (!enc) return false;
  const Pages& p = pl.pages;
  // L2 fetches what one row of one KV head covers and no more: with 256 bytes promoted, 64-wide bf16
  // heads (128 bytes) brought half of their neighbours along (669 MB for 452)
  const int row = pl.d * (pl.q8 ? 1 : 2);
  const CUtensorMapL2promotion promote = row == 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                         : row == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                      : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  if (pl.q8) {
    cuuint64_t dims[4] = {(cuuint64_t)pl.d, (cuuint64_t)p.page_rows, (cuuint64_t)p.h_kv, (cuuint64_t)p.num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)p.stride_row, (cuuint64_t)p.stride_head, (cuuint64_t)p.stride_page};
    cuuint32_t box[4] = {(cuuint32_t)pl.d, 16, 1, 1}, es[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, pl.d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  cuuint64_t dims[5] = {64, (cuuint64_t)p.page_rows, (cuuint64_t)pl.d / 64, (cuuint64_t)p.h_kv,
                        (cuuint64_t)p.num_pages};
  cuuint64_t strides[4] = {(cuuint64_t)p.stride_row * 2, 128, (cuuint64_t)p.stride_head * 2,
                           (cuuint64_t)p.stride_page * 2};
  cuuint32_t box[5] = {64, 16, (cuuint32_t)pl.d / 64, 1, 1}, es[5] = {1, 1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, promote,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool Q8, int HB, bool PRIOR>
int launch_pd(const PdPlan& pl, const PdArgs& a, cudaStream_t s) {
  CUtensorMap km, vm;
  if (!encode_pages(&km, pl.pages.k, pl) || !encode_pages(&vm, pl.pages.v, pl)) return AIRCACHE_ERR_UNSUPPORTED;
  constexpr int smem = PdCfg<D, Q8, HB>::kSmem;
  const auto kernel = pl.ranks > 0 ? &paged_decode_kernel<D, Q8, HB, true, PRIOR> : &paged_decode_kernel<D, Q8, HB, false, PRIOR>;
  if (allow_smem(reinterpret_cast<const void*>(kernel), smem) != cudaSuccess) return AIRCACHE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.ranks > 0 ? pl.ranks * pl.pages.num_seqs * pl.pages.h_kv : pl.grid);
  cfg.blockDim = dim3(kPdThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = std::max(pl.ranks, 1);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pl.ranks > 0 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kernel, km, vm, a) != cudaSuccess) return AIRCACHE_ERR_CUDA;
  if (pl.ranks > 0) return AIRCACHE_OK;
  cfg.numAttrs = 1;
  // As many CTAs as the attention has (a cut unit begins in one of them; so each looks at one unit and
  // g heads), or with the mass as many as the SMs hold and its tiles need
  static_assert(kPfHeads >= kPdGroup, "g heads for each CTA of the attention");
  cfg.gridDim = dim3((unsigned)std::max<int64_t>(
      pl.grid, a.mass_out ? std::min<int64_t>((pl.tiles + kPfThreads / 32 - 1) / (kPfThreads / 32), 4LL * pl.sms) : 0));
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = 0;
  const float undo = Q8 ? 1.f / kP16 : 1.f;
  if (cudaLaunchKernelEx(&cfg, a.mass_out ? paged_finish_kernel<D, true, PRIOR> : paged_finish_kernel<D, false, PRIOR>, a, undo) !=
      cudaSuccess)
    return AIRCACHE_ERR_CUDA;
  return AIRCACHE_OK;
}

template <int D, bool Q8>
int launch_pd(const PdPlan& pl, const PdArgs& a, cudaStream_t s) {
  if (a.prior.out) return pl.g <= 8 ? launch_pd<D, Q8, 1, true>(pl, a, s) : launch_pd<D, Q8, 2, true>(pl, a, s);
  return pl.g <= 8 ? launch_pd<D, Q8, 1, false>(pl, a, s) : launch_pd<D, Q8, 2, false>(pl, a, s);
}

}  // namespace

int paged_decode_run(const aircache_paged_decode_problem* p, const DecodePrior& prior, void* ws, size_t ws_bytes,
                     void* stream) {
  PdPlan pl;
  const int rc = pd_plan(p, pl);
  if (rc != AIRCACHE_OK) return rc;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) return AIRCACHE_ERR_INVALID_ARG;
  if (ws_bytes < pl.total) return AIRCACHE_ERR_WORKSPACE;
  if (p->pages->num_seqs == 0) return AIRCACHE_OK;
  uint8_t* w = static_cast<uint8_t*>(ws);
  PdArgs a;
  a.pages = pl.pages;
  a.q = static_cast<const __nv_bfloat16*>(p->q);
  a.q_stride_seq = p->q_stride_seq;
  a.q_stride_head = p->q_stride_head;
  a.out = static_cast<__nv_bfloat16*>(p->out);
  a.lse = p->lse;
  a.mass_out = p->mass_out;
  a.error = reinterpret_cast<int32_t*>(w);
  a.tiles = reinterpret_cast<int32_t*>(w + 64);
  a.cut = reinterpret_cast<int2*>(w + kPdHeader);
  a.unit = reinterpret_cast<int2*>(w + pl.unit_off);
  a.lse2 = reinterpret_cast<float*>(w + pl.lse_off);
  a.part_ml = reinterpret_cast<float4*>(w + pl.ml_off);
  a.part_o = reinterpret_cast<float*>(w + pl.o_off);
  a.info = reinterpret_cast<TileInfo*>(w + pl.info_off);
  a.logits = reinterpret_cast<float*>(w + pl.lg_off);
  a.prior = prior;
  a.total_rows = p->total_rows;
  a.h_q = p->h_q;
  a.group = pl.g;
  a.ctas = pl.grid;
  a.ranks = pl.ranks;
  a.scale_log2 = (float)(1.4426950408889634 * (double)p->scale);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (pl.q8) return pl.d == 128 ? launch_pd<128, true>(pl, a, s) : launch_pd<64, true>(pl, a, s);
  return pl.d == 128 ? launch_pd<128, false>(pl, a, s) : launch_pd<64, false>(pl, a, s);
}

int paged_decode_size(const aircache_paged_decode_problem* p, size_t& bytes) {
  PdPlan pl;
  const int rc = pd_plan(p, pl);
  bytes = pl.total;
  return rc;
}

}  // namespace aircache

using namespace aircache;

extern "C" {

size_t aircache_paged_decode_workspace_size(const aircache_paged_decode_problem* p) {
  PdPlan pl;
  return pd_plan(p, pl) == AIRCACHE_OK ? pl.total : 0;
}

int aircache_paged_decode(const aircache_paged_decode_problem* p, void* ws, size_t ws_bytes, void* stream) {
  return paged_decode_run(p, DecodePrior{nullptr, nullptr, nullptr, nullptr}, ws, ws_bytes, stream);
}

}  // extern "C"
