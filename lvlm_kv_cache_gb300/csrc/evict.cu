// Eviction from the paged cache by accumulated attention weight (aircache_evict).
//
// Of a sequence's n rows every KV head keeps the `keep` best (protected rows
// first, then by mass, ties to the lower row).  A row's rank is all that
// matters and attention does not mind the rows' order, so only kept rows
// behind `keep` move: the j-th of them into the j-th vacated row below
// `keep`.  That reads and writes each moved row once, and no destination is
// another move's source, so the moves need no order.
//
// select: one thread-block cluster (or, for short sequences, one CTA) per
// (sequence, KV head).  Each CTA holds the keys of a slice of the rows in
// shared memory (the mass as an order-preserving integer).  The threshold is
// found by histograms of 256 equal parts of the range that is left, from the
// keys' least to their largest, added up through distributed shared memory, and so on
// within the threshold's part: spread over their bins however the masses are (digits
// of fixed places would put most rows into a few bins and serialise their
// atomics).  Its warps then walk over consecutive rows, four to a lane, and list vacated rows
// and movers in order.  Bound by the
// chain of barriers and scans: 8 bytes a row are read.
// move: CTAs over all SMs copy the listed rows, 32 moves to a warp at a time.
// Bound by HBM.  Few rows are moved by the CTAs that selected them, in one kernel.
#include <algorithm>
#include <climits>

#include "pages.cuh"

namespace aircache {
namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvMaxCluster = 8;
constexpr int kMvThreads = 256, kMvCtas = 4;  // of the moves: threads of a CTA, CTAs to an SM
constexpr int kEvSlice = AIRCACHE_MAX_EVICT_ROWS / kEvMaxCluster;  // keys of one CTA, at most
// Rows of one CTA, at most, for it to move them too, in one kernel; twice as many where it has a (sequence, KV
// head) for itself (with the second kernel one of 1,088 takes 15 % longer, 8 x 4,000, in clusters of 2, 15 %, 48 x
// 4,000 int8 15 %; but 16 x 8,000, in clusters of 2, 7 % less, and 48 of up to 9,000 int8 4 % less)
constexpr int kEvShort = 2048;
constexpr int kEvHeader = 256;                                     // workspace: error word
constexpr uint32_t kProtected = 0xffffffffu;

struct EvArgs {
  Pages pages;
  const int32_t* keep;
  const int32_t* seen;
  int32_t* lens_out;
  float* mass_out;
  int32_t* order_out;
  int32_t* error;
  int32_t* moves;  // [units]: moves of each (sequence, KV head)
  int32_t* lists;  // [units][2][half]: vacated rows, movers
  int half;        // half of max_rows
  int max_rows, sink, recent;
};

// What a CTA adds to the ranks of the rows behind it.
struct Before {
  uint32_t ties, ties_low;  // rows at the threshold; those of them below keep
  uint32_t less, more;      // rows under the threshold below keep; rows over it at keep and behind
};

constexpr int kBinBits = 8, kBins = 1 << kBinBits;
constexpr int kNear = 256;  // keys that a warp can set aside

struct EvShared {
  uint32_t hist[4][kBins];
  Before warp[kEvWarps];
  Before sum;
  uint32_t scan[kEvWarps], scan2[kEvWarps], scan3[kEvWarps];
  uint32_t least, most, safe, bad;  // this CTA's least and largest key, protected rows, bad pages
  uint32_t bin, above, in_bin;
  uint32_t near[kEvWarps][kNear];  // the keys in the part of the range that the first histogram left
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Larger for the row to keep: fp32 order as integers, -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// RB: 16-byte pieces of a row of one KV head.  What a warp waits for is hidden
// by other warps, so few registers count for more than many loads of one warp
// (16 x 16k to half: 61 us with four row loads in flight and 32 warps to an SM,
// 73 with eight and 24), and nothing is stored before every load of the 32 moves' scales, mass
// and order and the first rows' has been issued.
template <int RB>
__device__ __forceinline__ void move_rows(const EvArgs& a, int s, int h, int moves, int first, int warps) {
  const Pages& p = a.pages;
  const int lane = threadIdx.x & 31;
  const int32_t* table = p.table + (int64_t)s * p.table_stride;
  const int32_t* list = a.lists + ((int64_t)s * p.h_kv + h) * 2 * a.half;
  constexpr int kAtOnce = 32 / (2 * RB);  // moves of one warp instruction
  const int piece = lane % RB, sub = lane / (2 * RB);
  uint8_t* const kv = ((lane / RB) & 1 ? p.v : p.k) + 16 * piece;
  const int size = p.k_scale ? 1 : 2;
  for (int m0 = 32 * first; m0 < moves; m0 += 32 * warps) {
    int64_t src = 0, dst = 0, ds = 0;
    const int cnt = min(32, moves - m0);
    float mass = 0.f, ks = 0.f, vs = 0.f;
    int32_t order = 0;
    if (lane < cnt) {
      const int to = list[m0 + lane], from = list[a.half + m0 + lane];
      int tr, fr;
      const int tx = page_of(p, to, tr), fx = page_of(p, from, fr);
      const int tp = table[tx], fp = table[fx];
      ds = page_slot(p, tp, h, tr);
      const int64_t ss = page_slot(p, fp, h, fr);
      dst = page_elem(p, tp, h, tr) * size;
      src = page_elem(p, fp, h, fr) * size;
      mass = p.mass[ss];
      if (a.order_out) order = p.order[ss];
      if (p.k_scale) ks = p.k_scale[ss], vs = p.v_scale[ss];
    }
    constexpr int kFlight = 4;
    for (int j0 = 0; j0 < cnt; j0 += kAtOnce * kFlight) {
      uint4 x[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int j = j0 + f * kAtOnce + sub;
        const int64_t from = __shfl_sync(0xffffffffu, src, j & 31);
        if (j < cnt) x[f] = *reinterpret_cast<const uint4*>(kv + from);
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const int j = j0 + f * kAtOnce + sub;
        const int64_t to = __shfl_sync(0xffffffffu, dst, j & 31);
        if (j < cnt) *reinterpret_cast<uint4*>(kv + to) = x[f];
      }
    }
    if (lane < cnt) {
      a.mass_out[ds] = mass;
      if (a.order_out) a.order_out[ds] = order;
      if (p.k_scale) p.k_scale[ds] = ks, p.v_scale[ds] = vs;
    }
  }
}

// R CTAs (a cluster) per (sequence, KV head).  What they tell each other is read
// by one lane per CTA at once, or by loads that do not wait for one another: a
// load from another CTA's shared memory takes several hundred cycles.  F groups of four rows
// load at once in a thread: eight with one CTA to an SM, four (and half the registers) with two
// (2 x 128k: 46 us, 10 % longer with four; ragged, 192 CTAs: 39 us, 6 % longer with eight).
// RB: the CTA also moves the rows (0: another kernel does).
template <int R, int F, int RB>
__global__ void __launch_bounds__(kEvThreads, F == 4 ? 2 : 1) evict_select_kernel(const __grid_constant__ EvArgs a) {
  extern __shared__ __align__(16) uint32_t ev_keys[];  // (read four at a time)
  __shared__ EvShared sh;
  const Pages& p = a.pages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr bool CL = R > 1;
  const int rank = CL ? blockIdx.x : 0;  // the cluster spans x
  const int h = blockIdx.y, s = blockIdx.z;
  auto sync_all = [] {
    if (CL)
      cluster_sync_all();
    else
      __syncthreads();
  };
  auto peer = [&](const uint32_t* x, int r) { return CL ? ld_cluster_u32(cluster_map(smem_u32(x), r)) : *x; };
  for (int i = tid; i < 4 * kBins; i += kEvThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) sh.bad = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  // the table's row comes to L1 while the length is waited for
  const int32_t* table = p.table + (int64_t)s * p.table_stride;
  for (int64_t i = 32LL * tid; i * p.page_rows < min(a.max_rows, p.max_rows); i += 32 * kEvThreads)
    asm volatile("prefetch.global.L1 [%0];\n" ::"l"(table + i));
  const int len = p.lens[s], keep = a.keep[s];
  const int32_t seen = a.recent ? a.seen[s] : 0;
  const bool sane = len >= 0 && len <= a.max_rows && len <= p.max_rows && keep >= 0 &&
                    (len <= keep || (int64_t)keep >= (int64_t)a.sink + a.recent);
  if (!sane && tid == 0) set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
  const int n = sane ? len : 0;
  const bool cut = sane && n > keep;
  const int per = ((n + R - 1) / R + 15) & ~15;
  const int lo = min(rank * per, n), mine = min(per, n - lo);  // this CTA's rows
  // protected are orders under `first` and over `last`: of all where seen - recent is below int32, and without
  // recent rows no order is over `last`
  const bool all_recent = a.recent && seen <= INT_MIN + a.recent;
  const int32_t first = all_recent ? INT_MAX : a.sink;
  const int32_t last = !a.recent ? INT_MAX : all_recent ? INT_MAX - 1 : seen - a.recent - 1;
  const bool aged = a.sink | a.recent;

  // Where mass and order go to other arrays, every row below the new length is
  // copied on the way; the moves overwrite the vacated ones
  const bool copy_mass = a.mass_out != p.mass, copy_order = a.order_out && a.order_out != p.order;
  const int new_len = cut ? keep : n;

  // ---- keys of the slice, their range and the protected rows.  Four rows a thread
  // (a page holds a multiple of 16)
  constexpr int kFlight = F;
  uint32_t least = kProtected, most = 0, safe = 0;
  for (int i0 = 4 * tid; i0 < mine; i0 += 4 * kFlight * kEvThreads) {
    int page[kFlight], at[kFlight];
    float4 m[kFlight];
    int4 o[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = i0 + 4 * f * kEvThreads, x = page_of(p, lo + i, at[f]);
      page[f] = i < mine ? table[x] : 0;
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = i0 + 4 * f * kEvThreads;
      m[f] = make_float4(0.f, 0.f, 0.f, 0.f);
      o[f] = make_int4(0, 0, 0, 0);
      if (i < mine) {
        if (page_ok(p, page[f])) {
          const int64_t slot = page_slot(p, page[f], h, at[f]);
          m[f] = *reinterpret_cast<const float4*>(p.mass + slot);
          if (aged || copy_order) o[f] = *reinterpret_cast<const int4*>(p.order + slot);
        } else {
          sh.bad = 1;
        }
      }
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = i0 + 4 * f * kEvThreads;
      if (i >= mine) break;
      const float mm[4] = {m[f].x, m[f].y, m[f].z, m[f].w};
      const int oo[4] = {o[f].x, o[f].y, o[f].z, o[f].w};
      const int keep_out = new_len - lo - i;  // of these four rows, how many lie below the new length
      if ((copy_mass || copy_order) && keep_out > 0 && page_ok(p, page[f])) {
        const int64_t slot = page_slot(p, page[f], h, at[f]);
        if (keep_out >= 4) {
          if (copy_mass) *reinterpret_cast<float4*>(a.mass_out + slot) = m[f];
          if (copy_order) *reinterpret_cast<int4*>(a.order_out + slot) = o[f];
        } else {
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            if (copy_mass && j < keep_out) a.mass_out[slot + j] = mm[j];
            if (copy_order && j < keep_out) a.order_out[slot + j] = oo[j];
          }
        }
      }
      uint32_t key[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = i + j < mine;
        key[j] = !in || (aged && (oo[j] < first || oo[j] > last)) ? kProtected : mass_key(mm[j]);
        least = min(least, key[j]);
        most = max(most, key[j] + 1);  // (a protected row wraps to 0)
        safe += in && key[j] == kProtected;
      }
      *reinterpret_cast<uint4*>(ev_keys + i) = make_uint4(key[0], key[1], key[2], key[3]);
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  safe = __reduce_add_sync(0xffffffffu, safe);
  if (lane == 0) sh.scan[warp] = least, sh.scan2[warp] = most, sh.scan3[warp] = safe;
  __syncthreads();
  if (warp == 0) {
    const bool in = lane < kEvWarps;
    least = __reduce_min_sync(0xffffffffu, in ? sh.scan[lane] : kProtected);
    most = __reduce_max_sync(0xffffffffu, in ? sh.scan2[lane] : 0u);
    safe = __reduce_add_sync(0xffffffffu, in ? sh.scan3[lane] : 0u);
    if (lane == 0) sh.least = least, sh.most = most, sh.safe = safe;
  }
  sync_all();
  const int from = min(lane, R - 1);
  least = __reduce_min_sync(0xffffffffu, peer(&sh.least, from));
  most = __reduce_max_sync(0xffffffffu, peer(&sh.most, from));
  safe = peer(&sh.safe, from);
  safe = __reduce_add_sync(0xffffffffu, lane < R ? safe : 0u);
  const bool bad = __reduce_max_sync(0xffffffffu, peer(&sh.bad, from)) != 0;
  if (bad && tid == 0) set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
  const bool go = cut && !bad;

  // ---- the threshold, and how many of the rows at it stay (`need`).  Protected
  // rows stay, unless there are more of them than places
  uint32_t prefix = kProtected, need = keep, near = 0;
  if (go && safe < (uint32_t)keep) {
    need = keep - safe;
    prefix = least;  // where the range that is left begins
    int shift = 32 - __clz(most - 1 - least);  // its keys: prefix .. prefix + 2^shift - 1
    for (int d = 0; shift > 0; ++d) {
      const uint32_t top = shift;
      shift = max(0, shift - kBinBits);
      // (no protected row, nor what fills the last group of four, lies in it)
      const uint32_t left = min(top > 31 ? 0xffffffffu : (1u << top) - 1, kProtected - 1 - prefix);
      // with the second histogram each warp sets the keys that it counts aside, and looks at these
      // alone in the later ones, if they have room (they have not with many equal keys)
      if (d > 1 && near <= kNear) {
        for (uint32_t i = lane; i < near; i += 32) {
          const uint32_t off = sh.near[warp][i] - prefix;
          if (off <= left) atomicAdd(&sh.hist[d][off >> shift], 1u);
        }
      } else {
        for (int i0 = 0; i0 < mine; i0 += 4 * kEvThreads) {
          const int i = i0 + 4 * tid;
          const uint4 k4 = i < mine ? *reinterpret_cast<const uint4*>(ev_keys + i)
                                    : make_uint4(kProtected, kProtected, kProtected, kProtected);
          const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
          bool in[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t off = key[j] - prefix;  // (a key below the range wraps past it)
            in[j] = off <= left;
            if (in[j]) atomicAdd(&sh.hist[d][off >> shift], 1u);
          }
          if (d == 1 && __any_sync(0xffffffffu, in[0] || in[1] || in[2] || in[3])) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t hits = __ballot_sync(0xffffffffu, in[j]);
              const uint32_t at = near + __popc(hits & ((1u << lane) - 1));
              if (in[j] && at < kNear) sh.near[warp][at] = key[j];
              near += __popc(hits);
            }
            __syncwarp();
          }
        }
      }
      sync_all();
      // from the largest bin down, a bin to each of the first threads
      uint32_t c = 0;
      if (tid < kBins) {
        uint32_t v[R];
#pragma unroll
        for (int x = 0; x < R; ++x) v[x] = peer(&sh.hist[d][kBins - 1 - tid], x);
#pragma unroll
        for (int x = 0; x < R; ++x) c += v[x];
      }
      uint32_t incl = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += t;
      }
      if (lane == 31) sh.scan[warp] = incl;
      __syncthreads();
      uint32_t above = incl - c;
#pragma unroll
      for (int w = 0; w < kBins / 32; ++w)
        if (w < warp) above += sh.scan[w];
      if (tid < kBins && above < need && above + c >= need) {
        sh.bin = kBins - 1 - tid;
        sh.above = above;
        sh.in_bin = c;
      }
      __syncthreads();
      prefix += sh.bin << shift;
      need -= sh.above;
      // all of the part's rows stay: it need not be divided further, and no row is at the threshold
      if (sh.in_bin == need) {
        prefix -= 1;
        need = 0;
        break;
      }
    }
  }

  // ---- ranks.  Of the rows at the threshold the `need` lowest stay, so with T
  // ties, L lesser rows (below keep) and M greater rows (at keep and behind) before a row, L + T -
  // min(T, need) rows were vacated and M + min(T, need) - min(ties below keep, need) moved.
  // A warp walks over consecutive rows, a lane over four of them at a time
  const int span = ((mine + kEvWarps - 1) / kEvWarps + 127) & ~127;
  const int w0 = min(warp * span, mine), w1 = min(w0 + span, mine);
  if (go) {
    Before b = {0, 0, 0, 0};
    for (int i0 = w0; i0 < w1; i0 += 128) {
      const int i = i0 + 4 * lane;
      if (i0 + 128 <= w1 && (lo + i0 + 128 <= keep || lo + i0 >= keep)) {  // all below keep, or none
        const uint4 k4 = *reinterpret_cast<const uint4*>(ev_keys + i);
        const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
        uint32_t tie = 0, over = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          tie += key[j] == prefix;
          over += key[j] > prefix;
        }
        b.ties += tie;
        if (lo + i0 >= keep)
          b.more += over;
        else
          b.ties_low += tie, b.less += 4 - tie - over;
      } else if (i < w1) {
        const uint4 k4 = *reinterpret_cast<const uint4*>(ev_keys + i);
        const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool in = i + j < w1, low = lo + i + j < keep, tie = in && key[j] == prefix;
          b.ties += tie;
          b.ties_low += tie && low;
          b.less += in && low && key[j] < prefix;
          b.more += in && !low && key[j] > prefix;
        }
      }
    }
    b.ties = __reduce_add_sync(0xffffffffu, b.ties);
    b.ties_low = __reduce_add_sync(0xffffffffu, b.ties_low);
    b.less = __reduce_add_sync(0xffffffffu, b.less);
    b.more = __reduce_add_sync(0xffffffffu, b.more);
    if (lane == 0) sh.warp[warp] = b;
    __syncthreads();
    if (tid == 0) {
      Before t = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kEvWarps; ++w) {
        t.ties += sh.warp[w].ties;
        t.ties_low += sh.warp[w].ties_low;
        t.less += sh.warp[w].less;
        t.more += sh.warp[w].more;
      }
      sh.sum = t;
    }
    sync_all();
    Before at = {0, 0, 0, 0};  // before this warp's rows
    const uint32_t t_ = peer(&sh.sum.ties, from), l_ = peer(&sh.sum.less, from), m_ = peer(&sh.sum.more, from),
                   tl_ = peer(&sh.sum.ties_low, from);
    at.ties = __reduce_add_sync(0xffffffffu, lane < rank ? t_ : 0u);
    at.less = __reduce_add_sync(0xffffffffu, lane < rank ? l_ : 0u);
    at.more = __reduce_add_sync(0xffffffffu, lane < rank ? m_ : 0u);
    const uint32_t ties_low = __reduce_add_sync(0xffffffffu, lane < R ? tl_ : 0u);
    const uint32_t less = __reduce_add_sync(0xffffffffu, lane < R ? l_ : 0u);
#pragma unroll
    for (int w = 0; w < kEvWarps; ++w)
      if (w < warp) at.ties += sh.warp[w].ties, at.less += sh.warp[w].less, at.more += sh.warp[w].more;
    const uint32_t stay_low = min(ties_low, need);
    int32_t* list = a.lists + ((int64_t)s * p.h_kv + h) * 2 * a.half;
    // the warp's rows are compacted over its own keys, vacated rows (below keep,
    // so they come first) before movers, and written out in whole lines
    const uint32_t hole0 = at.less + at.ties - min(at.ties, need);
    const uint32_t mover0 = at.more + min(at.ties + b.ties_low, need);
    const uint32_t holes = b.less + b.ties_low - (min(at.ties + b.ties_low, need) - min(at.ties, need));
    uint32_t* const packed = ev_keys + w0;
    for (int i0 = w0; i0 < w1 && keep > 0; i0 += 128) {
      const int i = i0 + 4 * lane;
      const uint4 k4 = i < w1 ? *reinterpret_cast<const uint4*>(ev_keys + i) : make_uint4(0, 0, 0, 0);
      const uint32_t key[4] = {k4.x, k4.y, k4.z, k4.w};
      const bool tied = key[0] == prefix || key[1] == prefix || key[2] == prefix || key[3] == prefix;
      if (i0 + 128 <= w1 && (lo + i0 + 128 <= keep || lo + i0 >= keep) && !__any_sync(0xffffffffu, tied)) {
        // 128 rows on one side of keep and off the threshold: only lesser or only greater rows
        // count.  (Taken 32 rows at a time here; the vote above is past every lane's reads.)
        const bool high = lo + i0 >= keep;
        const uint32_t stay = min(at.ties, need);
        uint32_t to = high ? holes + at.more + stay - mover0 : at.less + at.ties - stay - hole0;
        uint32_t row_key[4], all = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) row_key[j] = ev_keys[i0 + 32 * j + lane];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bool is = (row_key[j] > prefix) == high;
          const uint32_t hits = __ballot_sync(0xffffffffu, is);
          if (is) packed[to + all + __popc(hits & ((1u << lane) - 1))] = lo + i0 + 32 * j + lane;
          all += __popc(hits);
        }
        if (high)
          at.more += all;
        else
          at.less += all;
        continue;
      }
      uint32_t c = 0;  // ties, lesser, greater rows of this lane: ten bits each
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = i + j < w1, low = lo + i + j < keep;
        c += (in && key[j] == prefix) + ((uint32_t)(in && low && key[j] < prefix) << 10) +
             ((uint32_t)(in && !low && key[j] > prefix) << 20);
      }
      uint32_t incl = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += t;
      }
      const uint32_t all = __shfl_sync(0xffffffffu, incl, 31);
      incl -= c;
      __syncwarp();  // the keys of these rows are read, before earlier places are written
      uint32_t t = at.ties + (incl & 1023), l = at.less + (incl >> 10 & 1023), m = at.more + (incl >> 20);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = i + j < w1, low = lo + i + j < keep;
        const bool tie = key[j] == prefix, stays = key[j] > prefix || (tie && t < need);
        if (in && low && !stays) packed[l + t - min(t, need) - hole0] = lo + i + j;
        if (in && !low && stays) packed[holes + m + min(t, need) - mover0] = lo + i + j;
        t += in && tie;
        l += in && low && key[j] < prefix;
        m += in && !low && key[j] > prefix;
      }
      at.ties += all & 1023;
      at.less += all >> 10 & 1023;
      at.more += all >> 20;
    }
    __syncwarp();
    if (keep > 0) {
      const uint32_t movers = at.more + min(at.ties, need) - mover0;
      for (uint32_t e = lane; e < holes; e += 32) list[hole0 + e] = packed[e];
      for (uint32_t e = lane; e < movers; e += 32) list[a.half + mover0 - stay_low + e] = packed[holes + e];
    }
    const int moves = keep > 0 ? less + ties_low - stay_low : 0;
    if constexpr (RB > 0) {
      sync_all();  // the lists are written
      move_rows<RB>(a, s, h, moves, rank * kEvWarps + warp, R * kEvWarps);
    } else if (tid == 0 && rank == 0) {
      a.moves[(int64_t)s * p.h_kv + h] = moves;
    }
  } else if (RB == 0 && tid == 0 && rank == 0) {
    a.moves[(int64_t)s * p.h_kv + h] = 0;
  }
  if (tid == 0 && rank == 0 && h == 0) a.lens_out[s] = go ? keep : len;

  if (CL) cluster_sync_all();  // shared memory stays readable until every rank is done
}

template <int RB>
__global__ void __launch_bounds__(kMvThreads, kMvCtas) evict_move_kernel(const __grid_constant__ EvArgs a) {
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.y, s = blockIdx.z;
  const int moves = a.moves[(int64_t)s * a.pages.h_kv + h];
  move_rows<RB>(a, s, h, moves, blockIdx.x * (kMvThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kMvThreads / 32));
}

// ------------------------------------------------------------------ host

struct EvPlan {
  Pages pages;
  int ranks, row_bytes, half, sms;
  size_t smem, lists_off, total;
};

int ev_plan(const aircache_evict_problem* p, EvPlan& pl) {
  if (!p) return AIRCACHE_ERR_INVALID_ARG;
  const int rc = check_pages(p->pages, pl.pages);
  if (rc != AIRCACHE_OK) return rc;
  if (!p->keep || !p->lens_out || !p->pages->mass || !p->mass_out ||
      (!p->order_out) != (!p->pages->order) || (reinterpret_cast<uintptr_t>(p->mass_out) & 15) != 0 ||
      (reinterpret_cast<uintptr_t>(p->order_out) & 15) != 0 || p->sink < 0 || p->recent < 0 ||
      ((p->sink || p->recent) && !p->pages->order) || (p->recent && !p->seen) || p->max_rows < 1)
    return AIRCACHE_ERR_INVALID_ARG;
  auto al4 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 3) == 0; };
  if (!al4(p->keep) || !al4(p->seen) || !al4(p->lens_out)) return AIRCACHE_ERR_INVALID_ARG;
  // lens_out is an array of its own; mass_out and order_out are the cache's, or lie apart from them and each other
  const size_t lens_bytes = 4 * (size_t)p->pages->num_seqs, slots = slot_bytes(pl.pages);
  for (const int32_t* x : {p->pages->lens, p->keep, p->seen})
    if (x == p->lens_out || arrays_meet(p->lens_out, lens_bytes, x, lens_bytes)) return AIRCACHE_ERR_INVALID_ARG;
  auto meet = [&](const void* x, const void* y) { return arrays_meet(x, slots, y, slots); };
  if ((p->mass_out != p->pages->mass && meet(p->mass_out, p->pages->mass)) ||
      (p->order_out != p->pages->order && meet(p->order_out, p->pages->order)) || meet(p->mass_out, p->order_out) ||
      meet(p->mass_out, p->pages->order) || meet(p->pages->mass, p->order_out))
    return AIRCACHE_ERR_INVALID_ARG;
  if (p->max_rows > AIRCACHE_MAX_EVICT_ROWS) return AIRCACHE_ERR_UNSUPPORTED;
  pl.sms = device_sms();
  const int64_t units = (int64_t)p->pages->num_seqs * p->pages->h_kv;
  // CTAs per (sequence, KV head): as many as leave every CTA an SM of its own
  // (16 x 16k with 128 CTAs 60.5 us, with 256 61.3), but at least 2048 rows to a CTA (each rank costs every
  // barrier and histogram sum), and as many as the keys need room
  int ranks = 1;
  while (ranks < kEvMaxCluster && units * ranks * 2 <= pl.sms && p->max_rows > 2048LL * ranks) ranks *= 2;
  while (p->max_rows > (int64_t)kEvSlice * ranks) ranks *= 2;
  pl.ranks = ranks;
  pl.row_bytes = p->pages->head_dim * (p->pages->kv_dtype == AIRCACHE_INT8 ? 1 : 2);
  pl.half = (int)((p->max_rows + 1) / 2);
  pl.smem = sizeof(uint32_t) * (size_t)(((p->max_rows + ranks - 1) / ranks + 15) / 16 * 16);
  pl.lists_off = kEvHeader + (sizeof(int32_t) * (size_t)units + 255) / 256 * 256;
  pl.total = pl.lists_off + (sizeof(int32_t) * 2 * (size_t)pl.half * (size_t)units + 255) / 256 * 256;
  return AIRCACHE_OK;
}

template <int R, int F, int RB>
int launch_select(const EvPlan& pl, const EvArgs& a, cudaStream_t s) {
  if (allow_smem(reinterpret_cast<const void*>(&evict_select_kernel<R, F, RB>), (int)pl.smem) != cudaSuccess)
    return AIRCACHE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(R, a.pages.h_kv, a.pages.num_seqs);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = R;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = R > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<R, F, RB>, a) == cudaSuccess ? AIRCACHE_OK : AIRCACHE_ERR_CUDA;
}

template <int R, int RB>
int launch_select(const EvPlan& pl, const EvArgs& a, cudaStream_t s) {
  const int64_t ctas = (int64_t)R * a.pages.h_kv * a.pages.num_seqs;
  return ctas <= pl.sms ? launch_select<R, 8, RB>(pl, a, s) : launch_select<R, 4, RB>(pl, a, s);
}

template <int RB>
int pick_select(const EvPlan& pl, const EvArgs& a, cudaStream_t s) {
  switch (pl.ranks) {
    case 1: return launch_select<1, RB>(pl, a, s);
    case 2: return launch_select<2, RB>(pl, a, s);
    case 4: return launch_select<4, RB>(pl, a, s);
    default: return launch_select<8, RB>(pl, a, s);
  }
}

template <int RB>
int launch_move(const EvPlan& pl, const EvArgs& a, cudaStream_t s) {
  // four waves over all (sequence, KV head) pairs, which walk over their moves
  const int64_t units = (int64_t)a.pages.h_kv * a.pages.num_seqs;
  const int64_t x = std::min<int64_t>((pl.half + kMvThreads - 1) / kMvThreads, (4LL * kMvCtas * pl.sms + units - 1) / units);
  return launch_pdl(evict_move_kernel<RB>, dim3((unsigned)x, a.pages.h_kv, a.pages.num_seqs), dim3(kMvThreads), 0, s,
                    a) == cudaSuccess
             ? AIRCACHE_OK
             : AIRCACHE_ERR_CUDA;
}

}  // namespace
}  // namespace aircache

using namespace aircache;

extern "C" {

size_t aircache_evict_workspace_size(const aircache_evict_problem* p) {
  EvPlan pl;
  return ev_plan(p, pl) == AIRCACHE_OK ? pl.total : 0;
}

int aircache_evict(const aircache_evict_problem* p, void* ws, size_t ws_bytes, void* stream) {
  EvPlan pl;
  const int rc = ev_plan(p, pl);
  if (rc != AIRCACHE_OK) return rc;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) return AIRCACHE_ERR_INVALID_ARG;
  if (ws_bytes < pl.total) return AIRCACHE_ERR_WORKSPACE;
  if (p->pages->num_seqs == 0) return AIRCACHE_OK;
  EvArgs a;
  a.pages = pl.pages;
  a.keep = p->keep;
  a.seen = p->seen;
  a.lens_out = p->lens_out;
  a.mass_out = p->mass_out;
  a.order_out = p->order_out;
  a.error = static_cast<int32_t*>(ws);
  a.moves = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kEvHeader);
  a.lists = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + pl.lists_off);
  a.half = pl.half;
  a.max_rows = (int)p->max_rows;
  a.sink = p->sink;
  a.recent = p->recent;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->max_rows <= kEvShort * std::max<int64_t>(pl.ranks, 2)) {
    switch (pl.row_bytes) {
      case 256: return pick_select<16>(pl, a, s);
      case 128: return pick_select<8>(pl, a, s);
      default: return pick_select<4>(pl, a, s);
    }
  }
  const int sel = pick_select<0>(pl, a, s);
  if (sel != AIRCACHE_OK) return sel;
  switch (pl.row_bytes) {
    case 256: return launch_move<16>(pl, a, s);
    case 128: return launch_move<8>(pl, a, s);
    default: return launch_move<4>(pl, a, s);
  }
}

}  // extern "C"
