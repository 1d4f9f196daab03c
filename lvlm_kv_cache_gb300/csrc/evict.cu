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
// shared memory (the mass as an order-preserving integer); the threshold is
// found by radix selection, four digits of 8 bits, adding up the CTAs'
// histograms through distributed shared memory.  Its warps then walk over
// consecutive rows and list vacated rows and movers in order.  Bound by the
// chain of barriers and scans: 8 bytes a row are read.
// move: CTAs over all SMs copy the listed rows, 32 moves to a warp at a time.
// Bound by HBM.
#include <algorithm>

#include "pages.cuh"

namespace aircache {
namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvMaxCluster = 8;
constexpr int kMvThreads = 256;
constexpr int kEvSlice = AIRCACHE_MAX_EVICT_ROWS / kEvMaxCluster;  // keys of one CTA, at most
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

struct EvShared {
  uint32_t hist[4][256];
  uint32_t spread[256][8];  // the first digit's counts, eight copies: few values, many rows
  uint32_t total[256];
  Before warp[kEvWarps];
  Before sum;
  uint32_t digit, above;
  int bad;
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

// CL: a cluster of gridDim.x CTAs per (sequence, KV head); else one CTA.
template <bool CL>
__global__ void __launch_bounds__(kEvThreads) evict_select_kernel(const __grid_constant__ EvArgs a) {
  extern __shared__ uint32_t ev_keys[];
  __shared__ EvShared sh;
  const Pages& p = a.pages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ranks = CL ? gridDim.x : 1, rank = CL ? blockIdx.x : 0;  // the cluster spans x
  const int h = blockIdx.y, s = blockIdx.z;
  auto sync_all = [] {
    if (CL)
      cluster_sync_all();
    else
      __syncthreads();
  };
  auto peer = [&](const uint32_t* x, int r) { return CL ? ld_cluster_u32(cluster_map(smem_u32(x), r)) : *x; };
  pdl_trigger();
  for (int i = tid; i < 4 * 256; i += kEvThreads) (&sh.hist[0][0])[i] = 0;
  for (int i = tid; i < 8 * 256; i += kEvThreads) (&sh.spread[0][0])[i] = 0;
  if (tid == 0) sh.bad = 0;
  __syncthreads();
  pdl_wait();

  const int len = p.lens[s], keep = a.keep[s];
  const bool sane = len >= 0 && len <= a.max_rows && len <= p.max_rows && keep >= 0 &&
                    (len <= keep || (int64_t)keep >= (int64_t)a.sink + a.recent);
  if (!sane && tid == 0) set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
  const int n = sane ? len : 0;
  const bool cut = sane && n > keep;
  const int per = ((n + ranks - 1) / ranks + 15) & ~15;
  const int lo = min(rank * per, n), mine = min(per, n - lo);  // this CTA's rows
  const int32_t* table = p.table + (int64_t)s * p.table_stride;
  const int32_t fresh = a.seen && a.recent ? a.seen[s] - a.recent : 0x7fffffff;  // order from which rows are recent
  const bool aged = a.sink | a.recent;

  // ---- keys of the slice, and the first digit's counts.  Four rows a thread
  // (a page holds a multiple of 16), four such groups in flight
  constexpr int kFlight = 4;
  for (int i0 = 4 * tid; i0 < mine; i0 += 4 * kFlight * kEvThreads) {
    int page[kFlight];
    float4 m[kFlight];
    int4 o[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = i0 + 4 * f * kEvThreads;
      page[f] = i < mine ? table[(lo + i) / p.page_rows] : 0;
    }
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int i = i0 + 4 * f * kEvThreads;
      m[f] = make_float4(0.f, 0.f, 0.f, 0.f);
      o[f] = make_int4(0, 0, 0, 0);
      if (i < mine) {
        if (page_ok(p, page[f])) {
          const int64_t slot = page_slot(p, page[f], h, (lo + i) % p.page_rows);
          m[f] = *reinterpret_cast<const float4*>(p.mass + slot);
          if (aged) o[f] = *reinterpret_cast<const int4*>(p.order + slot);
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
      uint32_t key[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        key[j] = aged && (oo[j] < a.sink || oo[j] >= fresh) ? kProtected : mass_key(mm[j]);
        if (cut && i + j < mine) atomicAdd(&sh.spread[key[j] >> 24][lane & 7], 1u);
      }
      *reinterpret_cast<uint4*>(ev_keys + i) = make_uint4(key[0], key[1], key[2], key[3]);
    }
  }
  __syncthreads();
  if (tid < 256) {
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) c += sh.spread[tid][j];
    sh.hist[0][tid] = c;
  }
  sync_all();
  bool bad = false;
  for (int x = 0; x < ranks; ++x) bad |= peer(reinterpret_cast<const uint32_t*>(&sh.bad), x) != 0;
  if (bad && tid == 0) set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
  const bool go = cut && !bad;

  // ---- the keep-th largest key, digit by digit
  uint32_t prefix = 0, need = keep;  // need: rows still to take among those that share the prefix
  if (go && keep > 0) {
    for (int d = 0; d < 4; ++d) {
      const int shift = 24 - 8 * d;
      if (d > 0) {
        for (int i = tid; i < mine; i += kEvThreads) {
          const uint32_t key = ev_keys[i];
          if ((key >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&sh.hist[d][(key >> shift) & 255], 1u);
        }
        sync_all();
      }
      if (tid < 256) {
        uint32_t c = 0;
#pragma unroll
        for (int x = 0; x < (CL ? kEvMaxCluster : 1); ++x)
          if (x < ranks) c += peer(&sh.hist[d][tid], x);
        sh.total[tid] = c;
      }
      __syncthreads();
      if (warp == 0) {  // lane 0 has the largest digits
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i] = sh.total[255 - 8 * lane - i];
        uint32_t incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const uint32_t t = __shfl_up_sync(0xffffffffu, incl, off);
          if (lane >= off) incl += t;
        }
        uint32_t above = incl - sum;
        if (above < need && incl >= need) {
          int digit = 0;
          uint32_t over = 0;
          bool found = false;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (!found && above + c[i] >= need) found = true, digit = 255 - 8 * lane - i, over = above;
            above += c[i];
          }
          sh.digit = digit;
          sh.above = over;
        }
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      need -= sh.above;
    }
  }

  // ---- ranks.  Of the rows at the threshold the `need` lowest stay, so with T
  // ties, L lesser rows (below keep) and M greater rows (at keep and behind) before a row, L + T -
  // min(T, need) rows were vacated and M + min(T, need) - min(ties below keep, need) moved.
  // A warp walks over consecutive rows
  const int span = ((mine + kEvWarps - 1) / kEvWarps + 31) & ~31;
  const int w0 = min(warp * span, mine), w1 = min(w0 + span, mine);
  if (go) {
    Before b = {0, 0, 0, 0};
    for (int i = w0 + lane; i - lane < w1; i += 32) {
      const uint32_t key = i < w1 ? ev_keys[i] : 0;
      const bool in = i < w1, low = lo + i < keep;
      b.ties += __popc(__ballot_sync(0xffffffffu, in && key == prefix));
      b.ties_low += __popc(__ballot_sync(0xffffffffu, in && low && key == prefix));
      b.less += __popc(__ballot_sync(0xffffffffu, in && low && key < prefix));
      b.more += __popc(__ballot_sync(0xffffffffu, in && !low && key > prefix));
    }
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
    uint32_t ties_low = 0, less = 0;
    for (int x = 0; x < ranks; ++x) {
      const uint32_t t = peer(&sh.sum.ties, x), tl = peer(&sh.sum.ties_low, x), l = peer(&sh.sum.less, x),
                     m = peer(&sh.sum.more, x);
      if (x < rank) at.ties += t, at.less += l, at.more += m;
      ties_low += tl;
      less += l;
    }
#pragma unroll
    for (int w = 0; w < kEvWarps; ++w)
      if (w < warp) at.ties += sh.warp[w].ties, at.less += sh.warp[w].less, at.more += sh.warp[w].more;
    if (keep == 0) at.more = 0;
    const uint32_t stay_low = min(ties_low, need);
    int32_t* list = a.lists + ((int64_t)s * p.h_kv + h) * 2 * a.half;
    const uint32_t under = (1u << lane) - 1;
    for (int i = w0 + lane; i - lane < w1 && keep > 0; i += 32) {
      const uint32_t key = i < w1 ? ev_keys[i] : 0;
      const bool in = i < w1, low = lo + i < keep;
      const uint32_t tie = __ballot_sync(0xffffffffu, in && key == prefix);
      const uint32_t lesser = __ballot_sync(0xffffffffu, in && low && key < prefix);
      const uint32_t greater = __ballot_sync(0xffffffffu, in && !low && key > prefix);
      const uint32_t t = at.ties + __popc(tie & under);  // ties before this row
      const bool stays = key > prefix || (key == prefix && t < need);
      if (in && low && !stays) list[at.less + __popc(lesser & under) + t - min(t, need)] = lo + i;
      if (in && !low && stays)
        list[a.half + at.more + __popc(greater & under) + min(t, need) - stay_low] = lo + i;
      if (in) ev_keys[i] = stays;
      at.ties += __popc(tie);
      at.less += __popc(lesser);
      at.more += __popc(greater);
    }
    if (tid == 0 && rank == 0) a.moves[(int64_t)s * p.h_kv + h] = keep > 0 ? less + ties_low - stay_low : 0;
  } else if (tid == 0 && rank == 0) {
    a.moves[(int64_t)s * p.h_kv + h] = 0;
  }
  if (tid == 0 && rank == 0 && h == 0) a.lens_out[s] = go ? keep : len;

  // ---- rows that stay where they are: mass and order, if these go to other arrays
  const bool copy_mass = a.mass_out != p.mass, copy_order = a.order_out && a.order_out != p.order;
  if ((copy_mass || copy_order) && sane && !bad) {
    __syncthreads();
    const int new_len = cut ? keep : n;
    for (int i = tid; i < mine && lo + i < new_len; i += kEvThreads) {
      if (go && !ev_keys[i]) continue;
      const int64_t slot = page_slot(p, table[(lo + i) / p.page_rows], h, (lo + i) % p.page_rows);
      if (copy_mass) a.mass_out[slot] = p.mass[slot];
      if (copy_order) a.order_out[slot] = p.order[slot];
    }
  }
  if (CL) cluster_sync_all();  // shared memory stays readable until every rank is done
}

// RB: 16-byte pieces of a row of one KV head.
template <int RB>
__global__ void __launch_bounds__(kMvThreads) evict_move_kernel(const __grid_constant__ EvArgs a) {
  pdl_trigger();
  pdl_wait();
  const Pages& p = a.pages;
  const int lane = threadIdx.x & 31;
  const int h = blockIdx.y, s = blockIdx.z;
  const int64_t unit = (int64_t)s * p.h_kv + h;
  const int moves = a.moves[unit];
  const int32_t* table = p.table + (int64_t)s * p.table_stride;
  const int32_t* list = a.lists + unit * 2 * a.half;
  constexpr int kAtOnce = 32 / (2 * RB);  // moves of one warp instruction
  const int piece = lane % RB, sub = lane / (2 * RB);
  uint8_t* const kv = ((lane / RB) & 1 ? p.v : p.k) + 16 * piece;
  const int size = p.k_scale ? 1 : 2;
  for (int m0 = 32 * (blockIdx.x * (kMvThreads / 32) + (threadIdx.x >> 5)); m0 < moves;
       m0 += 32 * gridDim.x * (kMvThreads / 32)) {
    int64_t src = 0, dst = 0;
    const int cnt = min(32, moves - m0);
    if (lane < cnt) {
      const int to = list[m0 + lane], from = list[a.half + m0 + lane];
      const int tp = table[to / p.page_rows], fp = table[from / p.page_rows];
      const int tr = to % p.page_rows, fr = from % p.page_rows;
      const int64_t ds = page_slot(p, tp, h, tr), ss = page_slot(p, fp, h, fr);
      a.mass_out[ds] = p.mass[ss];
      if (a.order_out) a.order_out[ds] = p.order[ss];
      if (p.k_scale) {
        p.k_scale[ds] = p.k_scale[ss];
        p.v_scale[ds] = p.v_scale[ss];
      }
      dst = page_elem(p, tp, h, tr) * size;
      src = page_elem(p, fp, h, fr) * size;
    }
    constexpr int kFlight = 8;
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
  }
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
  if (!p->keep || !p->lens_out || p->lens_out == p->pages->lens || !p->pages->mass || !p->mass_out ||
      (!p->order_out) != (!p->pages->order) || p->sink < 0 || p->recent < 0 ||
      ((p->sink || p->recent) && !p->pages->order) || (p->recent && !p->seen) || p->max_rows < 1)
    return AIRCACHE_ERR_INVALID_ARG;
  if (p->max_rows > AIRCACHE_MAX_EVICT_ROWS) return AIRCACHE_ERR_UNSUPPORTED;
  int dev = 0;
  pl.sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&pl.sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t units = (int64_t)p->pages->num_seqs * p->pages->h_kv;
  // CTAs per (sequence, KV head): enough that the batch fills the SMs twice,
  // but at least 2048 rows to a CTA (each rank costs every barrier and
  // histogram sum), and as many as the keys need room
  int ranks = 1;
  while (ranks < kEvMaxCluster && (units * ranks * 2 <= 2 * pl.sms) && p->max_rows > 2048LL * ranks) ranks *= 2;
  while (p->max_rows > (int64_t)kEvSlice * ranks) ranks *= 2;
  pl.ranks = ranks;
  pl.row_bytes = p->pages->head_dim * (p->pages->kv_dtype == AIRCACHE_INT8 ? 1 : 2);
  pl.half = (int)((p->max_rows + 1) / 2);
  pl.smem = sizeof(uint32_t) * (size_t)(((p->max_rows + ranks - 1) / ranks + 15) / 16 * 16);
  pl.lists_off = kEvHeader + (sizeof(int32_t) * (size_t)units + 255) / 256 * 256;
  pl.total = pl.lists_off + (sizeof(int32_t) * 2 * (size_t)pl.half * (size_t)units + 255) / 256 * 256;
  return AIRCACHE_OK;
}

template <bool CL>
int launch_select(const EvPlan& pl, const EvArgs& a, cudaStream_t s) {
  if (allow_smem(reinterpret_cast<const void*>(&evict_select_kernel<CL>), (int)pl.smem) != cudaSuccess)
    return AIRCACHE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.ranks, a.pages.h_kv, a.pages.num_seqs);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = pl.ranks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CL ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel<CL>, a) == cudaSuccess ? AIRCACHE_OK : AIRCACHE_ERR_CUDA;
}

template <int RB>
int launch_move(const EvPlan& pl, const EvArgs& a, cudaStream_t s) {
  // two waves of eight CTAs to an SM over all (sequence, KV head) pairs, which
  // walk over their moves
  const int64_t units = (int64_t)a.pages.h_kv * a.pages.num_seqs;
  const int64_t x = std::min<int64_t>((pl.half + kMvThreads - 1) / kMvThreads, (16LL * pl.sms + units - 1) / units);
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
  const int sel = pl.ranks > 1 ? launch_select<true>(pl, a, s) : launch_select<false>(pl, a, s);
  if (sel != AIRCACHE_OK) return sel;
  switch (pl.row_bytes) {
    case 256: return launch_move<16>(pl, a, s);
    case 128: return launch_move<8>(pl, a, s);
    default: return launch_move<4>(pl, a, s);
  }
}

}  // extern "C"
