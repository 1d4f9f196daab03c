// Eviction from the paged cache by accumulated attention weight (aircache_evict).
//
// Of a sequence's n rows every KV head keeps the `keep` best (protected rows
// first, then by mass, ties to the lower row).  A row's rank is all that
// matters and attention does not mind the rows' order, so only kept rows
// behind `keep` move: the j-th of them into the j-th vacated row below
// `keep`.  That reads and writes each moved row once, and no destination is
// another move's source, so the moves need no order.
//
// One thread-block cluster per (sequence, KV head); each CTA holds the keys of
// a slice of the rows in shared memory (the mass as an order-preserving
// integer) and the cluster finds the threshold by radix selection, four
// digits of 8 bits, adding up the CTAs' histograms through distributed shared
// memory.  Ties, vacated rows and movers are ranked by scans over
// consecutive rows; the two lists go through the workspace, and the
// cluster's warps copy the rows, 32 moves at a time.  Bound by HBM (rows moved)
// for large batches, by the chain of cluster barriers for small ones.
#include <algorithm>

#include "pages.cuh"

namespace aircache {
namespace {

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvMaxCluster = 8;
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
  int32_t* lists;  // [units][2][half]: vacated rows, movers
  int half;        // max_rows / 2
  int max_rows, sink, recent;
};

struct EvShared {
  uint32_t hist[4][256];
  uint32_t total[256];
  uint64_t scan[kEvWarps];
  uint64_t count[2];  // this CTA's ties; its vacated rows and movers (low and high half)
  uint32_t digit, above;
  int bad;
};

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t addr) {
  uint64_t v;
  asm volatile("ld.shared::cluster.u64 %0, [%1];\n" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// Larger for the row to keep: fp32 order as integers, -0 as 0, NaN as -inf.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) x = -INFINITY;
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Sum of `x` over the threads before this one; the block's sum goes to *total.
__device__ __forceinline__ uint64_t block_before(uint64_t x, uint64_t* scan, uint64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint64_t t = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += t;
  }
  __syncthreads();  // an earlier scan is read
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  uint64_t before = incl - x, all = 0;
#pragma unroll
  for (int w = 0; w < kEvWarps; ++w) {
    if (w < warp) before += scan[w];
    all += scan[w];
  }
  if (threadIdx.x == 0) *total = all;
  return before;
}

// RB: 16-byte pieces of a row of one KV head.
template <int RB>
__global__ void __launch_bounds__(kEvThreads) evict_kernel(const __grid_constant__ EvArgs a) {
  extern __shared__ uint32_t ev_keys[];
  __shared__ EvShared sh;
  const Pages& p = a.pages;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ranks = gridDim.x, rank = blockIdx.x;  // the cluster spans x
  const int h = blockIdx.y, s = blockIdx.z;
  pdl_trigger();
  for (int i = tid; i < 4 * 256; i += kEvThreads) (&sh.hist[0][0])[i] = 0;
  if (tid == 0) sh.bad = 0;
  __syncthreads();
  pdl_wait();

  const int len = p.lens[s], keep = a.keep[s];
  const bool sane = len >= 0 && len <= a.max_rows && len <= p.max_rows && keep >= 0 &&
                    (len <= keep || (int64_t)keep >= (int64_t)a.sink + a.recent);
  if (!sane && tid == 0) set_error(a.error, AIRCACHE_ERR_DEVICE_BOUNDS);
  const int n = sane ? len : 0;
  const bool cut = sane && n > keep;
  const int per = (n + ranks - 1) / ranks;
  const int lo = min(rank * per, n), mine = min(per, n - lo);  // this CTA's rows
  const int32_t* table = p.table + (int64_t)s * p.table_stride;
  const int32_t fresh = a.seen && a.recent ? a.seen[s] - a.recent : 0x7fffffff;  // order from which rows are recent

  // ---- keys of the slice, and the first digit's counts
  for (int i = tid; i < mine; i += kEvThreads) {
    const int row = lo + i, page = table[row / p.page_rows];
    uint32_t key = 0;
    if (!page_ok(p, page)) {
      sh.bad = 1;
    } else {
      const int64_t slot = page_slot(p, page, h, row % p.page_rows);
      key = mass_key(p.mass[slot]);
      if (a.sink | a.recent) {
        const int32_t order = p.order[slot];
        if (order < a.sink || order >= fresh) key = kProtected;
      }
    }
    ev_keys[i] = key;
    if (cut) atomicAdd(&sh.hist[0][key >> 24], 1u);
  }
  cluster_sync_all();
  bool bad = false;
  for (int x = 0; x < ranks; ++x) bad |= ld_cluster_u32(cluster_map(smem_u32(&sh.bad), x)) != 0;
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
        cluster_sync_all();
      }
      if (tid < 256) {
        uint32_t c = 0;
        for (int x = 0; x < ranks; ++x) c += ld_cluster_u32(cluster_map(smem_u32(&sh.hist[d][tid]), x));
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
          int i = 0;
          while (i < 7 && above + c[i] < need) above += c[i++];
          sh.digit = 255 - 8 * lane - i;
          sh.above = above;
        }
      }
      __syncthreads();
      prefix |= sh.digit << shift;
      need -= sh.above;
      __syncthreads();
    }
  }

  // ---- which ties stay: the `need` lowest of them.  A thread walks over
  // consecutive rows; an odd number of them, so that a warp's keys lie in 32 banks
  const int seg = ((mine + kEvThreads - 1) / kEvThreads) | 1;
  const int i0 = min(tid * seg, mine), i1 = min(i0 + seg, mine);
  uint64_t moves = 0;
  if (go) {
    uint32_t ties = 0;
    for (int i = i0; i < i1; ++i) ties += ev_keys[i] == prefix;
    uint64_t tie = block_before(ties, sh.scan, &sh.count[0]);
    cluster_sync_all();
    for (int x = 0; x < rank; ++x) tie += ld_cluster_u64(cluster_map(smem_u32(&sh.count[0]), x));
    // ---- vacated rows below keep, movers at keep and behind
    uint32_t holes = 0, movers = 0;
    for (int i = i0; i < i1; ++i) {
      const uint32_t key = ev_keys[i];
      bool stay = key > prefix;
      if (key == prefix) stay = tie++ < need;
      if (keep == 0) stay = false;
      holes += !stay && lo + i < keep;
      movers += stay && lo + i >= keep;
      ev_keys[i] = stay;
    }
    uint64_t at = block_before((uint64_t)movers << 32 | holes, sh.scan, &sh.count[1]);
    cluster_sync_all();
    for (int x = 0; x < ranks; ++x) {
      const uint64_t c = ld_cluster_u64(cluster_map(smem_u32(&sh.count[1]), x));
      if (x < rank) at += c;
      moves += c & 0xffffffffu;
    }
    int32_t* list = a.lists + ((int64_t)s * p.h_kv + h) * 2 * a.half;
    uint32_t jh = (uint32_t)at, jm = (uint32_t)(at >> 32);
    for (int i = i0; i < i1; ++i) {
      const bool stay = ev_keys[i];
      if (!stay && lo + i < keep) list[jh++] = lo + i;
      if (stay && lo + i >= keep) list[a.half + jm++] = lo + i;
    }
    __threadfence();
  }
  cluster_sync_all();

  // ---- rows that stay where they are: mass and order, if these go to other arrays
  const bool copy_mass = a.mass_out != p.mass, copy_order = a.order_out && a.order_out != p.order;
  if ((copy_mass || copy_order) && sane && !bad) {
    const int new_len = cut ? keep : n;
    for (int i = tid; i < mine && lo + i < new_len; i += kEvThreads) {
      if (go && !ev_keys[i]) continue;
      const int64_t slot = page_slot(p, table[(lo + i) / p.page_rows], h, (lo + i) % p.page_rows);
      if (copy_mass) a.mass_out[slot] = p.mass[slot];
      if (copy_order) a.order_out[slot] = p.order[slot];
    }
  }
  if (tid == 0 && rank == 0 && h == 0) a.lens_out[s] = go ? keep : len;

  // ---- the moves: a warp takes 32 of them, 16 bytes of a key or value a lane
  const int32_t* list = a.lists + ((int64_t)s * p.h_kv + h) * 2 * a.half;
  constexpr int kAtOnce = 32 / (2 * RB);
  const int piece = lane % RB, sub = lane / (2 * RB);
  uint8_t* const kv = (lane / RB) & 1 ? p.v : p.k;
  for (uint64_t m0 = 32 * ((uint64_t)rank * kEvWarps + warp); m0 < moves; m0 += 32 * (uint64_t)ranks * kEvWarps) {
    int64_t src = 0, dst = 0;
    const int cnt = (int)(moves - m0 < 32 ? moves - m0 : 32);
    if (lane < cnt) {
      const int to = __ldcg(list + m0 + lane), from = __ldcg(list + a.half + m0 + lane);
      const int tp = table[to / p.page_rows], fp = table[from / p.page_rows];
      const int tr = to % p.page_rows, fr = from % p.page_rows;
      const int64_t ds = page_slot(p, tp, h, tr), ss = page_slot(p, fp, h, fr);
      a.mass_out[ds] = p.mass[ss];
      if (a.order_out) a.order_out[ds] = p.order[ss];
      if (p.k_scale) {
        p.k_scale[ds] = p.k_scale[ss];
        p.v_scale[ds] = p.v_scale[ss];
      }
      const int size = p.k_scale ? 1 : 2;
      dst = page_elem(p, tp, h, tr) * size;
      src = page_elem(p, fp, h, fr) * size;
    }
#pragma unroll 4
    for (int j = 0; j < 32; j += kAtOnce) {
      const int64_t from = __shfl_sync(0xffffffffu, src, j + sub), to = __shfl_sync(0xffffffffu, dst, j + sub);
      if (j + sub < cnt)
        *reinterpret_cast<uint4*>(kv + to + 16 * piece) = *reinterpret_cast<const uint4*>(kv + from + 16 * piece);
    }
  }
  cluster_sync_all();  // shared memory stays readable until every rank is done
}

// ------------------------------------------------------------------ host

struct EvPlan {
  Pages pages;
  int ranks, row_bytes, half;
  size_t smem, total;
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
  int dev = 0, sms = 152;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t units = (int64_t)p->pages->num_seqs * p->pages->h_kv;
  // CTAs per (sequence, KV head): enough that the batch fills the SMs twice,
  // but at least 1024 rows to a CTA (each rank costs every barrier and
  // histogram sum), and as many as the keys need room
  int ranks = 1;
  while (ranks < kEvMaxCluster && (units * ranks * 2 <= 2 * sms) && p->max_rows > 1024LL * ranks) ranks *= 2;
  while (p->max_rows > (int64_t)kEvSlice * ranks) ranks *= 2;
  pl.ranks = ranks;
  pl.row_bytes = p->pages->head_dim * (p->pages->kv_dtype == AIRCACHE_INT8 ? 1 : 2);
  pl.half = (int)((p->max_rows + 1) / 2);
  pl.smem = sizeof(uint32_t) * (size_t)((p->max_rows + ranks - 1) / ranks);
  pl.total = kEvHeader + (sizeof(int32_t) * 2 * (size_t)pl.half * (size_t)units + 255) / 256 * 256;
  return AIRCACHE_OK;
}

template <int RB>
int launch_evict(const EvPlan& pl, const EvArgs& a, cudaStream_t s) {
  if (allow_smem(reinterpret_cast<const void*>(&evict_kernel<RB>), (int)pl.smem) != cudaSuccess)
    return AIRCACHE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pl.ranks, a.pages.h_kv, a.pages.num_seqs);
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = pl.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = pl.ranks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_kernel<RB>, a) == cudaSuccess ? AIRCACHE_OK : AIRCACHE_ERR_CUDA;
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
  a.lists = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kEvHeader);
  a.half = pl.half;
  a.max_rows = (int)p->max_rows;
  a.sink = p->sink;
  a.recent = p->recent;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (pl.row_bytes) {
    case 256: return launch_evict<16>(pl, a, s);
    case 128: return launch_evict<8>(pl, a, s);
    default: return launch_evict<4>(pl, a, s);
  }
}

}  // extern "C"
