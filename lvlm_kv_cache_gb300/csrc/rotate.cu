// Norms of queries and keys for each head, the rotation by position and the
// append to the paged cache (aircache_rotate).
//
// Per token, head and element: x' = x rsqrt(mean x^2 + eps) w; the pairs
// (a, b) of the first R elements become (a cos - b sin, b cos + a sin).  A few
// operations per 4 bytes moved: bound by HBM, or by latency for a handful of
// tokens.
//
// D/8 lanes take one head's row, eight elements a lane, so a warp works on 2 (D =
// 128) or 4 (D = 64) rows at once; it walks over the query, key and value heads
// of ONE token, so that the token's sines and cosines are formed once, in the
// registers of the lanes that need them, multiplied by the norm's weights, and
// the slot in the cache is looked up once.  Both elements of a pair lie in one
// lane (half style: four elements and the four half a rotation further), so a
// row costs no shuffles but the norm's.  With few tokens a token's heads go to
// several warps.  Measured: 8 tokens of 28 + 4 heads of 128 in 2.8 us within a graph (a call by
// itself takes the host 3.9); 15,541 of them, the keys also dense, in 53 us (303 MB read and
// written, 5.8 TB/s), and into an int8 cache, without those, in 61.
//
// The angle: position * (hi + lo) turns is reduced before it is rounded.  The
// position splits into two parts of at most 20 bits (exact in fp32), each
// product with hi is taken with its rounding error (one multiplication and one
// fused multiply-add, an error-free product), whole turns are dropped, and
// the rest goes to sincospif: to about 2^-24 turns up to position 2^24, and to
// 2^-19 turns at the far end of int32, where lo's own last bit shows.
#include <algorithm>

#include "int8code.cuh"
#include "pages.cuh"

namespace aircache {
namespace {

// A CTA is one warp: the next token starts as soon as one is done (15,541 tokens: 6 % longer with
// four warps to a CTA, 5 % with two).
// NB: rows a lane group works on at a time, while as many load.  Two, with 32 warps
// to an SM (15,541 tokens of 28 + 4 heads of 128: 14 % longer with four); four, with 24 warps,
// where whole tokens do not fill those, so that a warp has to keep more loads of its own in flight
// (3,447 tokens of 32 + 32 heads of 64: 12 % longer with two).
constexpr int kRotMany = 32, kRotFew = 24;  // warps to an SM
// (The bounds on the kernels' registers: as 32 CTAs of 32 threads for NB = 2 and, though it is launched
// with 32 threads, as 6 of 128 for NB = 4; the other way round 4 and 6 % longer.)

struct RotArgs {
  const __nv_bfloat16* src[3];  // q, k, v
  int64_t src_tok[3], src_head[3];
  __nv_bfloat16* out[2];  // q_out, k_out
  int64_t out_tok[2], out_head[2];
  const __nv_bfloat16* weight[2];
  const float2* turns;
  const int32_t* positions;
  const int32_t* cu_tokens;
  const int32_t* seen;
  int32_t* status;
  int64_t num_tokens;
  Pages pages;
  int num_seqs, h_q, h_kv, heads;  // heads: rows of one token that the call touches
  int rot, axes, sec0, sec1, has_pages;
  int per, shares;  // heads of one token that one warp takes, and warps to a token
  float eps;
};

// Sequence of token t: the last s with cu[s] <= t; 32 candidates a step.
__device__ __forceinline__ int find_seq(const int32_t* cu, int n, int t, int lane) {
  int lo = 0, len = n + 1;  // entries lo .. lo+len-1 may hold it
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int i = lo + lane * step;
    const bool le = lane * step < len && cu[i] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) return -1;
    lo += (c - 1) * step;
    len = min(step, len - (c - 1) * step);
  }
  return lo;
}

__device__ __forceinline__ void unpack8(const uint4& w, float x[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float x[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 t = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&t);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// sin and cos of 2 pi * position * (hi + lo)
__device__ __forceinline__ void turn(int pos, float2 f, float& sn, float& cs) {
  const float a = (float)(pos & ~0xfff), b = (float)(pos & 0xfff);
  const float p1 = __fmul_rn(a, f.x), p2 = __fmul_rn(b, f.x);
  const float e1 = __fmaf_rn(a, f.x, -p1), e2 = __fmaf_rn(b, f.x, -p2);
  const float rest = (e1 + e2) + __fmaf_rn(a, f.y, __fmul_rn(b, f.y));
  float r = (p1 - rintf(p1)) + (p2 - rintf(p2));
  r = (r - rintf(r)) + rest;
  sincospif(2.f * r, &sn, &cs);
}

// What a lane does to each row of its token.
struct Lane {
  int e0, e1;           // its elements: e0 .. e0+3 and e1 .. e1+3
  float cs[4], sn[4];   // of its four pairs
  bool turned;          // false: elements behind rotary_dim
  int page, row, order; // the token's slot (page < 0: none)
};

// The next rows of a token's queries, keys or values, a lane's eight elements of each.
template <int NB>
struct Batch {
  uint2 lo[NB], hi[NB];
};
// WIDE: the eight elements are one 16-byte piece (interleaved pairs, and values, which do not turn).
template <int D, bool WIDE, int NB>
__device__ __forceinline__ void load_rows(Batch<NB>& r, const __nv_bfloat16* src, int64_t head_stride, int j0, int last,
                                          int e0, int e1, int lane) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int j = j0 + b * kRows + lane / kLanes;
    r.lo[b] = r.hi[b] = make_uint2(0u, 0u);
    if (j < last) {
      const __nv_bfloat16* from = src + j * head_stride;
      if (WIDE) {
        const uint4 v = *reinterpret_cast<const uint4*>(from + 8 * (lane % kLanes));
        r.lo[b] = make_uint2(v.x, v.y);
        r.hi[b] = make_uint2(v.z, v.w);
      } else {
        r.lo[b] = *reinterpret_cast<const uint2*>(from + e0);
        r.hi[b] = *reinterpret_cast<const uint2*>(from + e1);
      }
    }
  }
}

// Heads first .. last-1 of the token: KIND 0 queries, 1 keys, 2 values.  `r` holds the first of them.
template <int D, bool Q8, bool INTER, int KIND, int NB>
__device__ __forceinline__ void rows_of_token(const RotArgs& a, const Lane& x, int64_t t, int first, int last,
                                              int lane, Batch<NB>& r) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  constexpr bool kWide = INTER || KIND == 2;
  const int l = lane % kLanes, grp = lane / kLanes;
  const __nv_bfloat16* src = a.src[KIND] + t * a.src_tok[KIND];
  // pair (u, v) of elements: u' = u c0 - v s1, v' = v c1 + u s0 (the weights inside)
  float c0[4], c1[4], s0[4], s1[4];
  const __nv_bfloat16* weight = KIND < 2 ? a.weight[KIND < 2 ? KIND : 0] : nullptr;
  if (KIND < 2) {
    float w[8] = {1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f};
    if (weight) {
      const uint2 wl = *reinterpret_cast<const uint2*>(weight + x.e0);
      const uint2 wh = *reinterpret_cast<const uint2*>(weight + x.e1);
      unpack8(make_uint4(wl.x, wl.y, wh.x, wh.y), w);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float wu = INTER ? w[2 * e] : w[e], wv = INTER ? w[2 * e + 1] : w[4 + e];
      c0[e] = x.cs[e] * wu;
      c1[e] = x.cs[e] * wv;
      s0[e] = x.sn[e] * wu;
      s1[e] = x.sn[e] * wv;
    }
  }
  for (int j0 = first; j0 < last; j0 += kRows * NB) {
    // the next rows load while these are worked on
    Batch<NB> next;
    load_rows<D, kWide>(next, src, a.src_head[KIND], j0 + kRows * NB, last, x.e0, x.e1, lane);
    uint2* const lo = r.lo;
    uint2* const hi = r.hi;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if (j0 + b * kRows >= last) break;  // (uniform in the warp)
      const int j = j0 + b * kRows + grp;
      float y[8];
      unpack8(make_uint4(lo[b].x, lo[b].y, hi[b].x, hi[b].y), y);
      if (KIND < 2) {
        float rms = 1.f;
        if (weight) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += y[e] * y[e];
#pragma unroll
          for (int off = kLanes / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          rms = rsqrtf(ss * (1.f / D) + a.eps);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float& yu = INTER ? y[2 * e] : y[e];
          float& yv = INTER ? y[2 * e + 1] : y[4 + e];
          const float u = yu * rms, v = yv * rms;
          yu = u * c0[e];
          yv = v * c1[e];
          if (x.turned) {  // (not by a zero sine: an infinite neighbour would spoil the element)
            yu -= v * s1[e];
            yv += u * s0[e];
          }
        }
        const uint4 bits = pack8(y);
        lo[b] = make_uint2(bits.x, bits.y);
        hi[b] = make_uint2(bits.z, bits.w);
      }
      float sc = 0.f;
      if constexpr (Q8 && KIND > 0) {
        float m = 0.f;  // (NaN from any of them stays, and the scale says so)
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(y[e]));
#pragma unroll
        for (int off = kLanes / 2; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off));
        sc = __fdiv_rn(m, 127.f);
      }
      if (j >= last) continue;
      if (KIND < 2 && a.out[KIND < 2 ? KIND : 0]) {
        __nv_bfloat16* to = a.out[KIND < 2 ? KIND : 0] + t * a.out_tok[KIND < 2 ? KIND : 0] +
                            j * a.out_head[KIND < 2 ? KIND : 0];
        if (kWide) {
          *reinterpret_cast<uint4*>(to + 8 * l) = make_uint4(lo[b].x, lo[b].y, hi[b].x, hi[b].y);
        } else {
          *reinterpret_cast<uint2*>(to + x.e0) = lo[b];
          *reinterpret_cast<uint2*>(to + x.e1) = hi[b];
        }
      }
      if (KIND == 0 || x.page < 0) continue;
      uint8_t* base = KIND == 1 ? a.pages.k : a.pages.v;
      const int64_t at = page_elem(a.pages, x.page, j, x.row);
      if constexpr (Q8) {
        uint32_t p0 = 0u, p1 = 0u;
        if (sc > 0.f) {
          const float rs = __frcp_rn(sc);
          p0 = pack4(code(y[0], sc, rs), code(y[1], sc, rs), code(y[2], sc, rs), code(y[3], sc, rs));
          p1 = pack4(code(y[4], sc, rs), code(y[5], sc, rs), code(y[6], sc, rs), code(y[7], sc, rs));
        }
        if (kWide) {
          *reinterpret_cast<uint2*>(base + at + 8 * l) = make_uint2(p0, p1);
        } else {
          *reinterpret_cast<uint32_t*>(base + at + x.e0) = p0;
          *reinterpret_cast<uint32_t*>(base + at + x.e1) = p1;
        }
      } else if (kWide) {
        *reinterpret_cast<uint4*>(base + 2 * (at + 8 * l)) = make_uint4(lo[b].x, lo[b].y, hi[b].x, hi[b].y);
      } else {
        *reinterpret_cast<uint2*>(base + 2 * (at + x.e0)) = lo[b];
        *reinterpret_cast<uint2*>(base + 2 * (at + x.e1)) = hi[b];
      }
      if (l == 0 && (KIND == 1 || Q8)) {
        const int64_t slot = page_slot(a.pages, x.page, j, x.row);
        if (Q8) (KIND == 1 ? a.pages.k_scale : a.pages.v_scale)[slot] = sc;
        if (KIND == 1 && a.pages.mass) a.pages.mass[slot] = 0.f;
        if (KIND == 1 && a.pages.order) a.pages.order[slot] = x.order;
      }
    }
    r = next;
  }
}

template <int D, bool Q8, bool INTER, int NB>
__global__ void __launch_bounds__(NB == 2 ? 32 : 128, NB == 2 ? kRotMany : kRotFew / 4)
    rotate_kernel(const __grid_constant__ RotArgs a) {
  constexpr int kLanes = D / 8;
  const int lane = threadIdx.x, l = lane % kLanes;
  const int64_t w = blockIdx.x;
  const int64_t t = w / a.shares;  // neighbouring warps share a token's heads
  pdl_wait();
  pdl_trigger();
  const int first = (int)(w % a.shares) * a.per, last = min(first + a.per, a.heads);
  const int q_end = min(last, a.h_q), k_end = min(last, a.h_q + a.h_kv);

  // ---- this lane's elements, and its first rows, which load while the rest is looked up
  Lane x;
  const int pairs = a.rot / 8;  // lanes whose elements turn
  x.turned = l < pairs;
  if (INTER) {
    x.e0 = 8 * l;
    x.e1 = 8 * l + 4;
  } else {
    x.e0 = x.turned ? 4 * l : 8 * l;
    x.e1 = x.turned ? a.rot / 2 + 4 * l : 8 * l + 4;
  }
  const int kind = first < a.h_q ? 0 : first < a.h_q + a.h_kv ? 1 : 2;
  const int kind0 = kind == 0 ? 0 : kind == 1 ? a.h_q : a.h_q + a.h_kv;
  Batch<NB> r;
  const __nv_bfloat16* from = a.src[kind] + t * a.src_tok[kind];
  const int from_end = (kind == 0 ? q_end : kind == 1 ? k_end : last) - kind0;
  if (INTER || kind == 2)
    load_rows<D, true>(r, from, a.src_head[kind], first - kind0, from_end, x.e0, x.e1, lane);
  else
    load_rows<D, false>(r, from, a.src_head[kind], first - kind0, from_end, x.e0, x.e1, lane);

  // ---- the token's positions, sequence, order and slot.  What is loaded here is used as late as
  // may be, the place in the cache behind the queries (15,541 tokens: 2.5 % longer with each lookup waited for)
  constexpr int kMine = 4 * kLanes / 32;
  const int grp = lane / kLanes;
  const bool turns = x.turned && first < a.h_q + a.h_kv;
  float2 turn_of[kMine];
  int pos[kMine];
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    const int i = 4 * l + grp * kMine + q;
    turn_of[q] = make_float2(0.f, 0.f);
    pos[q] = 0;
    if (turns) {
      turn_of[q] = a.turns[i];
      if (a.positions) {
        const int axis = a.axes == 1 ? 0 : i < a.sec0 ? 0 : i < a.sec0 + a.sec1 ? 1 : 2;
        pos[q] = a.positions[axis * a.num_tokens + t];
      }
    }
  }
  int s = 0, back = 0, len = 0;
  x.order = 0;
  if (a.cu_tokens) {
    if (w == 0 && lane == 0 && a.status && a.cu_tokens[a.num_seqs] > a.num_tokens)
      set_error(a.status, AIRCACHE_ERR_DEVICE_BOUNDS);  // tokens that the batch does not have
    s = find_seq(a.cu_tokens, a.num_seqs, (int)t, lane);
    if (s < 0 || s >= a.num_seqs) return;  // padding
    back = a.cu_tokens[s + 1] - (int)t;
    if (a.seen) x.order = a.seen[s] - back;
    if (a.has_pages) len = a.pages.lens[s];
  }

  // ---- its angles
  // the lanes of the warp's other rows need the same ones: each forms its share, and they are exchanged
  float sn[kMine], cs[kMine];
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    sn[q] = 0.f, cs[q] = 1.f;
    if (turns) turn(a.positions ? pos[q] : x.order, turn_of[q], sn[q], cs[q]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x.sn[e] = __shfl_sync(0xffffffffu, sn[e % kMine], (e / kMine) * kLanes + l);
    x.cs[e] = __shfl_sync(0xffffffffu, cs[e % kMine], (e / kMine) * kLanes + l);
  }
  x.page = -1;
  x.row = 0;
  const bool appends = a.has_pages && last > a.h_q;
  if (appends) {
    if (back >= 1 && len >= back && len <= a.pages.max_rows) {
      const int i = len - back;  // (formed only here: a length near int32's lowest would wrap to a row)
      const int nth = a.pages.max_rows < (1 << 24) ? page_of(a.pages, i, x.row) : i / a.pages.page_rows;
      x.row = i - nth * a.pages.page_rows;
      x.page = a.pages.table[s * a.pages.table_stride + nth];
    }
  }
  if (first < q_end) rows_of_token<D, Q8, INTER, 0>(a, x, t, first, q_end, lane, r);
  if (appends) {
    if (!page_ok(a.pages, x.page)) x.page = -1;
    if (x.page < 0 && lane == 0 && a.status) set_error(a.status, AIRCACHE_ERR_DEVICE_BOUNDS);
  }
  if (max(first, a.h_q) < k_end) {
    const int from = max(first, a.h_q) - a.h_q, to = k_end - a.h_q;
    if (kind < 1) load_rows<D, INTER>(r, a.src[1] + t * a.src_tok[1], a.src_head[1], from, to, x.e0, x.e1, lane);
    rows_of_token<D, Q8, INTER, 1>(a, x, t, from, to, lane, r);
  }
  if (max(first, a.h_q + a.h_kv) < last) {
    const int from = max(first, a.h_q + a.h_kv) - a.h_q - a.h_kv, to = last - a.h_q - a.h_kv;
    if (kind < 2) load_rows<D, true>(r, a.src[2] + t * a.src_tok[2], a.src_head[2], from, to, x.e0, x.e1, lane);
    rows_of_token<D, Q8, INTER, 2>(a, x, t, from, to, lane, r);
  }
}

template <int D>
auto rotate_pick(bool q8, bool inter, bool few) -> void (*)(RotArgs) {
  if (few)
    return q8 ? (inter ? rotate_kernel<D, true, true, 4> : rotate_kernel<D, true, false, 4>)
              : (inter ? rotate_kernel<D, false, true, 4> : rotate_kernel<D, false, false, 4>);
  return q8 ? (inter ? rotate_kernel<D, true, true, 2> : rotate_kernel<D, true, false, 2>)
            : (inter ? rotate_kernel<D, false, true, 2> : rotate_kernel<D, false, false, 2>);
}

}  // namespace
}  // namespace aircache

using namespace aircache;

extern "C" int aircache_rotate(const aircache_rotate_problem* p, int32_t* status, void* stream) {
  if (!p) return AIRCACHE_ERR_INVALID_ARG;
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  auto strides = [](int64_t tok, int64_t head) { return tok >= 0 && head >= 0 && tok % 8 == 0 && head % 8 == 0; };
  if (p->dtype != AIRCACHE_BF16 || (p->head_dim != 64 && p->head_dim != 128) || p->num_tokens < 0 ||
      p->num_tokens > 0x7fffffffLL || p->num_seqs < 0 || p->num_seqs > 65535 || p->reserved0 != 0 ||
      (p->interleaved & ~1) != 0 || !(p->eps >= 0.f) || (!p->q && !p->k) || (!p->q) != (!p->q_out) ||
      (p->q && p->h_q <= 0) || (p->k && p->h_kv <= 0) || p->h_q > 65535 || p->h_kv > 65535 ||
      (p->k && !p->k_out && !p->pages) || (!p->k && (p->k_out || p->pages)) || (!p->v) != (!p->pages))
    return AIRCACHE_ERR_INVALID_ARG;
  if (p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->rotary_dim % 16 != 0 || (p->rotary_dim && !p->turns) ||
      (p->axes != 1 && p->axes != 3) || (p->axes == 3 && (p->section0 < 0 || p->section1 < 0 ||
       (int64_t)p->section0 + p->section1 > p->rotary_dim / 2 || !p->positions)))
    return AIRCACHE_ERR_INVALID_ARG;
  auto al4 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 3) == 0; };
  if (!al4(p->positions) || !al4(p->cu_tokens) || !al4(p->seen) || !al4(status)) return AIRCACHE_ERR_INVALID_ARG;
  if (!al16(p->q) || !al16(p->k) || !al16(p->v) || !al16(p->q_out) || !al16(p->k_out) || !al16(p->q_weight) ||
      !al16(p->k_weight) || !al16(p->turns) || (p->q && !strides(p->q_stride_tok, p->q_stride_head)) ||
      (p->k && !strides(p->k_stride_tok, p->k_stride_head)) || (p->v && !strides(p->v_stride_tok, p->v_stride_head)) ||
      (p->q_out && !strides(p->qo_stride_tok, p->qo_stride_head)) ||
      (p->k_out && !strides(p->ko_stride_tok, p->ko_stride_head)))
    return AIRCACHE_ERR_INVALID_ARG;
  // rows of an output do not overlap: neither along a token's heads nor along the tokens, and where one axis does
  // not lie within the other's step, no head's row meets an earlier head's of another token
  auto apart = [&](int64_t tok, int64_t head, int heads) {
    const int64_t d = p->head_dim, tokens = p->num_tokens;
    if ((tokens > 1 && tok < d) || (heads > 1 && head < d)) return false;
    if (tokens <= 1 || heads <= 1 || head <= (tok - d) / (heads - 1) || tok <= (head - d) / (tokens - 1)) return true;
    for (int64_t h = 1; h < heads; ++h) {
      const int64_t t = h * head / tok, past = h * head % tok;
      if ((t < tokens && past < d) || (t + 1 < tokens && tok - past < d)) return false;
    }
    return true;
  };
  if ((p->q_out && !apart(p->qo_stride_tok, p->qo_stride_head, p->h_q)) ||
      (p->k_out && !apart(p->ko_stride_tok, p->ko_stride_head, p->h_kv)))
    return AIRCACHE_ERR_INVALID_ARG;
  // an output lies on no other input or output (k's and v's rows of the cache are outputs too)
  if ((p->q_out && (p->q_out == p->k || p->q_out == p->v || p->q_out == p->k_out)) ||
      (p->k_out && (p->k_out == p->q || p->k_out == p->v)) || (p->pages && p->pages->k == p->pages->v))
    return AIRCACHE_ERR_INVALID_ARG;
  // in place means the same rows, not shifted ones
  if ((p->q && p->q_out == p->q && (p->qo_stride_tok != p->q_stride_tok || p->qo_stride_head != p->q_stride_head)) ||
      (p->k_out && p->k_out == p->k &&
       (p->ko_stride_tok != p->k_stride_tok || p->ko_stride_head != p->k_stride_head)))
    return AIRCACHE_ERR_INVALID_ARG;
  RotArgs a = {};
  bool q8 = false;
  if (p->pages) {
    const int rc = check_pages(p->pages, a.pages);
    if (rc != AIRCACHE_OK) return rc;
    if (p->pages->num_seqs != p->num_seqs || p->pages->h_kv != p->h_kv || p->pages->head_dim != p->head_dim ||
        !p->cu_tokens || (p->pages->order && !p->seen))
      return AIRCACHE_ERR_INVALID_ARG;
    q8 = p->pages->kv_dtype == AIRCACHE_INT8;
  }
  if (p->rotary_dim && !p->positions && (!p->seen || !p->cu_tokens)) return AIRCACHE_ERR_INVALID_ARG;
  if (p->num_tokens == 0 || (p->cu_tokens && p->num_seqs == 0)) return AIRCACHE_OK;
  a.src[0] = static_cast<const __nv_bfloat16*>(p->q);
  a.src[1] = static_cast<const __nv_bfloat16*>(p->k);
  a.src[2] = static_cast<const __nv_bfloat16*>(p->v);
  a.src_tok[0] = p->q_stride_tok, a.src_head[0] = p->q_stride_head;
  a.src_tok[1] = p->k_stride_tok, a.src_head[1] = p->k_stride_head;
  a.src_tok[2] = p->v_stride_tok, a.src_head[2] = p->v_stride_head;
  a.out[0] = static_cast<__nv_bfloat16*>(p->q_out);
  a.out[1] = static_cast<__nv_bfloat16*>(p->k_out);
  a.out_tok[0] = p->qo_stride_tok, a.out_head[0] = p->qo_stride_head;
  a.out_tok[1] = p->ko_stride_tok, a.out_head[1] = p->ko_stride_head;
  a.weight[0] = static_cast<const __nv_bfloat16*>(p->q_weight);
  a.weight[1] = static_cast<const __nv_bfloat16*>(p->k_weight);
  a.turns = reinterpret_cast<const float2*>(p->turns);
  a.positions = p->positions;
  a.cu_tokens = p->cu_tokens;
  a.seen = p->seen;
  a.status = status;
  a.num_tokens = p->num_tokens;
  a.num_seqs = p->num_seqs;
  a.h_q = p->q ? p->h_q : 0;
  a.h_kv = p->k ? p->h_kv : 0;
  a.heads = a.h_q + a.h_kv + (p->pages ? a.h_kv : 0);
  a.rot = p->rotary_dim;
  a.axes = p->axes;
  a.sec0 = p->section0;
  a.sec1 = p->section1;
  a.has_pages = p->pages != nullptr;
  a.eps = p->eps;
  // How many warps share a token's heads.  A warp's time is about that of its rows' steps and three
  // more (the token's place and angles), the SMs hold kRotMany warps at once, and starting
  // them takes a step for every ten to an SM: a rough model, which need not find the best number.  (5,000
  // tokens of 32 + 32 heads of 64: 29 us with one warp to a token and 26 with the two that it gives, though
  // 24 with three; 3,000 of 32 + 32 heads of 128: 34, and 28 with its three; 200 of 28 + 4: 7.0, and 4.4
  // with its nine)
  const int sms = device_sms();
  const int at_once = p->head_dim == 128 ? 2 : 4;
  const int steps = (a.heads + at_once - 1) / at_once;
  const int64_t slots = (int64_t)kRotMany * sms;
  int64_t least = INT64_MAX;
  int best = p->num_tokens >= 8 * slots ? steps : 1;
  const bool ask = best == 1 && p->num_tokens * steps > 20LL * sms;  // (below, a step to a warp costs least)
  for (int i = 1; ask && i <= std::min(steps, 17); ++i) {
    const int n = i == 17 ? 1 : (steps + i - 1) / i;  // (16 shares at most, or a step to each)
    const int64_t warps = p->num_tokens * ((steps + n - 1) / n);
    const int64_t cost = 10LL * sms * ((warps + slots - 1) / slots) * (n + 3) + warps;
    if (cost < least) least = cost, best = n;
  }
  a.per = best * at_once;
  a.shares = (a.heads + a.per - 1) / a.per;
  const int64_t warps = p->num_tokens * a.shares;
  const bool few = a.shares == 1 && p->num_tokens <= (int64_t)kRotFew * sms;
  const dim3 grid((unsigned)warps), block(32);  // (many tokens have one share: 2^31 - 1 at most)
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  void (*kernel)(RotArgs) = p->head_dim == 128 ? rotate_pick<128>(q8, p->interleaved != 0, few)
                                               : rotate_pick<64>(q8, p->interleaved != 0, few);
  return launch_pdl(kernel, grid, block, 0, s, a) == cudaSuccess ? AIRCACHE_OK : AIRCACHE_ERR_CUDA;
}
