// The paged cache as the kernels of rotate.cu, paged_decode.cu and evict.cu see
// it, and the host checks they share.
#pragma once

#include <cuda_bf16.h>

#include "internal.cuh"
#include "ptx.cuh"

namespace aircache {

// Device-visible description of one layer's pages (host checks done).
struct Pages {
  uint8_t* k;
  uint8_t* v;
  int64_t stride_page, stride_row, stride_head;  // elements
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  float* k_scale;
  float* v_scale;
  float* mass;
  int32_t* order;
  int64_t num_pages;
  int num_seqs, h_kv, page_rows, max_rows;  // max_rows: the table's capacity of one sequence
  uint32_t page_inv;                        // 2^32 / (page_rows / 16), rounded up (0: page_rows is 16)
};

// row / page_rows and row % page_rows for rows below 2^24: pages hold d = page_rows / 16
// pieces of 16 rows, and piece * page_inv / 2^32 is off by less than 1 / d, since piece * d < 2^32.
__device__ __forceinline__ int page_of(const Pages& p, int row, int& in_page) {
  const uint32_t piece = (uint32_t)row >> 4;
  const int page = (int)(p.page_inv ? __umulhi(piece, p.page_inv) : piece);
  in_page = row - page * p.page_rows;
  return page;
}

// The slot of (page, row) of KV head h in the scale, mass and order arrays.
__device__ __forceinline__ int64_t page_slot(const Pages& p, int page, int h, int row) {
  return ((int64_t)page * p.h_kv + h) * p.page_rows + row;
}
// Element offset of (page, row) of KV head h in k and v.
__device__ __forceinline__ int64_t page_elem(const Pages& p, int page, int h, int row) {
  return (int64_t)page * p.stride_page + (int64_t)row * p.stride_row + (int64_t)h * p.stride_head;
}
__device__ __forceinline__ bool page_ok(const Pages& p, int page) { return page >= 0 && page < p.num_pages; }

// Host: AIRCACHE_OK and the device description, or why not.
inline int check_pages(const aircache_pages* p, Pages& d) {
  if (!p || p->num_seqs < 0 || p->num_seqs > 65535 || p->h_kv <= 0 || p->h_kv > 65535 ||
      (p->head_dim != 64 && p->head_dim != 128) || (p->kv_dtype != AIRCACHE_BF16 && p->kv_dtype != AIRCACHE_INT8) ||
      p->page_rows < 16 || p->page_rows > 4096 || p->page_rows % 16 != 0 || p->max_pages < 1 ||
      (int64_t)p->max_pages * p->page_rows > 0x7fff0000LL || p->num_pages < 1 || p->num_pages > 0x7fffffffLL ||
      p->table_stride < p->max_pages || !p->k || !p->v || !p->table || !p->lens)
    return AIRCACHE_ERR_INVALID_ARG;
  const bool q8 = p->kv_dtype == AIRCACHE_INT8;
  const int64_t unit = q8 ? 16 : 8;
  // scales, mass and order are read in pieces of 4 and 16 values: they start on 16 bytes too
  auto al16 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15) == 0; };
  if (!al16(p->k) || !al16(p->v) || p->stride_page <= 0 || p->stride_row <= 0 || p->stride_head <= 0 ||
      p->stride_page % unit != 0 || p->stride_row % unit != 0 || p->stride_head % unit != 0 ||
      (q8 && (!p->k_scale || !p->v_scale || !al16(p->k_scale) || !al16(p->v_scale))))
    return AIRCACHE_ERR_INVALID_ARG;
  auto al4 = [](const void* x) { return (reinterpret_cast<uintptr_t>(x) & 3) == 0; };
  if (!al4(p->table) || !al4(p->lens) || !al16(p->mass) || !al16(p->order)) return AIRCACHE_ERR_INVALID_ARG;
  d.k = static_cast<uint8_t*>(p->k);
  d.v = static_cast<uint8_t*>(p->v);
  d.stride_page = p->stride_page;
  d.stride_row = p->stride_row;
  d.stride_head = p->stride_head;
  d.table = p->table;
  d.table_stride = p->table_stride;
  d.lens = p->lens;
  d.k_scale = q8 ? p->k_scale : nullptr;
  d.v_scale = q8 ? p->v_scale : nullptr;
  d.mass = p->mass;
  d.order = p->order;
  d.num_pages = p->num_pages;
  d.num_seqs = p->num_seqs;
  d.h_kv = p->h_kv;
  d.page_rows = p->page_rows;
  d.max_rows = p->max_pages * p->page_rows;
  const uint64_t pieces = p->page_rows / 16;
  d.page_inv = pieces == 1 ? 0u : (uint32_t)(((1ull << 32) + pieces - 1) / pieces);
  return AIRCACHE_OK;
}

// Host: whether two arrays of `bytes` and `other` bytes share any.
inline bool arrays_meet(const void* x, size_t bytes, const void* y, size_t other) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
  return x && y && a < b + other && b < a + bytes;
}
// Host: the bytes of an array of the mass's and the order's shape.
inline size_t slot_bytes(const Pages& p) { return 4 * (size_t)p.num_pages * p.h_kv * p.page_rows; }

}  // namespace aircache
