// Attention of several query tokens over paged rows (paged_attend.cu), as the shared-prefix decode
// (shared_decode.cu) takes part in it.
#pragma once

#include <cuda_bf16.h>

#include "pages.cuh"

namespace aircache {

// Results kept in fp32 for a later join, of [token][query head]: the output [..][head_dim], and the log-sum-exp in
// base 2 (-inf: the token saw no row, and its output is 0).
// Their weights meet V in 16 bits, as those of the decode step that joins them.
struct AttendPart {
  float* out;
  float* lse2;
};

struct AttendPlan {
  Pages pages;
  bool q8;
  int d, g, h_q;
  int tok_tile;   // tokens of a stream's 128 query rows
  int slots;      // bound of the batch's units for one KV head
  int grid, rows_cap;
  size_t cut_off, start_off, range_off, ml_off, o_off, total;
};

// Checks a problem and lays out its workspace.  `part`: the results go to fp32 arrays and p->out is not looked at.
int attend_plan(const aircache_paged_attend_problem* p, bool part, AttendPlan& pl);
// Enqueues it; `ws` holds pl.total bytes, `error` the device error word.
int attend_launch(const aircache_paged_attend_problem* p, const AttendPlan& pl, const AttendPart& part, uint8_t* ws,
                  int32_t* error, cudaStream_t s);

// griddepcontrol.wait where a kernel has already begun to work: the kernel before has completed.
__device__ __forceinline__ void prior_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }

// A result over other rows that a decode step joins with its own: fp32 outputs [S][h_q][head_dim] and log-sum-exps in
// base 2 [S][h_q], of sequences *from .. *num - 1 (out == nullptr: of none).
struct DecodePrior {
  const float* out;
  const float* lse2;
  const int32_t *from, *num;  // device
};
// aircache_paged_decode, joined with a prior result; and the workspace it takes (AIRCACHE_OK, or why not).
int paged_decode_run(const aircache_paged_decode_problem* p, const DecodePrior& prior, void* ws, size_t ws_bytes,
                     void* stream);
int paged_decode_size(const aircache_paged_decode_problem* p, size_t& bytes);

}  // namespace aircache
