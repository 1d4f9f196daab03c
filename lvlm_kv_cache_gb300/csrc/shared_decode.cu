// One decode step of a batch whose sequences share prefixes (aircache_shared_decode).
//
// Softmax over a prefix's rows and a sequence's own, put together from the two halves:
//   o = (2^{L_p} o_p + 2^{L_o} o_o) / (2^{L_p} + 2^{L_o}),  L = log2 sum 2^x.
// A prefix's rows are read once for all sequences that share it: their queries are the tokens of one attention
// without a mask over the prefix (paged_attend.cu; 128 query rows to a tile of keys, where the decode kernel reads
// every row again for each sequence), whose fp32 results the decode step over the own rows (paged_decode.cu) joins
// where it writes its outputs, log-sum-exps and mass.
//
// Bound by HBM in the decode step, by launches and the chain of loads between its three or four kernels in small
// calls.  The prefix is not left to run beside the own rows: with half of the SMs to each, 64 sequences took up to a
// fifth longer, as the decode step wants all of them.  Its kernels start early instead (programmatic launch), and only
// its joins wait.
//
// The weights of a prefix's rows hold 16 bits, as the decode step's own (a sum of two bf16; one alone would take 17, 61 and
// 76 us below, and leave outputs 0.0019 to 0.0025 of their norm from a form that holds 24 bits instead of 0.0002).
//
// Measured (28 query and 4 KV heads of 128, bf16, calls back to back): 8 sequences with up to 64 own rows behind one
// prefix of 2,048 18 us; 64 with 100 to 2,000 behind one of 16,384 64 us (163 MB, 24 us at the copy
// rate); 24 with up to 256 behind one of 131,072 (275 MB, 41 us) 87 us.
#include "attend.cuh"

namespace aircache {
namespace {

struct SdPlan {
  aircache_paged_attend_problem at;
  AttendPlan attend;
  size_t attend_off, out_off, lse_off, total;
};

inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Whether an output lies on another, or on what the step reads.  (mass_out may be the own rows' mass, and lie on the
// prefixes', which may be of the same pool: they are neither read nor written.)
bool outputs_meet(const aircache_shared_decode_problem* p) {
  const aircache_paged_decode_problem& o = p->own;
  Pages own, prefix;
  const bool shared = p->prefix->num_seqs > 0 && check_pages(p->prefix, prefix) == AIRCACHE_OK;
  if (check_pages(o.pages, own) != AIRCACHE_OK || own.num_seqs == 0) return false;
  const int64_t S = own.num_seqs, H = o.h_q, d = o.pages->head_dim;
  const struct {
    const void* at;
    size_t bytes;
  } outs[3] = {{o.out, span_bytes(o.out, {{S, H * d}}, H * d, 2)},
               {o.lse, span_bytes(o.lse, {{S, H}}, H, 4)},
               {o.mass_out, o.mass_out ? slot_bytes(own) : 0}};
  const size_t nq = span_bytes(o.q, {{S, o.q_stride_seq}, {H, o.q_stride_head}}, d, 2);
  for (int i = 0; i < 3; ++i) {
    const void* x = outs[i].at;
    const size_t n = outs[i].bytes;
    if (!x) continue;
    for (int j = 0; j < i; ++j)
      if (arrays_meet(x, n, outs[j].at, outs[j].bytes)) return true;
    if (arrays_meet(x, n, o.q, nq) || meets_cache(o.pages, own, x, n) ||
        (shared && (meets_cache(p->prefix, prefix, x, n) ||
                    arrays_meet(x, n, p->cu_seqs, 4 * ((size_t)prefix.num_seqs + 1)))) ||
        (i < 2 && o.mass_out && arrays_meet(x, n, own.mass, slot_bytes(own))))
      return true;
  }
  return false;
}

int sd_plan(const aircache_shared_decode_problem* p, SdPlan& pl) {
  if (!p || !p->prefix) return AIRCACHE_ERR_INVALID_ARG;
  size_t own = 0;
  int rc = paged_decode_size(&p->own, own);
  if (rc != AIRCACHE_OK) return rc;
  const aircache_pages* o = p->own.pages;
  if (p->prefix->h_kv != o->h_kv || p->prefix->head_dim != o->head_dim) return AIRCACHE_ERR_INVALID_ARG;
  pl.attend_off = up256(own);
  pl.total = pl.attend_off;
  if (outputs_meet(p)) return AIRCACHE_ERR_INVALID_ARG;
  if (p->prefix->num_seqs == 0) return AIRCACHE_OK;  // (its arrays have no elements, and need no address)
  pl.at = aircache_paged_attend_problem{};
  pl.at.pages = p->prefix;
  pl.at.num_tokens = o->num_seqs;
  pl.at.h_q = p->own.h_q;
  pl.at.dtype = p->own.dtype;
  pl.at.scale = p->own.scale;
  pl.at.cu_tokens = p->cu_seqs;
  pl.at.q = p->own.q;
  pl.at.q_stride_tok = p->own.q_stride_seq;
  pl.at.q_stride_head = p->own.q_stride_head;
  rc = attend_plan(&pl.at, true, pl.attend);
  if (rc != AIRCACHE_OK) return rc;
  const size_t heads = (size_t)o->num_seqs * p->own.h_q;
  pl.out_off = pl.attend_off + pl.attend.total;
  pl.lse_off = pl.out_off + up256(sizeof(float) * heads * o->head_dim);
  pl.total = pl.lse_off + up256(sizeof(float) * heads);
  return AIRCACHE_OK;
}

}  // namespace
}  // namespace aircache

using namespace aircache;

extern "C" {

size_t aircache_shared_decode_workspace_size(const aircache_shared_decode_problem* p) {
  SdPlan pl;
  return sd_plan(p, pl) == AIRCACHE_OK ? pl.total : 0;
}

int aircache_shared_decode(const aircache_shared_decode_problem* p, void* ws, size_t ws_bytes, void* stream) {
  SdPlan pl;
  int rc = sd_plan(p, pl);
  if (rc != AIRCACHE_OK) return rc;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) != 0) return AIRCACHE_ERR_INVALID_ARG;
  if (ws_bytes < pl.total) return AIRCACHE_ERR_WORKSPACE;
  if (p->own.pages->num_seqs == 0) return AIRCACHE_OK;
  uint8_t* w = static_cast<uint8_t*>(ws);
  DecodePrior prior = {nullptr, nullptr, nullptr, nullptr};
  if (p->prefix->num_seqs > 0) {
    const AttendPart part = {reinterpret_cast<float*>(w + pl.out_off), reinterpret_cast<float*>(w + pl.lse_off)};
    rc = attend_launch(&pl.at, pl.attend, part, w + pl.attend_off, reinterpret_cast<int32_t*>(w),
                       static_cast<cudaStream_t>(stream));
    if (rc != AIRCACHE_OK) return rc;
    prior = {part.out, part.lse2, p->cu_seqs, p->cu_seqs + p->prefix->num_seqs};
  }
  return paged_decode_run(&p->own, prior, ws, pl.attend_off, stream);
}

}  // extern "C"
