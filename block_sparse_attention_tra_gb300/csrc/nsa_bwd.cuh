// nsa_bwd.cuh -- what the two translation units of the NSA selection
// attention's backward share (nsa_bwd.cu: lists and the general kernels;
// nsa_bwd_tc.cu: the tcgen05 pass).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace bsa {

constexpr float NSA_LOG2E = 1.4426950408889634f;

struct NsaBwdArgs {
  const __nv_bfloat16 *q, *k, *v, *out, *dout;
  const int32_t* idx;
  const float* lse;
  __nv_bfloat16 *dq, *dk, *dv;
  int B, Hq, Hkv, T, bs, S;
};

// Pieces of the workspace.  list: the queries of every block, ascending, as
// i * 32 + slot; items: {block, first list entry, queries, items of its
// block}; part: fp32 dk, dv of each item of a block with several; dq_part,
// dq_scale (tcgen05 pass): f16 dQ rows [slot of the index tensor][head][D] and
// their factors, one row a slot; for blocks of 128 tokens two a slot, one for
// each half of its block: [slot][half][head][D].
struct NsaBwdScratch {
  float2* stats;
  int* list;
  int4* items;
  const int* n_items;
  float* part;
  __nv_bfloat16* rows;
  __half* dq_part;
  float* dq_scale;
  long long max_items;
};

int launch_nsa_bwd_tc(const NsaBwdArgs& a, const NsaBwdScratch& w, int D, cudaStream_t stream);

}  // namespace bsa
