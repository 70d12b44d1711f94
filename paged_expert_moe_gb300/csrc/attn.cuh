// Shared by the attention kernels: their arguments, the partial results and the split rules.
#pragma once

#include "pmoe_internal.h"

namespace pmoe {
namespace attn {

constexpr int kMaxGroup = 64;  // query heads of a kv head

struct Args {
  pmoe_kv_desc kv;
  const __nv_bfloat16* q;
  int64_t q_stride;
  int T, q_heads, group;   // group = q_heads / kv_heads
  float scale;             // scores are in units of log 2: softmax scale * log2(e)
  const int32_t* prefix_pages;
  int prefix_len;
  const int32_t* page_table;
  int table_stride, sequences;
  const int32_t* row_seq;
  const int32_t* suffix_len;
  int max_suffix;
  __nv_bfloat16* out;
  float* lse;
  int32_t* err;
  // Partial results: part p of row-head i = t * q_heads + h. o: sum of weights x values
  // (not normalised), ml: (largest score, sum of weights). Parts 0 .. prefix_parts - 1 hold
  // the prefix, the next ceil(suffix_len / chunk) the suffix.
  float* o_part;    // [parts][T * q_heads][head_dim]
  float2* ml_part;  // [parts][T * q_heads]
  int prefix_parts, prefix_chunk;  // keys per prefix part (a multiple of 64)
  int suffix_parts, suffix_chunk;
  int row_tiles;    // row tiles of the prefix
};

__device__ __forceinline__ int suffix_keys(const Args& a, int t) {
  if (a.max_suffix == 0) return 0;
  const int n = a.suffix_len[t];
  if ((unsigned)n > (unsigned)a.max_suffix) {
    if (a.err != nullptr) atomicOr(a.err, kErrBadLength);
    return n < 0 ? 0 : a.max_suffix;
  }
  return n;
}

}  // namespace attn
}  // namespace pmoe
