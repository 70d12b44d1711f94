// What a call of moe_prefix_attention does, worked out on the host alone. For the Python binding,
// which takes a call's scratch, and for the tests, which need to know the kernels that a size
// reaches; not part of the C ABI.
#pragma once

#include "../../include/pagedmoe.h"

typedef struct {
  uint64_t scratch_bytes;  // what this call needs
  uint64_t scratch_bound;  // what it and every smaller one need (moe_prefix_attention_scratch_bytes)
  int32_t cluster;         // CTAs of an item that a CTA or cluster takes whole; 0: parts, and their join
  int32_t tc_ctas;         // CTAs of the tensor-core prefix kernel, 0: it does not run
  int32_t prefix_parts, suffix_parts;  // at most, of a row-head
  int32_t join_warps;      // warps of a row-head in the joining kernel
} pmoe_attention_plan_desc;

#ifdef __cplusplus
extern "C"
#endif
    // sms: SMs of the device, 0: the current one's
    PMOE_API int
    pmoe_attention_plan(const pmoe_kv_desc* kv, int T, int q_heads, int prefix_len, int max_suffix, int sms,
                        pmoe_attention_plan_desc* out);
