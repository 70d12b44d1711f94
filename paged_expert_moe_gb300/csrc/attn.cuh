// Shared by the attention kernels: their arguments, the partial results and the split rules.
#pragma once

#include "pmoe_internal.h"

#include <cuda_fp16.h>

namespace pmoe {
namespace attn {

constexpr int kMaxGroup = 64;  // query heads of a kv head

constexpr int kRowBlock = 2048;  // query rows whose suffixes one stream launch takes

struct Args {
  pmoe_kv_desc kv;
  const __nv_bfloat16* q;
  int64_t q_stride;
  int T, q_heads, group;   // group = q_heads / kv_heads
  uint32_t group_magic;    // 2^32 / group + 1
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
  // (not normalised), ml: (base of the weights' exponents, sum of weights). Parts 0 ..
  // prefix_parts - 1 hold the prefix, the others the suffix.
  float* o_part;    // [prefix_parts + suffix_parts][T * q_heads][head_dim]
  float2* ml_part;  // [prefix_parts + suffix_parts][T * q_heads]
  int prefix_parts, suffix_parts;  // at most
  // The tensor-core prefix kernel (tc_ctas > 0): units of one 128-key tile for one (256-row
  // tile, kv head) group, tc_tiles units to a group, in group order; CTA c takes units
  // [c * U / tc_ctas, (c + 1) * U / tc_ctas). A group's parts are numbered from its first CTA.
  int row_tiles, tc_ctas, tc_tiles;
  // The stream kernel: units of one 16-key tile for one (up to 16 query rows, kv head) item;
  // see prefix_attention.cu. pre_tiles: its tiles of the prefix (0: the tensor-core kernel's),
  // pre_items its items.
  int warps, min_share, pre_tiles, pre_items, head_items, whole;
  int64_t* base;    // [row blocks][kRowBlock + 1] first unit of each row; last: all units
};

constexpr int kTcRows = 256;  // query rows of a group
constexpr int kTcKeys = 128;  // keys of a tile

__host__ __device__ inline int64_t tc_units(const Args& a) { return (int64_t)a.row_tiles * a.kv.kv_heads * a.tc_tiles; }
// the CTA that takes unit u: the largest c with c * U / C <= u
__host__ __device__ inline int tc_cta_of(int64_t u, int64_t units, int ctas) { return (int)(((u + 1) * ctas - 1) / units); }
// prefix parts of query row r (of T * group) and kv head h
__host__ __device__ inline int tc_parts(const Args& a, int r, int h) {
  const int64_t units = tc_units(a), u = ((int64_t)(r / kTcRows) * a.kv.kv_heads + h) * a.tc_tiles;
  return tc_cta_of(u + a.tc_tiles - 1, units, a.tc_ctas) - tc_cta_of(u, units, a.tc_ctas) + 1;
}

double prefix_tc_cost(const Args& a, int ctas, int* used);
void plan_prefix_tc(Args* a, int ctas);
int launch_prefix_tc(const Args& a, cudaStream_t s);

constexpr float kLog2e = 1.44269504088896f, kLn2 = 0.693147180559945f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// two e4m3 codes (low 16 bits) -> fp16 pair, exact
__device__ __forceinline__ uint32_t e4m3x2(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((unsigned short)v));
  return r;
}
// The power of two a query row is divided by on its way to fp16: that of its largest
// element. What lies within 2^-14 of that one is exact. Zero, infinite and NaN rows: 2^0.
__device__ __forceinline__ int row_exponent(float largest) {
  const int e = (int)(__float_as_uint(largest) >> 23) - 127;
  return e < -126 || e > 127 ? 0 : min(e, 126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// r / group for r < 2^24 and group <= 64
__device__ __forceinline__ int row_token(const Args& a, int r) {
  return a.group == 1 ? r : (int)__umulhi((uint32_t)r, a.group_magic);
}

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
