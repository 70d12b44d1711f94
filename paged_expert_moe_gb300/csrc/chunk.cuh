// Shared by the kernels of moe_chunk_attention: arguments, the plan in scratch, what a row sees.
#pragma once

#include "attn_tc.cuh"

namespace pmoe {
namespace chunk {

using namespace attn;

// A tile of query rows: up to tile_tokens tokens of one request, times the query heads of a kv head.
struct Item {
  int32_t req;    // request
  int32_t tok0;   // its first token's row of q
  int32_t ntok;   // tokens
  int32_t p0;     // the first one's position
  int32_t nt;     // key tiles that some row sees: first the sinks' (below lo), then from lo on
  int32_t lo;
  int64_t base;   // units before it; its own: nt a kv head
};

struct Args {
  pmoe_kv_desc kv;
  const __nv_bfloat16* q;
  int64_t q_stride;
  int T, q_heads, group, R;
  uint32_t group_magic;  // 2^32 / group + 1
  float scale;           // scores are in units of log 2: softmax scale * log2(e)
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  int table_stride;
  int window, sinks;     // window 0: none
  __nv_bfloat16* out;
  float* lse;
  int32_t* err;
  int ctas, tile_tokens, part_rows;
  // scratch
  int64_t* plan;   // [2]: units, CTAs that have some
  int32_t* first;  // [ctas] the item of each CTA's first unit
  Item* items;
  // Parts of items that a CTA does not take whole: slot 0 where it continues one, slot 1 where it
  // begins one. o: sum of weights x values, ml: (base of the weights' exponents, sum of weights).
  float* o_part;    // [ctas][2][part_rows][head_dim]
  float2* ml_part;  // [ctas][2][part_rows]
};

// Visible keys of a row at position p: j <= p, and with a window j > p - window or j < sinks.
__device__ __forceinline__ bool sees(const Args& a, int p, int j) {
  return j <= p && (a.window == 0 || j > p - a.window || j < a.sinks);
}
// Of the rows at p0..p1: whether any sees key j, and whether all do.
__device__ __forceinline__ bool any_sees(const Args& a, int p0, int p1, int j) {
  return j <= p1 && (a.window == 0 || j > p0 - a.window || j < a.sinks);
}
__device__ __forceinline__ bool all_see(const Args& a, int p0, int p1, int j) {
  return j <= p0 && (a.window == 0 || j > p1 - a.window || j < a.sinks);
}
// whether all see the n keys from k0 on
__device__ __forceinline__ bool all_see_tile(const Args& a, int p0, int p1, int k0, int n) {
  return k0 + n - 1 <= p0 && (a.window == 0 || k0 > p1 - a.window || k0 + n <= a.sinks);
}

__device__ __forceinline__ int64_t run_start(int64_t units, int ctas, int c) { return units * c / ctas; }

// r / group for r < 2^24 and group <= 64
__device__ __forceinline__ int row_token(const Args& a, int r) {
  return a.group == 1 ? r : (int)__umulhi((uint32_t)r, a.group_magic);
}

// One segment of a CTA's run: key tiles [t0, t1) of an item's nt, for one kv head.
struct Segment {
  Item it;
  int h, t0, t1;
  __device__ __forceinline__ int p1() const { return it.p0 + it.ntok - 1; }
  __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == it.nt; }
};
// The first key of tile t of an item.
template <int KEYS>
__device__ __forceinline__ int tile_key(const Args& a, const Item& it, int t) {
  const int st = a.window > 0 ? min((a.sinks + KEYS - 1) / KEYS, it.lo) : 0;
  return (t < st ? t : it.lo + t - st) * KEYS;
}
struct Walk {
  int item, h, t;
  int64_t left;
  __device__ __forceinline__ bool next(const Args& a, Segment* s) {
    if (left <= 0) return false;
    s->it = a.items[item];
    s->h = h;
    s->t0 = t;
    s->t1 = (int)min((int64_t)s->it.nt, t + left);
    left -= s->t1 - t;
    t = s->t1;
    if (t == s->it.nt) {
      t = 0;
      if (++h == a.kv.kv_heads) h = 0, ++item;
    }
    return true;
  }
};

}  // namespace chunk
}  // namespace pmoe
