// Shared by the kernels of moe_chunk_attention: arguments, the plan in scratch, what a row sees.
#pragma once

#include "attn_tc.cuh"

namespace pmoe {
namespace chunk {

using namespace attn;

// Empty units at the start of an item, for each kv head: what its start and end cost beside its tiles.
constexpr int kHead = 2;

// A tile of query rows: up to tile_tokens tokens of one request, times the query heads of a kv head.
struct Item {
  int32_t req;    // request
  int32_t tok0;   // its first token's row of q
  int32_t ntok;   // tokens
  int32_t p0;     // the first one's position
  int32_t nt;     // key tiles that some row sees: first the sinks' (below lo), then from lo on
  int32_t lo;
  int64_t base;   // units before it; its own: kHead + nt a kv head
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
  int ctas, tile_tokens, few_tokens, part_rows;
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

// One segment of a CTA's run: key tiles [t0, t1) of an item, for one kv head. Items of up to 128 rows
// take one query tile's warps and accumulators, in turn the first's and the second's (`lane`): one's
// end then overlaps with the other's beginning.
struct __align__(16) Segment {
  int32_t req, tok0, p0, lo;  // as the item's
  int32_t h, t0, t1;
  int32_t bits;               // tokens, and from bit 16 on: two query tiles, lane, all of the item's tiles
  __device__ __forceinline__ int ntok() const { return bits & 0xffff; }
  __device__ __forceinline__ bool two() const { return bits >> 16 & 1; }
  __device__ __forceinline__ int lane() const { return bits >> 17 & 1; }
  __device__ __forceinline__ bool whole() const { return bits >> 18 & 1; }
  __device__ __forceinline__ int p1() const { return p0 + ntok() - 1; }
  __device__ __forceinline__ bool has(int q) const { return two() || lane() == q; }
};
// The first key of tile t.
template <int KEYS>
__device__ __forceinline__ int tile_key(const Args& a, const Segment& s, int t) {
  const int st = a.window > 0 ? min((a.sinks + KEYS - 1) / KEYS, s.lo) : 0;
  return (t < st ? t : s.lo + t - st) * KEYS;
}
// A CTA's segments in order; the item after the present one is on its way.
struct Walk {
  int item, h, at;  // at: position in the item's units for this head, kHead empty ones first
  int64_t left;
  int lane;
  Item cur, ahead;
  __device__ __forceinline__ void begin(const Args& a, int cta) {
    const int64_t units = a.plan[0];
    const int ctas = (int)a.plan[1];
    left = 0;
    if (cta >= ctas) return;
    const int64_t u0 = run_start(units, ctas, cta);
    left = run_start(units, ctas, cta + 1) - u0;
    item = a.first[cta];
    cur = a.items[item];
    const int64_t in = u0 - cur.base;
    const int n = cur.nt + kHead;
    h = (int)(in / n);
    at = (int)(in - (int64_t)h * n);
    lane = 1;
    if (left > (int64_t)(a.kv.kv_heads - h) * n - at) ahead = a.items[item + 1];
  }
  __device__ __forceinline__ bool next(const Args& a, Segment* s) {
    while (left > 0) {
      const int n = cur.nt + kHead, to = (int)min((int64_t)n, at + left);
      s->req = cur.req, s->tok0 = cur.tok0, s->p0 = cur.p0, s->lo = cur.lo;
      s->h = h;
      s->t0 = max(at - kHead, 0);
      s->t1 = max(to - kHead, 0);
      const bool two = cur.ntok * a.group > 128, whole = s->t0 == 0 && s->t1 == cur.nt;
      if (!two && s->t1 > s->t0) lane ^= 1;
      s->bits = cur.ntok | (two ? 1 << 16 : 0) | lane << 17 | (whole ? 1 << 18 : 0);
      left -= to - at;
      at = to;
      if (at == n) {
        at = 0;
        if (++h == a.kv.kv_heads) {
          h = 0;
          ++item;
          if (left > 0) {
            cur = ahead;
            if (left > (int64_t)(cur.nt + kHead) * a.kv.kv_heads) ahead = a.items[item + 1];
          }
        }
      }
      if (s->t1 > s->t0) return true;  // (else only empty units of it are in this run)
    }
    return false;
  }
};

}  // namespace chunk
}  // namespace pmoe
