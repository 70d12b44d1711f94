// moe_chunk_attention: its arguments, what a row sees, and a CTA's share of the work.
#pragma once

#include "attn_tc.cuh"
#include "runs.h"

namespace pmoe {
namespace chunk {

using namespace attn;

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
  int ctas, tile_tokens, few_tokens, part_rows, few;
  // Empty units at the start of an item, for each kv head: what its start and end cost beside its tiles.
  int head;
  // scratch
  // Parts of items that a CTA does not take whole: slot 0 where it continues one, slot 1 where it
  // begins one. o: sum of weights x values, ml: (base of the weights' exponents, sum of weights).
  float* o_part;    // [ctas][2][part_rows][head_dim]
  float2* ml_part;  // [ctas][2][part_rows]
  uint32_t* done;   // [ctas][2] parts written of the item that begins in a CTA and ends in another, by query tile
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

// r / group for r < 2^24 and group <= 64
__device__ __forceinline__ int row_token(const Args& a, int r) {
  return a.group == 1 ? r : (int)__umulhi((uint32_t)r, a.group_magic);
}

// Cutting an item costs a part and a join, some four tiles of few rows and more of many. So where runs are
// short a run's boundary moves to the start or the end of its item, whichever is nearer, if the item is
// short too, and else if it lies within `slack` tiles of it. Measured with 14 / 0 tiles as short for more than 32
// rows: prompts of 512 tokens 17.8 / 29.6 us, 1,024 24.7 / 48, 1,600 41 / 49, 4 of 1,000 55 / 69, 400 on 900 keys 28.6 / 36
// (16: 2,048 tokens, heads of 64, 53 / 47); with 6 / 0 for few: one token on 500 keys 14.2 / 16.8, 16 on 600 17.3 / 20.6. In runs of
// 50 units slack of 2 costs more unevenness than it saves (61 tokens and 3 pieces of 1,500 243 / 223), and for few
// rows it never pays (4 tokens on 2,000 keys with 0, 1, 2 18.6, 19.4, 20.9).
__device__ __forceinline__ bool short_run(int64_t units, int ctas, int limit) { return units < (int64_t)limit * ctas; }
__device__ __forceinline__ int slack(const Args& a, int64_t units, int ctas, int ntok) {
  return ntok * a.group > 32 && short_run(units, ctas, 12) ? 2 : 0;
}
__device__ __forceinline__ bool never_cut(const Args& a, int64_t units, int ctas, int tiles, int ntok) {
  return ntok * a.group > 32 ? tiles <= 14 && short_run(units, ctas, 48) : tiles <= 6 && short_run(units, ctas, 12);
}
// Where a boundary at unit `at` of an item's n goes.
__device__ __forceinline__ int moved(const Args& a, int64_t units, int ctas, int at, int n, int ntok) {
  const int behind = max(at - a.head, 0), ahead = n - at;
  if (min(behind, ahead) > slack(a, units, ctas, ntok) && !never_cut(a, units, ctas, n - a.head, ntok)) return at;
  return behind <= ahead ? 0 : n;
}

// A request's rows of this step.
struct Request {
  int start, n, len;
  bool bad;
};
// `r`'s, before what the rows of the ones ahead of it leave of T.
__device__ __forceinline__ Request request(const Args& a, int r) {
  Request q{0, 0, 0, false};
  if (r >= a.R) return q;
  const int s0 = a.q_start[r], s1 = a.q_start[r + 1], len = a.kv_len[r];
  q.start = min(max(s0, 0), a.T);
  const int end = min(max(s1, 0), a.T);
  q.n = max(end - q.start, 0);
  const int64_t room = (int64_t)a.table_stride * a.kv.page_size;
  q.len = (int)min((int64_t)max(len, 0), room);
  q.bad = s0 != q.start || s1 != end || end < q.start || len != q.len;
  return q;
}

// A tile of query rows (an item): up to tile_tokens tokens of one request, times the query heads of
// a kv head. lo: the first of its key tiles beside the sinks'. Returns how many it has.
__device__ __forceinline__ int key_tiles(const Args& a, int p0, int ntok, int* lo) {
  const int p1 = p0 + ntok - 1;
  *lo = a.window > 0 ? max(p0 - a.window + 1, 0) / kTcKeys : 0;
  if (p1 < 0) return 1;  // rows before the first key: a tile of which they see nothing
  const int st = a.window > 0 ? min((a.sinks + kTcKeys - 1) / kTcKeys, *lo) : 0;
  return p1 / kTcKeys + 1 - *lo + st;
}

// One segment of a CTA's run: key tiles [t0, t1) of an item, for one kv head. Items of up to 128 rows
// take one query tile's warps and accumulators, in turn the first's and the second's (`lane`): one's
// end then overlaps with the other's beginning.
struct __align__(16) Segment {
  int32_t req, tok0, p0, lo;  // request, first row of q, its position, first key tile beside the sinks'
  int32_t t0, t1;
  int32_t join;  // of a part: the CTA with the item's first tile, and from bit 16 on the number of parts
  int32_t bits;  // tokens, and from bit 10 on: two query tiles, lane, all of the item's tiles; 13: kv head
  int32_t part0, part1, part2;  // tiles that some row does not see in full: [part0, part1), and from part2 on
  int32_t pad;
  __device__ __forceinline__ int ntok() const { return bits & 1023; }
  __device__ __forceinline__ bool two() const { return bits >> 10 & 1; }
  __device__ __forceinline__ int lane() const { return bits >> 11 & 1; }
  __device__ __forceinline__ bool whole() const { return bits >> 12 & 1; }
  __device__ __forceinline__ int h() const { return bits >> 13; }
  __device__ __forceinline__ int p1() const { return p0 + ntok() - 1; }
  __device__ __forceinline__ bool has(int q) const { return two() || lane() == q; }
  // Whose scores' place tile t of a segment of one query tile takes: in turn both query tiles', its own last.
  __device__ __forceinline__ int place(int t) const { return ((t1 - 1 - t) & 1) ^ lane(); }
  __device__ __forceinline__ bool partly(int t) const { return t >= part2 || (t >= part0 && t < part1); }
};
// The first key of tile t.
template <int KEYS>
__device__ __forceinline__ int tile_key(const Args& a, const Segment& s, int t) {
  const int st = a.window > 0 ? min((a.sinks + KEYS - 1) / KEYS, s.lo) : 0;
  return (t < st ? t : s.lo + t - st) * KEYS;
}

// Where a CTA's run of units begins and ends. An item has a.head + its key tiles units a kv head, items
// come request by request; runs are equal but for boundaries that move (above).
struct Run {
  // all units, the run's, its first one, the one behind its last; rows of the requests up to its first
  int64_t units, left, u, end, before;
  int ctas, req, tile, h, at;      // request, tile of its rows, kv head, unit of the item
  int start, n, len;               // of the request
};

// Of a partly visible tile from key k0 on: keys that some row sees lie in [first, end), by steps of
// 16 (the K of an MMA), and of these all rows see those in [low, high), but for sinks.
struct Span {
  int first, end, low, high;
};
template <int KEYS>
__device__ __forceinline__ Span seen_span(const Args& a, const Segment& s, int k0) {
  Span p{0, 0, 0, 0};
  const int p1 = s.p1();
  if (a.window > 0 && a.sinks <= k0) p.first = min(max(s.p0 - a.window + 1 - k0, 0), KEYS - 1) & ~15;
  p.end = min((max(p1 - k0 + 1, 1) + 15) & ~15, KEYS);
  if (p.end <= p.first) p.end = p.first + 16;  // (no row sees a key: one step of zeros all the same)
  p.low = a.window > 0 ? min(max(p1 - a.window + 1 - k0, p.first), p.end) : p.first;
  p.high = min(max(s.p0 + 1 - k0, p.low), p.end);
  return p;
}

// Which tiles are partly visible: a tile from key k0 on is seen by all rows if its last key is by the
// first row (k0 + KEYS - 1 <= p0), and with a window if its first key is by the last row (k0 > p1 -
// window) or all of it is sinks. (Where sinks reach into the window's own tiles some of these count as
// partly visible although all rows see them.)
template <int KEYS>
__device__ __forceinline__ void mark_parts(const Args& a, Segment* s) {
  const int st = a.window > 0 ? min((a.sinks + KEYS - 1) / KEYS, s->lo) : 0, p1 = s->p1();
  const int full = max(s->p0 + 1, 0) / KEYS;  // key tiles that the first row is past
  s->part0 = s->part1 = 0;
  if (a.window > 0) {
    s->part0 = min(a.sinks / KEYS, st);
    s->part1 = st + max((max(p1 - a.window + 1, 0) + KEYS - 1) / KEYS - s->lo, 0);
  }
  s->part2 = full > s->lo ? st + full - s->lo : min(full, st);
}

// A CTA's segments in order, by a whole warp.
struct Walk {
  Run run;
  int64_t first;  // unit of the item's first tile, for this head
  int lane, p0, ntok, tok0, nt, lo;
  int batch;      // the requests from this one on, one a lane, once the first request is through
  Request mine;
  uint32_t some;  // lanes whose requests have rows and are still to come

  __device__ __forceinline__ void load(const Args& a) {
    const int l = threadIdx.x & 31;
    mine = request(a, batch + l);
    int64_t upto = mine.n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t d = __shfl_up_sync(0xffffffffu, upto, o);
      if (l >= o) upto += d;
    }
    if (run.before + upto > a.T) mine.n = 0;
    run.before += __shfl_sync(0xffffffffu, upto, 31);
    some = __ballot_sync(0xffffffffu, mine.n > 0);
  }
  __device__ __forceinline__ void item(const Args& a) {
    const int i0 = run.tile * a.tile_tokens;
    tok0 = run.start + i0;
    ntok = min(a.tile_tokens, run.n - i0);
    p0 = run.len - run.n + i0;
    nt = key_tiles(a, p0, ntok, &lo);
  }
  // The next request with rows; false: there is none.
  __device__ __forceinline__ bool request_after(const Args& a) {
    while (some == 0) {
      if (batch + 32 >= a.R) return false;
      batch += 32;
      load(a);
    }
    const int k = __ffs(some) - 1;
    some &= some - 1;
    run.req = batch + k;
    run.start = __shfl_sync(0xffffffffu, mine.start, k);
    run.n = __shfl_sync(0xffffffffu, mine.n, k);
    run.len = __shfl_sync(0xffffffffu, mine.len, k);
    return true;
  }
  __device__ __forceinline__ void begin(const Args& a, const Run& r) {
    run = r;
    run.left = run.end - run.u;
    if (run.left <= 0) return;
    lane = 1;
    batch = run.req + 1 - 32;
    some = 0;
    item(a);
    first = run.u - run.at + a.head;
  }
  __device__ __forceinline__ bool next(const Args& a, Segment* s) {
    while (run.left > 0) {
      const int n = nt + a.head, to = (int)min((int64_t)n, run.at + run.left);
      s->req = run.req, s->tok0 = tok0, s->p0 = p0, s->lo = lo;
      s->t0 = max(run.at - a.head, 0);
      s->t1 = max(to - a.head, 0);
      const bool two = ntok * a.group > 128, whole = s->t0 == 0 && s->t1 == nt;
      if (!two && s->t1 > s->t0) lane ^= 1;
      s->bits = ntok | (two ? 1 << 10 : 0) | lane << 11 | (whole ? 1 << 12 : 0) | run.h << 13;
      s->join = 0;
      if (!whole) {
        const int k = slack(a, run.units, run.ctas, ntok), c0 = cta_of(run.units, run.ctas, first + k);
        s->join = c0 | (cta_of(run.units, run.ctas, first + nt - 1 - k) - c0 + 1) << 16;
      }
      run.left -= to - run.at;
      run.at = to;
      if (to == n && run.left > 0) {
        run.at = 0;
        first += n;
        if (++run.h == a.kv.kv_heads) {
          run.h = 0;
          ++run.tile;
          if (run.tile * a.tile_tokens >= run.n) {
            run.tile = 0;
            // (some units are left, so some request has rows; if its numbers are still the same)
            if (!request_after(a)) run.left = 0;
          }
          item(a);
        }
      }
      mark_parts<kTcKeys>(a, s);
      if (s->t1 > s->t0) return true;  // (else only empty units of it are in this run)
    }
    return false;
  }
};

}  // namespace chunk
}  // namespace pmoe
