// moe_chunk_attention: each request's new tokens over its own pages of a paged cache, with causal
// limits and, where asked for, a sliding window and first keys that stay visible.
//
// A tile of query rows is up to 256 / group tokens of one request times the query heads of one kv
// head, so that all its rows meet the same keys: S = Q K^T and O += P V on the tensor cores, 128
// keys at a time, as two 128-row query tiles that share each K and V tile. Rows of a tile differ in
// what they see only in its last key tiles and at a window's edge; all others take no masks.
//
// Work: the lengths are on the device, so each CTA adds up the key tiles that all tiles of rows need
// and takes its share, one of (nearly) equal runs, one CTA an SM. What a run has of a tile of rows without having
// all of it is left as a part in scratch; whoever writes the last part of a tile joins them, in order.
//
// Warps: 0-3 and 4-7 own one query tile each, a thread one row (a TMEM lane): scores from TMEM,
// weights back to TMEM in their place as the 16-bit A operand of the second product. Warp 8 issues
// the MMAs, warp 9 works out the CTA's segments for all and loads K and V tiles by TMA, one box a page
// and 64 columns, warp 10 loads q. In partly visible tiles a value that some row must not use may be
// anything, and 0 x NaN is NaN: with a bf16 cache warps 10 and 11 look at those tiles before the MMAs
// do, clear the rows that no query row sees and what is not finite in the others; with an e4m3 cache
// warps 12-15, which convert keys, values and q to fp16, do. What was cleared is added to the rows that
// do see it at the end.
//
// Bounds, and what it measures (heads 32 / 4 x 128, bf16, a GPU of 152 SMs; in a loop, pages of 64, but where said).
// Prompts: the tensor cores. 8,192 tokens 380 us (1,450 TFLOP/s; 1,920 is what a library product reaches), in pages of
// 16 404, and 418-425 with cold caches; 4,096 tokens on 60,001 keys 2.5-2.7 ms by power (1,530-1,650), cold 2.8-2.9. The
// issuing warp is what they wait for: it sees keys, values and weights in one look, and its inner loop holds nothing but tiles that
// all rows see. Many single tokens: HBM; 64 on up to 16,000 keys 172 us (6.0 TB/s), 256 with a window of 4,096 314 us
// (6.1 TB/s). Single tokens with an 8-bit cache or heads of 64: the chain of a tile (scores, softmax, products), as one CTA
// an SM has one such item at a time; 64 with e4m3 187 us, with heads of 64 and 40 / 8 of them 204 us (5.1 TB/s), with both
// 267 us. Few calls' worth of work: start and end, 18 us for four tokens on up to 2,000 keys. A negative scale (or key
// scale) takes every tile through the masks' pass in TMEM: a prompt of 8,192 tokens 516 us, with e4m3 626 (465), 64 single tokens 217.
// Sixteen bits for the weights, as the second product takes them: at most half a unit of bf16's or fp16's last
// place each, or with fp16 2^-32 of the row's largest, while their sum and the products' stay fp32.
#include "chunk.cuh"
#include "tc_gemm.h"

#include <algorithm>
#include <limits.h>
#include <math.h>

namespace pmoe {
namespace chunk {
namespace {

constexpr int kKeys = kTcKeys;  // of a tile
constexpr int kRows = 256;      // of a query tile pair

// ---------------------------------------------------------------- the plan

// Sums over the threads before this one; *total: over all of them. warps: [2][32].
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warps, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  // every warp adds up the warps' sums for itself
  int64_t w = lane < NT / 32 ? warps[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  __syncthreads();
  return (warp > 0 ? before : 0) + x - v;
}

template <int NT>
struct PlanSmem {
  int64_t warps[32], rows[NT];  // rows of the requests up to each
  int upto[NT + 1];             // tiles before each request of the turn
  int start[NT], n[NT], len[NT];
};

// The start and end of this CTA's run, by all NT threads: the units of all items are added up, NT requests and
// NT items at a time, and the items that its boundaries lie in are looked for; where one turn has them all
// they are at hand, else in a second pass.
template <int NT>
__device__ void find_run(const Args& a, PlanSmem<NT>& m, Run* run) {
  const int tid = threadIdx.x;
  int64_t units = 0;
  int ctas = 0;
  if (tid == 0) run->u = run->end = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int64_t sum = 0, rows = 0;
    for (int r0 = 0; r0 < a.R; r0 += NT) {
      Request q = request(a, r0 + tid);
      // starts that go back may name more rows than there are
      int64_t some, all;
      const int n = q.n;
      const int64_t before = rows + block_scan<NT>(n, m.warps, &some);
      if (before + q.n > a.T) q.bad = true, q.n = 0;
      if (q.bad && pass == 0 && blockIdx.x == 0 && a.err != nullptr) atomicOr(a.err, kErrBadLength);
      rows += some;
      m.upto[tid] = (int)block_scan<NT>((q.n + a.tile_tokens - 1) / a.tile_tokens, m.warps, &all);
      m.start[tid] = q.start, m.n[tid] = q.n, m.len[tid] = q.len, m.rows[tid] = before + n;
      if (tid == 0) m.upto[NT] = (int)all;
      __syncthreads();
      for (int j0 = 0; j0 < all; j0 += NT) {
        const int j = j0 + tid;
        int lo = 0, hi = NT, len = 0, i = 0, ntok = 0;  // upto[lo] <= j < upto[hi]
        if (j < all) {
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (m.upto[mid] <= j)
              lo = mid;
            else
              hi = mid;
          }
          i = j - m.upto[lo];
          const int i0 = i * a.tile_tokens;
          int first;
          ntok = min(a.tile_tokens, m.n[lo] - i0);
          len = a.head + key_tiles(a, m.len[lo] - m.n[lo] + i0, ntok, &first);
        }
        int64_t more;
        const int64_t base = sum + block_scan<NT>((int64_t)len * a.kv.kv_heads, m.warps, &more);
        sum += more;
        const bool single = a.R <= NT && all <= NT;
        if (single) units = sum;
        if (pass == 1 || single) {
          // runs of four units at least
          ctas = (int)min((int64_t)a.ctas, (units + 3) / 4);
          if ((int)blockIdx.x < ctas)
            for (int side = 0; side < 2; ++side) {
              const int64_t in = run_start(units, ctas, blockIdx.x + side) - base;
              if (in < 0 || in >= (int64_t)len * a.kv.kv_heads) continue;
              const int h = in >> 32 ? (int)(in / len) : (int)((uint32_t)in / (uint32_t)len);
              const int at = moved(a, units, ctas, (int)(in - (int64_t)h * len), len, ntok);
              const int64_t u = base + (int64_t)h * len + at;
              if (side == 1) {
                run->end = u;
              } else {
                run->u = u, run->units = units, run->ctas = ctas, run->req = r0 + lo, run->tile = i, run->h = h, run->at = at;
                run->start = m.start[lo], run->n = m.n[lo], run->len = m.len[lo], run->before = m.rows[lo];
              }
            }
          if (tid == 0 && (int)blockIdx.x + 1 == ctas) run->end = units;
        }
        if (single) pass = 2;
      }
    }
    if (sum == 0) break;
    units = sum;
  }
  fence_async();  // what this wrote, TMA will write again
  __syncthreads();
}

// The same by one warp, where neither requests nor items can be more than 32.
__device__ __forceinline__ void find_run_of_few(const Args& a, int8_t* list, Run* run) {
  const int lane = threadIdx.x & 31;
  auto scan = [&](int64_t v) {  // up to and with each lane
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    return v;
  };
  Request q = request(a, lane);
  const int64_t rows = scan(q.n);
  if (rows > a.T) q.bad = true, q.n = 0;
  if (q.bad && blockIdx.x == 0 && a.err != nullptr) atomicOr(a.err, kErrBadLength);
  // the items, request by request; lane j then takes the j-th
  const int tiles = (q.n + a.tile_tokens - 1) / a.tile_tokens, upto = (int)scan(tiles);
#pragma unroll 1
  for (int i = 0; i < tiles; ++i) list[upto - tiles + i] = (int8_t)lane;
  __syncwarp();
  const bool live = lane < __shfl_sync(0xffffffffu, upto, 31);
  const int r = live ? list[lane] : 0;
  const int i = lane - __shfl_sync(0xffffffffu, upto - tiles, r), start = __shfl_sync(0xffffffffu, q.start, r),
            n = __shfl_sync(0xffffffffu, q.n, r), len = __shfl_sync(0xffffffffu, q.len, r);
  const int64_t before = __shfl_sync(0xffffffffu, rows, r);
  const int ntok = min(a.tile_tokens, n - i * a.tile_tokens);
  int span = 0, lo;
  if (live) span = a.head + key_tiles(a, len - n + i * a.tile_tokens, ntok, &lo);
  const int64_t mine = (int64_t)span * a.kv.kv_heads, end = scan(mine), units = __shfl_sync(0xffffffffu, end, 31);
  const int ctas = (int)min((int64_t)a.ctas, (units + 3) / 4);
  if (lane == 0) run->u = 0, run->end = (int)blockIdx.x + 1 == ctas ? units : 0;
  __syncwarp();
  if ((int)blockIdx.x < ctas)
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const int64_t in = run_start(units, ctas, blockIdx.x + side) - (end - mine);
      if (in < 0 || in >= mine) continue;
      const int h = in >> 32 ? (int)(in / span) : (int)((uint32_t)in / (uint32_t)span);
      const int at = moved(a, units, ctas, (int)(in - (int64_t)h * span), span, ntok);
      const int64_t u = end - mine + (int64_t)h * span + at;
      if (side == 1) {
        run->end = u;
      } else {
        run->units = units, run->u = u, run->ctas = ctas, run->h = h, run->at = at;
        run->req = r, run->tile = i, run->start = start, run->n = n, run->len = len, run->before = before;
      }
    }
  __syncwarp();
}

// Clears the counts of an item's parts.
__global__ void __launch_bounds__(256) clear_kernel(uint32_t* done, int n) {
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < n; i += 256) done[i] = 0;
}

// ---------------------------------------------------------------- the tensor cores

template <int D, bool F8>
struct Cfg {
  static constexpr int kTileBytes = kKeys * D * 2;        // one K or V tile, 16-bit operands
  static constexpr int kQBytes = kRows * D * 2;           // both query tiles: [D / 64][256 rows][128 bytes]
  static constexpr int kSlots = D == 128 ? 5 : 8;         // ring of K and V tiles
  static constexpr int kThreads = F8 ? 512 : 384;         // whole warpgroups
  // Registers a thread, by warpgroup: what the other roles give up the softmax takes. The
  // launch has 168 (bf16) or 128 (e4m3) of them for each of its threads.
  static constexpr int kSoftmaxRegs = F8 ? 184 : 200, kMmaRegs = F8 ? 72 : 104, kLoaderRegs = F8 ? 72 : 0;
  static_assert(kSoftmaxRegs * 256 + (kMmaRegs + kLoaderRegs) * 128 <= (F8 ? 128 : 168) * kThreads, "register shares");
  static constexpr int kRing = kSlots * kTileBytes;
  // e4m3: where TMA puts a tile's bytes for the conversion. Heads of 128: the upper half of the
  // tile's slot, whose line of row r also takes that row's upper 64 values, so that the warp that
  // converts a row reads it before it writes. Heads of 64: a ring of their own.
  static constexpr int kRawBytes = kKeys * D, kRawRing = F8 && D == 64 ? kSlots * kRawBytes : 0;
  static __device__ __forceinline__ uint8_t* raw(uint8_t* smem, uint32_t slot) {
    return D == 64 ? smem + kRing + slot * kRawBytes : smem + slot * kTileBytes + kRawBytes;
  }
  static constexpr int kSmem = kRing + kRawRing + kQBytes + 1024 /* alignment */ + 1024 /* row exponents */ + 1024;
  static constexpr int kTmemCols = 512;                   // S0 S1 at 0 and 128, O0 O1 at 256 and 384
  // Whether segments of one query tile have their scores made two tiles ahead, in both query tiles' places: a chain
  // of few rows' tiles then has no wait for scores in it. 64 single tokens on 16,000 keys at most: heads of 64
  // 199 us (without 245), prompt of 8,192 tokens 331 (318). Not with e4m3 (225 / 267, but 377 / 359), whose softmax
  // has no registers left for it, and not with heads of 128 (189 / 172), whose ring is too short.
  static constexpr bool kAhead = D == 64 && !F8;
  static constexpr int kGuards = F8 ? 4 : 2;              // warps that look at partly visible values
  // The base of the weights' exponents lies so far below the largest score, which may outgrow it by 8 more before
  // the base moves. So fp16 weights reach 2^15 at most and the largest one is 2^7 or more: the rounding to fp16's smallest
  // step, 2^-24, is by 2^-32 of the largest at most. (With the base at the largest score it was 2^-25, and a million
  // keys of 2^-25.5 each were lost while the weights' sum held them.) bf16 has fp32's range.
  static constexpr float kLift = F8 ? 7.f : 0.f;
};

constexpr int kSegs = 8;

struct Bars {
  uint64_t full[8], empty[8], raw[8];
  uint64_t vok[8];  // partly visible values are cleared
  uint64_t sfull[4] /* by query tile and place */, pready[2] /* by place */, odone[2], joined[2], qfull, qraw, qempty, drain;
  uint32_t tmem;
  int abort;
  int last[2];  // whether a query tile's last part was the item's
  Run run;
  uint8_t poison[4][16];  // [guard warp][segment % 16]: cleared values that some row sees
  // The segments, which the loader works out for all, in a ring that needs no way back: when it writes
  // segment s + 8, the tiles of s + 3 are done with (a ring of tiles holds four), hence
  // both query tiles with a segment after s, as those of one query tile come in turn (so are `poison`,
  // of 16, and the e4m3 row exponents, of 4, whose writers wait for the segment before).
  uint64_t segready[kSegs];
  Segment segs[kSegs];
};
static_assert(sizeof(Bars) <= 1024, "room behind the row exponents");

// Segment i; false after the last one, or where a wait gave up.
__device__ __forceinline__ bool get_segment(Bars& b, uint32_t i, Segment* s, volatile int* abort_flag, int32_t* err) {
  if (!warp_wait(&b.segready[i % kSegs], i / kSegs & 1, abort_flag, err)) return false;
  const volatile int4* p = reinterpret_cast<const volatile int4*>(&b.segs[i % kSegs]);
  s->req = p[0].x, s->tok0 = p[0].y, s->p0 = p[0].z, s->lo = p[0].w;
  s->t0 = p[1].x, s->t1 = p[1].y, s->join = p[1].z, s->bits = p[1].w;
  s->part0 = p[2].x, s->part1 = p[2].y, s->part2 = p[2].z;
  return s->bits != 0;
}

// the larger of two pairs of bf16
__device__ __forceinline__ uint32_t max2(uint32_t x, uint32_t y) {
  const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&x), *reinterpret_cast<const __nv_bfloat162*>(&y));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// the lowest n bits, n below 0 and above 32 as 0 and 32
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; }

// bf16 pairs with an element that is not finite: the top bits of the 16-bit halves say which
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; }

// What column d of the values adds to a row at position p beyond its finite values: the sum of
// the infinities and NaNs among the values that it sees, in the segment's partly visible tiles.
template <int D, bool F8>
__device__ __noinline__ float poison_of(const Args& a, const Segment& sg, int p, int d) {
  float sum = 0.f;
  const int psh = 31 - __clz(a.kv.page_size);
  for (int t = sg.t0; t < sg.t1; ++t) {
    const int k0 = tile_key<kKeys>(a, sg, t);
    if (!sg.partly(t)) continue;
    for (int j = k0; j < k0 + kKeys && j <= p; ++j) {
      if (!sees(a, p, j)) continue;
      const int page = a.page_table[(int64_t)sg.req * a.table_stride + (j >> psh)];
      if ((unsigned)page >= (unsigned)a.kv.num_pages) continue;
      const int64_t at = page * a.kv.page_stride + ((int64_t)sg.h() * a.kv.page_size + (j & (a.kv.page_size - 1))) * D + d;
      float v;
      if (F8) {
        const uint8_t c = static_cast<const uint8_t*>(a.kv.v)[at];
        v = (c & 0x7f) == 0x7f ? __uint_as_float(0x7fc00000) : 0.f;
      } else {
        v = __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.kv.v)[at] << 16);
      }
      if (!(fabsf(v) < INFINITY)) sum += v;
    }
  }
  return sum;
}

// log of a sum of weights to base m of their exponents, in units of log 2
__device__ __forceinline__ float lse_of(float m, float l) { return m == -INFINITY ? -INFINITY : (m + __log2f(l)) * kLn2; }
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : __frcp_rn(l); }

// Joins the parts of `rows` rows from row i0 of an item on, in the order of the CTAs, by the four warps
// of a query tile, w this one. Little code: it runs once in a while, and what is not in the instruction
// cache costs more than what it does. First a row's base and sum, then its weighted sums, 16 bytes a lane.
template <int D>
__device__ __noinline__ void join(const Args& a, const Segment& sg, int i0, int rows, int w) {
  constexpr int L = D / 4, S = 32 / L;  // lanes of a row, rows at a time
  const int lane = threadIdx.x & 31, sub = lane / L, c = lane % L * 4;
  const int c0 = sg.join & 0xffff, parts = sg.join >> 16;
  const int64_t stride = 2 * a.part_rows;
  const int64_t at0 = (int64_t)c0 * stride + i0;  // of part p: + p stride, and one slot further for p = 0
  const uint32_t row0 = (uint32_t)sg.tok0 * a.q_heads + sg.h() * a.group;
  auto part_at = [&](int p) { return at0 + p * stride + (p == 0 ? a.part_rows : 0); };
  auto put = [&](int r, const float (&acc)[4], float inv) {
    const int i = i0 + r;
    const uint32_t row = row0 + i + row_token(a, i) * (a.q_heads - a.group);
    *reinterpret_cast<uint2*>(a.out + (int64_t)row * D + c) =
        make_uint2(pack2<false>(acc[0] * inv, acc[1] * inv), pack2<false>(acc[2] * inv, acc[3] * inv));
  };
  if (rows <= 8) {
    // a warp two rows, 8 parts of them at a time
    constexpr int U = 2 / S, P = 8;
    const int r0 = w * 2 + sub;
    float m[U], l[U], acc[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k) m[k] = -INFINITY, l[k] = acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
#pragma unroll 1
    for (int p0 = 0; p0 < parts; p0 += P) {
      float2 ml[P][U];
      float4 o[P][U];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int64_t at = part_at(min(p0 + p, parts - 1));
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int r = min(r0 + k, rows - 1);
          ml[p][k] = __ldcg(a.ml_part + at + r);
          o[p][k] = __ldcg(reinterpret_cast<const float4*>(a.o_part + (at + r) * D + c));
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        float top = m[k];
#pragma unroll
        for (int p = 0; p < P; ++p) top = fmaxf(top, ml[p][k].x);
        const float base = top == -INFINITY ? 0.f : top, f = ex2(m[k] - base);
        m[k] = top;
        l[k] *= f, acc[k][0] *= f, acc[k][1] *= f, acc[k][2] *= f, acc[k][3] *= f;
#pragma unroll
        for (int p = 0; p < P; ++p)
          if (p0 + p < parts) {
            const float g = ex2(ml[p][k].x - base);
            l[k] = fmaf(ml[p][k].y, g, l[k]);
            acc[k][0] = fmaf(o[p][k].x, g, acc[k][0]), acc[k][1] = fmaf(o[p][k].y, g, acc[k][1]);
            acc[k][2] = fmaf(o[p][k].z, g, acc[k][2]), acc[k][3] = fmaf(o[p][k].w, g, acc[k][3]);
          }
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (r0 + k < rows) {
        put(r0 + k, acc[k], inverse(l[k]));
        if (a.lse != nullptr && c == 0)
          a.lse[row0 + i0 + r0 + k + row_token(a, i0 + r0 + k) * (a.q_heads - a.group)] = lse_of(m[k], l[k]);
      }
    return;
  }
  // a warp 32 rows: a lane a row, for the base and the sum; then 8 rows at a time
  const int b0 = w * 32;
  if (b0 >= rows) return;
  const int mine = min(b0 + lane, rows - 1);
  float m = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int p = 0; p < parts; ++p) {
    const float2 ml = __ldcg(a.ml_part + part_at(p) + mine);
    const float top = fmaxf(m, ml.x), base = top == -INFINITY ? 0.f : top;
    l = l * ex2(m - base) + ml.y * ex2(ml.x - base);
    m = top;
  }
  const float base = m == -INFINITY ? 0.f : m, inv = inverse(l);
  if (a.lse != nullptr && b0 + lane < rows) a.lse[row0 + i0 + mine + row_token(a, i0 + mine) * (a.q_heads - a.group)] = lse_of(m, l);
  constexpr int U = 8;
#pragma unroll 1
  for (int g0 = 0; g0 < min(32, rows - b0); g0 += U * S) {
    float acc[U][4];
#pragma unroll
    for (int k = 0; k < U; ++k) acc[k][0] = acc[k][1] = acc[k][2] = acc[k][3] = 0.f;
#pragma unroll 2
    for (int p = 0; p < parts; ++p) {
      const float f = ex2(__ldcg(a.ml_part + part_at(p) + mine).x - base);
      const float* src = a.o_part + (part_at(p) + b0) * D + c;
      float4 o[U];
#pragma unroll
      for (int k = 0; k < U; ++k)  // (rows beyond the last: the last, of the item's part all the same)
        o[k] = __ldcg(reinterpret_cast<const float4*>(src + min(g0 + k * S + sub, rows - 1 - b0) * D));
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float g = __shfl_sync(0xffffffffu, f, (g0 + k * S + sub) & 31);
        acc[k][0] = fmaf(o[k].x, g, acc[k][0]), acc[k][1] = fmaf(o[k].y, g, acc[k][1]);
        acc[k][2] = fmaf(o[k].z, g, acc[k][2]), acc[k][3] = fmaf(o[k].w, g, acc[k][3]);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int r = g0 + k * S + sub;
      const float v = __shfl_sync(0xffffffffu, inv, r & 31);
      if (b0 + r < rows) put(b0 + r, acc[k], v);
    }
  }
}

// 4 x 4 units of 32 bytes turned over among four lanes: lane j of the four leaves with unit j of each.
__device__ __forceinline__ void turn_units(uint32_t (&r)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int bit = 1; bit <= 2; bit <<= 1) {
    const bool up = lane & bit;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (u & bit) continue;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t give = up ? r[u * 8 + k] : r[(u + bit) * 8 + k];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, give, bit);
        if (up)
          r[u * 8 + k] = got;
        else
          r[(u + bit) * 8 + k] = got;
      }
    }
  }
}

// q_many, q_few: boxes of tile_tokens and of few_tokens tokens of q, all heads of a kv head (bf16 caches)
template <int D, bool F8>
__global__ void __launch_bounds__(Cfg<D, F8>::kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                 const __grid_constant__ CUtensorMap q_many, const __grid_constant__ CUtensorMap q_few, const Args a) {
  using C = Cfg<D, F8>;
  constexpr int kSlots = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = smem + C::kRing + C::kRawRing;
  // e4m3: the power of two that each row of q was divided by, of four segments in turn
  volatile int8_t* qexp = reinterpret_cast<volatile int8_t*>(qs + C::kQBytes);  // [4][256]
  Bars& b = *reinterpret_cast<Bars*>(qs + C::kQBytes + 1024);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &b.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&b.full[i], F8 ? 4 : 1);
      // the MMAs' commit, and the guards, which keep in step with the ring
      mbar_init(&b.empty[i], F8 ? 1 : 1 + C::kGuards);
      mbar_init(&b.raw[i], 1);
      mbar_init(&b.vok[i], C::kGuards);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.sfull[2 * i], 1);
      mbar_init(&b.sfull[2 * i + 1], 1);
      mbar_init(&b.pready[i], 4);
      mbar_init(&b.odone[i], 1);
      mbar_init(&b.joined[i], 4);
    }
    mbar_init(&b.qfull, F8 ? 4 : 1);
    mbar_init(&b.qraw, 1);
    mbar_init(&b.qempty, 1);
    for (int i = 0; i < kSegs; ++i) mbar_init(&b.segready[i], 1);
    mbar_init(&b.drain, 1);
    b.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&map_k);
    prefetch_map(&map_v);
    prefetch_map(&q_few);
    prefetch_map(&q_many);
  }
  pdl_wait();
  pdl_trigger();
  // (the ring is not in use yet)
  if (a.few)
    __syncthreads();
  else
    find_run<C::kThreads>(a, *reinterpret_cast<PlanSmem<C::kThreads>*>(smem), &b.run);
  // The issuing warp allocates all 512 columns: the base is column 0, lane 0. The other roles
  // touch TMEM only after its first products.
  constexpr uint32_t tmem = 0;
  const int psh = 31 - __clz(a.kv.page_size);
  Segment sg;
  auto load_q = [&](const Segment& s, uint64_t* bar) {
    if (lane == 0) {
      const bool few = s.ntok() <= a.few_tokens;
      mbar_arrive_expect_tx(bar, (few ? a.few_tokens : a.tile_tokens) * a.group * D * 2);
#pragma unroll
      for (int hf = 0; hf < D / 64; ++hf)
        tma_load_3d(qs + hf * (kRows * 128), few ? &q_few : &q_many, bar, hf * 64, s.h() * a.group, s.tok0);
    }
    __syncwarp();
  };

  if (warp < 8) {
    // ---------------- softmax: one thread a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    const int q = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = lanes + 256 + q * 128;
    uint32_t segs = 0;         // segments of this query tile so far
    uint32_t n = 0, other = 0;  // its tiles with the scores in its place, in the other's
    uint32_t tiles = 0;        // key tiles so far
    bool ok = true;
    auto lifted = [](float top) {  // the base for a largest score
      if constexpr (F8) return top - C::kLift;
      return top;
    };
    for (uint32_t all = 0; ok && get_segment(b, all, &sg, abort_flag, a.err); tiles += sg.t1 - sg.t0, ++all) {
      if (!sg.has(q)) continue;
      const bool ahead = C::kAhead && !sg.two();
      const int i = (sg.two() ? q * 128 : 0) + row;  // row of the item
      const int rows = sg.ntok() * a.group;
      const bool live = i - lane < rows;           // any row of this warp
      const int tok = row_token(a, i), pos = sg.p0 + tok;  // (of rows beyond the last: any)
      // What a score is multiplied by, scale x key scale x the row's power of two, has to be above
      // zero: then the largest score stays the largest, and a masked one -inf. So a sign goes
      // to the scores, and where the factor is 0 (or vanishes in fp32) q is 0 and it is 1.
      const float ks = F8 ? a.kv.k_scale[sg.h()] : 1.f;
      const bool negate = (a.scale < 0.f) != (ks < 0.f);
      float mul = 1.f;
      float m = -INFINITY, l = 0.f;
      for (int t = sg.t0; t < sg.t1; ++t) {
        const int place = ahead ? sg.place(t) : q;
        const uint32_t turn = place == q ? n++ : other++;
        const uint32_t ts = lanes + place * 128;
        if (!warp_wait(&b.sfull[q * 2 + place], turn & 1, abort_flag, a.err)) {
          ok = false;
          break;
        }
        if (!live) {  // (whatever the scores are, as weights they reach their own rows only)
          warp_arrive(&b.pready[place]);
          continue;
        }
        fence_after();
        if (t == sg.t0) {
          // (the scores are there, so q's rows were)
          if (F8) {
            const float factor = fabsf(a.scale) * fabsf(ks) * pow2(qexp[(all & 3) * 256 + i]);
            mul = factor != 0.f ? factor : 1.f;
          } else {
            // (scale 0: times 2^-149 the largest score is below 2^-20)
            mul = a.scale != 0.f ? fabsf(a.scale) : __uint_as_float(1);
          }
        }
        const int k0 = tile_key<kKeys>(a, sg, t);
        if (negate || sg.partly(t)) {
          // masked in TMEM: seldom needed code that does not displace the loop's from the cache
          const int hi = pos - k0 + 1, lo = a.window > 0 ? hi - a.window : 0, sink = a.sinks - k0;
          const uint32_t sign = negate ? 0x80000000u : 0u;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            uint32_t r[32];
            tmem_ld32(ts + c, r);
            const uint32_t see = low_bits(hi - c) & (~low_bits(lo - c) | low_bits(sink - c));
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) r[k] = see >> k & 1 ? r[k] ^ sign : 0xff800000u;
            tmem_st16(ts + c, *reinterpret_cast<const uint32_t(*)[16]>(r));
            tmem_st16(ts + c + 16, *reinterpret_cast<const uint32_t(*)[16]>(r + 16));
          }
          tmem_wait_st();
        }
        float s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, reinterpret_cast<uint32_t*>(s) + 32 * c);
        tmem_wait_ld();
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 128; c += 2) x[(c >> 1) & 3] = max3(x[(c >> 1) & 3], s[c], s[c + 1]);
        const float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * mul;
        if (t == sg.t0) {
          m = lifted(mx);
        } else {
          const bool grow = mx > m + (8.f + C::kLift);
          if (__any_sync(0xffffffffu, grow)) {
            // the products so far are done: these scores were issued after them, or the last one's values are
            // released
            if (ahead) {
              const uint32_t i = 2 * (tiles + t - sg.t0) - 1;
              if (!warp_wait(&b.empty[i % kSlots], i / kSlots & 1, abort_flag, a.err)) {
                ok = false;
                break;
              }
              fence_after();
            }
            const float f = grow ? ex2(m - lifted(mx)) : 1.f;
            if (grow) m = lifted(mx);
            l *= f;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16(to + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(to + c, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        const uint64_t mul2 = pair(mul, mul), base2 = pair(-base, -base);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t p[16];
          const float* sc = s + 32 * c;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float y, z;
            unpair(fma2(pair(sc[2 * k], sc[2 * k + 1]), mul2, base2), y, z);
            y = ex2(y), z = ex2(z);
            sum[k & 1] = add2(sum[k & 1], pair(y, z));
            p[k] = pack2<F8>(y, z);
          }
          tmem_st16(ts + 16 * c, p);
        }
        tmem_wait_st();
        fence_before();
        warp_arrive(&b.pready[place]);
        float y, z;
        unpair(add2(sum[0], sum[1]), y, z);
        l += y + z;
      }
      if (!ok || !warp_wait(&b.odone[q], segs++ & 1, abort_flag, a.err)) break;
      if (live) {
        fence_after();
        bool poisoned = false;
#pragma unroll
        for (int k = 0; k < C::kGuards; ++k) poisoned |= *(volatile uint8_t*)&b.poison[k][all & 15] != 0;
        if (poisoned) {
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tmem_ld16(to + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              o[k] = __float_as_uint(__uint_as_float(o[k]) + (i < rows ? poison_of<D, F8>(a, sg, pos, c + k) : 0.f));
            tmem_st16(to + c, o);
            tmem_wait_st();
          }
        }
        // 128 bytes of each row at a time, turned over among four lanes, so that a store covers half of each
        // of 8 lines (a row a lane covers 16 bytes of 32 lines: 5,000 cycles for an item, 1,900 so)
        const bool whole = sg.whole();
        const float vs = (F8 ? a.kv.v_scale[sg.h()] : 1.f) * (whole ? inverse(l) : 1.f);
        const uint32_t head = (uint32_t)(sg.tok0 + tok) * a.q_heads + sg.h() * a.group + i - tok * a.group;
        const uint32_t part = (blockIdx.x * 2 + (sg.t0 == 0)) * a.part_rows + i;
        uint8_t* dst[4];  // of rows (lane & ~3) + k, from this lane's unit on
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t of = __shfl_sync(0xffffffffu, whole ? head : part, rows > 32 ? (lane & ~3) + k : lane);
          dst[k] = (whole ? reinterpret_cast<uint8_t*>(a.out + (int64_t)of * D) : reinterpret_cast<uint8_t*>(a.o_part + (int64_t)of * D)) +
                   (rows > 32 ? lane & 3 : k) * 32;
        }
        // of the four stores' rows these are there; few rows stay a lane each
        const int mine = rows > 32 ? rows - (i - lane) - (lane & ~3) : i < rows ? 4 : 0;
#pragma unroll 1
        for (int c = 0; c < D; c += whole ? 64 : 32) {
          uint32_t o[32];
          tmem_ld32(to + c, o);
          tmem_wait_ld();
          if (whole) {
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = pack2<false>(__uint_as_float(o[2 * k]) * vs, __uint_as_float(o[2 * k + 1]) * vs);
            uint32_t o2[32];
            tmem_ld32(to + c + 32, o2);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              o[16 + k] = pack2<false>(__uint_as_float(o2[2 * k]) * vs, __uint_as_float(o2[2 * k + 1]) * vs);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * vs);
          }
          if (rows > 32) turn_units(o);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (k < mine) {
              reinterpret_cast<uint4*>(dst[k])[0] = make_uint4(o[8 * k], o[8 * k + 1], o[8 * k + 2], o[8 * k + 3]);
              reinterpret_cast<uint4*>(dst[k])[1] = make_uint4(o[8 * k + 4], o[8 * k + 5], o[8 * k + 6], o[8 * k + 7]);
            }
            dst[k] += 128;
          }
        }
        if (i < rows) {
          if (!whole)
            a.ml_part[part] = make_float2(m, l);
          else if (a.lse != nullptr)
            a.lse[head] = lse_of(m, l);
        }
        fence_before();
      }
      if (!sg.whole()) {
        // the query tile's four warps, the ones without rows too, and one of them counts the part
        __threadfence();
        warp_arrive(&b.joined[q]);
        if (!warp_wait(&b.joined[q], 0, abort_flag, a.err)) break;
        if ((warp & 3) == 0 && lane == 0) {
          const int half = sg.two() ? q : 0;
          *(volatile int*)&b.last[q] = atomicAdd(&a.done[(sg.join & 0xffff) * 2 + half], 1u) + 1 == (uint32_t)(sg.join >> 16);
        }
        warp_arrive(&b.joined[q]);
        if (!warp_wait(&b.joined[q], 1, abort_flag, a.err)) break;
        if (*(volatile int*)&b.last[q]) {
          __threadfence();
          const int i0 = i - row;
          join<D>(a, sg, i0, min(128, rows - i0), warp & 3);
        }
      }
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kMmaRegs));
    if (warp == 8) {
      // ---------------- MMA issuer
      asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&b.tmem)),
                   "r"(C::kTmemCols)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
      const uint32_t is = idesc_bf16(128, kKeys) & (F8 ? ~((1u << 7) | (1u << 10)) : ~0u);
      const uint32_t io = (idesc_bf16(128, D) & (F8 ? ~((1u << 7) | (1u << 10)) : ~0u)) | (1u << 16);  // B: N contiguous
      const uint32_t ring = smem_u32(smem), qa = smem_u32(qs);
      uint32_t kv = 0;               // K and V tiles so far
      uint32_t part = 0;             // by slot, whether an odd number of partly visible tiles was there
      uint32_t segs = 0;
      uint32_t pn[2] = {0, 0};       // products with V of each query tile so far
      auto wait = [&](uint64_t* bar, uint32_t parity) { return warp_wait(bar, parity & 1, abort_flag, a.err); };
      // three at once, where all are there already (one after another they take 500 cycles): with it a prompt
      // of 8,192 tokens, 32 / 4 heads of 128, takes 383 us (was 407), with heads of 64 333 (was 325)
      auto there = [&](uint64_t* x, uint32_t px, uint64_t* y, uint32_t py, uint64_t* z, uint32_t pz) {
        const bool rx = mbar_try_wait(x, px & 1), ry = mbar_try_wait(y, py & 1), rz = mbar_try_wait(z, pz & 1);
        return __all_sync(0xffffffffu, rx && ry && rz) != 0;
      };
      auto wait_kv = [&](uint32_t i) { return wait(&b.full[i % kSlots], i / kSlots); };
      // scores by query tile q, whose rows are at qq, to a place in TMEM; the last query tile's are the last on this K tile,
      // and with a segment's last tile on its q
      auto scores = [&](int q, int place, uint32_t qq, uint32_t slot, bool last, bool end) {
        if (converged_lane()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t in = (k % 4) * 32;
            mma_bf16(tmem + place * 128, sw128_desc(qq + (k / 4) * (kRows * 128) + in),
                     sw128_desc(ring + slot * C::kTileBytes + (k / 4) * (kKeys * 128) + in), is, k > 0);
          }
          mma_commit(&b.sfull[q * 2 + place]);
          if (last) mma_commit(&b.empty[slot]);
          if (end) mma_commit(&b.qempty);
        }
        __syncwarp();
      };
      // weights x values of tile t of sg by query tile q
      auto products = [&](int t, int q, int place, uint32_t slot, bool last) {
        const uint32_t o = tmem + 256 + q * 128, p = tmem + place * 128, v = ring + slot * C::kTileBytes;
        if (converged_lane()) {
#pragma unroll
          for (int k = 0; k < kKeys / 16; ++k) mma_f16_ts(o, p + k * 8, v_desc(v + k * 2048), io, t > sg.t0 || k > 0);
          if (last) mma_commit(&b.empty[slot]);
        }
        __syncwarp();
      };
      // the same of any tile: of a partly visible one only the steps of 16 keys that some row sees
      auto any_products = [&](int t, int q, int place, uint32_t slot, bool last) {
        const uint32_t o = tmem + 256 + q * 128, p = tmem + place * 128, v = ring + slot * C::kTileBytes;
        int step0 = 0, step1 = kKeys / 16;
        if (sg.partly(t)) {
          const Span pt = seen_span<kKeys>(a, sg, tile_key<kKeys>(a, sg, t));
          step0 = pt.first / 16, step1 = pt.end / 16;
        }
        if (converged_lane()) {
#pragma unroll 1
          for (int k = step0; k < step1; ++k) mma_f16_ts(o, p + k * 8, v_desc(v + k * 2048), io, t > sg.t0 || k > step0);
          if (t + 1 == sg.t1) mma_commit(&b.odone[q]);
          if (last) mma_commit(&b.empty[slot]);
        }
        __syncwarp();
      };
      auto wait_v = [&](int t, uint32_t i) {
        if (!wait_kv(i)) return false;
        if (F8 || !sg.partly(t)) return true;
        const uint32_t slot = i % kSlots;
        if (!wait(&b.vok[slot], part >> slot)) return false;
        part ^= 1u << slot;
        return true;
      };
      auto q_rows = [&](const Segment& s, int q) { return qa + (s.two() && q ? 128 * 128 : 0); };
      // all scores of a segment's first tile
      auto first_scores = [&](const Segment& s, uint32_t slot) {
        const bool end = s.t0 + 1 == s.t1;
        for (int q = s.two() ? 0 : s.lane(); q < (s.two() ? 2 : s.lane() + 1); ++q) {
          const bool last = !s.two() || q == 1;
          scores(q, C::kAhead && !s.two() ? s.place(s.t0) : q, q_rows(s, q), slot, last, last && end);
        }
      };
      bool ok = true, have = get_segment(b, 0, &sg, abort_flag, a.err);
      if (have) {
        ok = wait(&b.qfull, segs) && wait_kv(kv);
        fence_after();
        if (ok) first_scores(sg, kv % kSlots);
      }
      while (ok && have) {
        const int qb = sg.two() ? 0 : sg.lane(), qe = sg.two() ? 2 : sg.lane() + 1;
        int t = sg.t0;
        if (C::kAhead && !sg.two()) {
          // scores two tiles ahead, in turn in both query tiles' places: the second tile's now, the others' with the
          // products of the tile whose place they take
          auto next = [&](int u, uint32_t i) {
            if (!wait_kv(i)) return false;
            fence_after();
            scores(qb, sg.place(u), qa, i % kSlots, true, u + 1 == sg.t1);
            return true;
          };
          if (t + 1 < sg.t1) ok = next(t + 1, kv + 2);
          for (; ok && t + 1 < sg.t1; ++t, kv += 2) {
            const int place = sg.place(t);
            const bool plain = t + 2 < sg.t1 && !sg.partly(t);
            const bool all = plain && there(&b.full[(kv + 1) % kSlots], (kv + 1) / kSlots, &b.pready[place], pn[place],
                                            &b.full[(kv + 4) % kSlots], (kv + 4) / kSlots);
            if (!all && !(wait_v(t, kv + 1) && wait(&b.pready[place], pn[place]))) {
              ok = false;
              break;
            }
            ++pn[place];
            fence_after();
            if (plain)
              products(t, qb, place, (kv + 1) % kSlots, true);
            else
              any_products(t, qb, place, (kv + 1) % kSlots, true);
            if (t + 2 < sg.t1) ok = next(t + 2, kv + 4);
          }
          if (!ok) break;
        }
        // (a query tile's weights come after it has read its accumulators of the segment before)
        while (t + 1 < sg.t1) {
          // a run of tiles that all rows see, in as few instructions as can be: this warp's are what the
          // tensor cores wait for (with the other tiles' case in the loop 60,000 keys take 7% longer)
          const int stop = min(t < sg.part0 ? sg.part0 : t < sg.part1 ? t : sg.part2, sg.t1 - 1);
          for (; t < stop; ++t, kv += 2) {
            const uint32_t vslot = (kv + 1) % kSlots, kslot = (kv + 2) % kSlots;
            const bool all = D == 128 && there(&b.full[kslot], (kv + 2) / kSlots, &b.full[vslot], (kv + 1) / kSlots, &b.pready[qb], pn[qb]);
            if (!all && (!wait_kv(kv + 2) || !wait_kv(kv + 1))) {
              ok = false;
              break;
            }
            const bool end = t + 2 == sg.t1;
            for (int q = qb; q < qe; ++q) {
              if (!(all && q == qb) && !wait(&b.pready[q], pn[q])) {
                ok = false;
                break;
              }
              ++pn[q];
              fence_after();
              products(t, q, q, vslot, q + 1 == qe);
              scores(q, q, q_rows(sg, q), kslot, q + 1 == qe, end && q + 1 == qe);
            }
            if (!ok) break;
          }
          if (!ok) break;
          if (t + 1 == sg.t1) break;
          if (!wait_kv(kv + 2) || !wait_v(t, kv + 1)) {
            ok = false;
            break;
          }
          for (int q = qb; q < qe; ++q) {
            if (!wait(&b.pready[q], pn[q])) {
              ok = false;
              break;
            }
            ++pn[q];
            fence_after();
            any_products(t, q, q, (kv + 1) % kSlots, q + 1 == qe);
            scores(q, q, q_rows(sg, q), (kv + 2) % kSlots, q + 1 == qe, t + 2 == sg.t1 && q + 1 == qe);
          }
          if (!ok) break;
          ++t, kv += 2;
        }
        if (!ok) break;
        // the last tile: the next segment's scores come before and between its products with V, but where q
        // is late
        Segment nx;
        const bool more = get_segment(b, segs + 1, &nx, abort_flag, a.err);  // (made known behind this tile)
        if (__any_sync(0xffffffffu, *abort_flag)) break;
        const uint32_t vslot = (kv + 1) % kSlots, kslot = (kv + 2) % kSlots;
        const bool early = more && __all_sync(0xffffffffu, mbar_try_wait(&b.qfull, (segs + 1) & 1));
        // the other query tile's turn: at once, where the place of its scores is not still to be read
        const bool first = early && !sg.two() && !nx.two() && (!C::kAhead || nx.place(nx.t0) != sg.lane());
        const bool late = !early || (C::kAhead && !nx.two() && !first);
        if (early && !wait_kv(kv + 2)) break;
        fence_after();
        if (first) first_scores(nx, kslot);
        if (!wait_v(t, kv + 1)) break;
        for (int q = 0; q < 2; ++q) {
          if (sg.has(q)) {
            if (!wait(&b.pready[q], pn[q])) {
              ok = false;
              break;
            }
            ++pn[q];
            fence_after();
            any_products(t, q, q, vslot, q + 1 == qe);
          }
          if (!late && !first && nx.has(q)) {
            const bool last = !nx.two() || q == 1;
            scores(q, q, q_rows(nx, q), kslot, last, last && nx.t0 + 1 == nx.t1);
          }
        }
        if (!ok) break;
        if (more && late) {
          if (!early && (!wait(&b.qfull, segs + 1) || !wait_kv(kv + 2))) break;
          fence_after();
          first_scores(nx, kslot);
        }
        kv += 2;
        sg = nx;
        have = more;
        ++segs;
      }
      // every MMA and its arrival are done before the CTA leaves
      if (converged_lane()) {
        mma_commit(&b.drain);
        const long long t0 = clock64();
        while (!mbar_try_wait(&b.drain, 0) && clock64() - t0 < kWaitLimit) {
        }
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---------------- TMA loader: lane i issues box i % halves of page box i / halves
      constexpr int kHalves = F8 ? 1 : D / 64, kBytes = F8 ? 1 : 2;
      uint64_t* arrive = F8 ? b.raw : b.full;
      const int box = min(a.kv.page_size, kKeys), boxes = kKeys / box;
      uint32_t kv = 0;
      bool ok = true;
      Walk walk;
      if (a.few) find_run_of_few(a, reinterpret_cast<int8_t*>(&b.segs[kSegs - 1]), &b.run);  // (a place not yet in use)
      walk.begin(a, b.run);
      for (uint32_t i = 0; ok; ++i) {
        if (!walk.next(a, &sg)) sg.bits = 0;
        if (lane == 0) {
          b.segs[i % kSegs] = sg;
          mbar_arrive(&b.segready[i % kSegs]);
        }
        __syncwarp();
        if (sg.bits == 0) break;
        const int32_t* table = a.page_table + (int64_t)sg.req * a.table_stride;
        // the ids of 32 pages from `first` on, one a lane: a tile's own would cost it the latency of a load
        int first = INT_MAX, ids = 0;
        for (int t = sg.t0; t < sg.t1 && ok; ++t) {
          const int pb = lane / kHalves, hf = lane % kHalves;
          const int key0 = tile_key<kKeys>(a, sg, t), key = key0 + pb * box, page0 = key0 >> psh;
          if (page0 < first || page0 + boxes > first + 32) {
            first = page0;
            ids = 0;
            if (page0 + lane <= max(sg.p1(), 0) >> psh) ids = __ldg(table + page0 + lane);
          }
          int id = __shfl_sync(0xffffffffu, ids, ((key >> psh) - first) & 31);
          // pages with a key that some row sees
          bool use = pb < boxes && key <= sg.p1();
          if (use && a.window > 0) use = key + box - 1 > sg.p0 - a.window || key < a.sinks;
          if (use && (unsigned)id >= (unsigned)a.kv.num_pages) {
            if (a.err != nullptr) atomicOr(a.err, kErrBadPage);
            id = a.kv.num_pages;  // out of the map's range: reads as zeros
          }
          const int used = __popc(__ballot_sync(0xffffffffu, use));
          for (int v = 0; v < 2; ++v, ++kv) {
            const uint32_t slot = kv % kSlots;
            if (!warp_wait(&b.empty[slot], ((kv / kSlots) & 1) ^ 1, abort_flag, a.err)) {
              ok = false;
              break;
            }
            if (lane == 0) mbar_arrive_expect_tx(&arrive[slot], used * box * (F8 ? D : 64) * kBytes);
            __syncwarp();
            uint8_t* dst = F8 ? C::raw(smem, slot) + pb * box * D : smem + slot * C::kTileBytes + hf * (kKeys * 128) + pb * box * 128;
            if (use)
              tma_load_4d(dst, v ? &map_v : &map_k, &arrive[slot], hf * 64, key & (a.kv.page_size - 1), sg.h(), id);
          }
        }
      }
      // copies in flight land before the CTA leaves, even where another role gave up
      for (uint32_t i = kv > kSlots ? kv - kSlots : 0; i < kv; ++i) {
        const long long t0 = clock64();
        while (!mbar_try_wait(&arrive[i % kSlots], (i / kSlots) & 1) && clock64() - t0 < kWaitLimit) {
        }
      }
    } else if constexpr (!F8) {
      // ---------------- guards: warps 10 and 11 look at the values of partly visible tiles;
      // warp 10 also loads q. A box holds whole tokens, so rows beyond the item's are the next tokens' or zero.
      const int gw = warp - 10;
      uint32_t kv = 0, segs = 0, loads = 0;
      bool ok = get_segment(b, 0, &sg, abort_flag, a.err);
      if (gw == 0 && ok) load_q(sg, &b.qfull), ++loads;
      while (ok) {
        Segment nx;
        bool more = false;
        if (lane == 0) *(volatile uint8_t*)&b.poison[gw][segs & 15] = 0;
        __syncwarp();
        for (int t = sg.t0; t < sg.t1 && ok; ++t) {
          const int k0 = tile_key<kKeys>(a, sg, t);
          for (int v = 0; v < 2; ++v, ++kv) {
            const uint32_t slot = kv % kSlots;
            if (!warp_wait(&b.full[slot], (kv / kSlots) & 1, abort_flag, a.err)) {
              ok = false;
              break;
            }
            if (v == 1 && t + 1 == sg.t1) {
              // the next segment's q, once this one's last scores are there
              more = get_segment(b, segs + 1, &nx, abort_flag, a.err);
              if (more && gw == 0) {
                if (!warp_wait(&b.qempty, segs & 1, abort_flag, a.err)) {
                  ok = false;
                  break;
                }
                load_q(nx, &b.qfull);
                ++loads;
              }
            }
            if (v == 1 && sg.partly(t)) {
              bool found = false;
              const Span pt = seen_span<kKeys>(a, sg, k0);
              const int below = pt.low - pt.first, rows = below + pt.end - pt.high;
#pragma unroll 1
              for (int i = gw * 32 + lane; i < rows * (D / 8); i += 64) {
                const int n = i / (D / 8), c = i % (D / 8), r = n < below ? pt.first + n : pt.high + n - below;
                if (all_see(a, sg.p0, sg.p1(), k0 + r)) continue;
                uint4* at = reinterpret_cast<uint4*>(smem + slot * C::kTileBytes + (c / 8) * (kKeys * 128) + r * 128 + (c & 7) * 16);
                if (!any_sees(a, sg.p0, sg.p1(), k0 + r)) {
                  *at = make_uint4(0, 0, 0, 0);
                  continue;
                }
                const uint4 x = *at;
                uint32_t w[4] = {x.x, x.y, x.z, x.w};
                if (not_finite(w[0]) | not_finite(w[1]) | not_finite(w[2]) | not_finite(w[3])) {
                  found = true;
#pragma unroll
                  for (int k = 0; k < 4; ++k) {
                    const uint32_t bad = not_finite(w[k]);
                    w[k] &= ~((bad & 0x8000u ? 0xffffu : 0u) | (bad & 0x80000000u ? 0xffff0000u : 0u));
                  }
                  *at = make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
              if (found) *(volatile uint8_t*)&b.poison[gw][segs & 15] = 1;
              fence_async();
              warp_arrive(&b.vok[slot]);
            }
            warp_arrive(&b.empty[slot]);
          }
        }
        ok = ok && more;
        sg = nx;
        ++segs;
      }
      // q's copy in flight lands before the CTA leaves
      if (loads > 0) {
        const long long t0 = clock64();
        while (!mbar_try_wait(&b.qfull, (loads - 1) & 1) && clock64() - t0 < kWaitLimit) {
        }
      }
    } else {
      // ---------------- e4m3: warp 10 loads q
      uint32_t loads = 0;
      if (warp == 10)
        for (; get_segment(b, loads, &sg, abort_flag, a.err); ++loads) {
          if (loads > 0 && !warp_wait(&b.qempty, (loads - 1) & 1, abort_flag, a.err)) break;
          load_q(sg, &b.qraw);
        }
      // q's copy in flight lands before the CTA leaves
      if (loads > 0) {
        const long long t0 = clock64();
        while (!mbar_try_wait(&b.qraw, (loads - 1) & 1) && clock64() - t0 < kWaitLimit) {
        }
      }
    }
  } else if constexpr (F8) {
    // ---------------- e4m3 conversion: 16 codes a thread and step, to fp16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLoaderRegs));
    constexpr int CH = D / 16;  // 16-code chunks of a row
    constexpr int N = kKeys * CH / 128;
    const int tid = threadIdx.x - 12 * 32, ch = tid % CH, r0 = tid / CH;
    uint32_t kv = 0, segs = 0;
    bool ok = true;
    for (; ok && get_segment(b, segs, &sg, abort_flag, a.err); ++segs) {
      if (lane == 0) *(volatile uint8_t*)&b.poison[warp - 12][segs & 15] = 0;
      __syncwarp();
      {  // q in place, divided by each row's power of two; rows beyond the item's stay what they were
        constexpr int LPR = D / 8, U = 4, kStep = 128 / LPR;  // threads of a row, chunks at once, rows at a time
        const int rows = sg.ntok() * a.group, c = tid % LPR;
        const float factor = fabsf(a.scale) * fabsf(a.kv.k_scale[sg.h()]);
        if (!warp_wait(&b.qraw, segs & 1, abort_flag, a.err)) break;
        uint8_t* q0 = qs + (c / 8) * (kRows * 128);
#pragma unroll 1
        for (int i0 = 0; i0 < rows; i0 += U * kStep) {
          const int ra = i0 + tid / LPR;
          uint4 v[U];
          uint32_t mx[U];
#pragma unroll
          for (int p = 0; p < U; ++p) {
            const int r = min(ra + p * kStep, kRows - 1);
            v[p] = *reinterpret_cast<const uint4*>(q0 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            mx[p] = max2(max2(v[p].x & 0x7fff7fffu, v[p].y & 0x7fff7fffu), max2(v[p].z & 0x7fff7fffu, v[p].w & 0x7fff7fffu));
            mx[p] = max2(mx[p], mx[p] >> 16);
          }
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1)
#pragma unroll
            for (int p = 0; p < U; ++p) mx[p] = max2(mx[p], __shfl_xor_sync(0xffffffffu, mx[p], o));
#pragma unroll
          for (int p = 0; p < U; ++p) {
            const int r = ra + p * kStep;
            const int e = row_exponent(__uint_as_float(mx[p] << 16));
            const float down = factor * pow2(e) != 0.f ? pow2(-e) : 0.f;
            uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              w[k] = pack2<true>(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
            if (r < rows) {
              if (c == 0) qexp[(segs & 3) * 256 + r] = (int8_t)e;
              *reinterpret_cast<uint4*>(q0 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        fence_async();
        warp_arrive(&b.qfull);
      }
      for (int i2 = 2 * sg.t0; i2 < 2 * sg.t1; ++i2, ++kv) {  // K and V of each tile
        const uint32_t slot = kv % kSlots;
        if (!warp_wait(&b.raw[slot], (kv / kSlots) & 1, abort_flag, a.err)) {
          ok = false;
          break;
        }
        uint8_t* src = C::raw(smem, slot);
        const int k0 = tile_key<kKeys>(a, sg, i2 / 2);
        auto at = [&](int r) { return D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4); };
        if ((i2 & 1) && sg.partly(i2 / 2)) {
          bool found = false;
#pragma unroll 1
          for (int i = 0; i < N; ++i) {
            const int r = r0 + i * (128 / CH), j = k0 + r;
            if (all_see(a, sg.p0, sg.p1(), j)) continue;
            const uint32_t any = any_sees(a, sg.p0, sg.p1(), j) ? ~0u : 0u;
            uint4 x = *reinterpret_cast<const uint4*>(src + at(r));
            uint32_t* w = &x.x;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t nan = ((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u & any;  // the code 0x7f of either sign
              found |= nan != 0;
              w[k] = w[k] & ~((nan >> 7) * 0xffu) & any;
            }
            *reinterpret_cast<uint4*>(src + at(r)) = x;
          }
          if (found) *(volatile uint8_t*)&b.poison[warp - 12][segs & 15] = 1;
        }
        uint4 raw[N];
#pragma unroll
        for (int i = 0; i < N; ++i) raw[i] = *reinterpret_cast<const uint4*>(src + at(r0 + i * (128 / CH)));
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = r0 + i * (128 / CH);
          uint8_t* dst = smem + slot * C::kTileBytes + (ch / 4) * (kKeys * 128) + r * 128;
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          uint32_t f[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) f[2 * k] = e4m3x2(w[k] & 0xffffu), f[2 * k + 1] = e4m3x2(w[k] >> 16);
          // 8 threads hold a row of 128: the upper four write their halves the other way
          // round, so that the two 64-value blocks meet on different banks
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int kk = k ^ (ch / 4 & 1);
            *reinterpret_cast<uint4*>(dst + (((2 * (ch % 4) + kk) ^ (r & 7)) << 4)) =
                kk ? make_uint4(f[4], f[5], f[6], f[7]) : make_uint4(f[0], f[1], f[2], f[3]);
          }
        }
        fence_async();
        warp_arrive(&b.full[slot]);
      }
    }
  }
  fence_before();
  __syncthreads();
  fence_after();
  if (warp == 8)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kTmemCols) : "memory");
}

// ---------------------------------------------------------------- host side

int sm_count() {
  static std::atomic<int> count[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < 64 && (n = count[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
  if (dev < 64) count[dev].store(n, std::memory_order_relaxed);
  return n;
}

int make_map(const Args& a, void* base, CUtensorMap* m) {
  const bool f8 = a.kv.dtype == PMOE_KV_E4M3;
  const uint64_t D = a.kv.head_dim, page = a.kv.page_size, eb = f8 ? 1 : 2;
  const uint64_t dims[4] = {D, page, (uint64_t)a.kv.kv_heads, (uint64_t)a.kv.num_pages};
  const uint64_t strides[3] = {D * eb, page * D * eb, (uint64_t)a.kv.page_stride * eb};
  const uint32_t box[4] = {f8 ? (uint32_t)D : 64u, (uint32_t)std::min<uint64_t>(page, kKeys), 1, 1};
  return tc_encode_map(m, base, 4, dims, strides, box, !f8 ? kTcMapBf16Sw128 : D == 128 ? kTcMapBytesSw128 : kTcMapBytesSw64);
}

int make_q_map(const Args& a, int tokens, CUtensorMap* m) {
  const uint64_t D = a.kv.head_dim;
  const uint64_t dims[3] = {D, (uint64_t)a.q_heads, (uint64_t)a.T};
  const uint64_t strides[2] = {D * 2, (uint64_t)a.q_stride * 2};
  const uint32_t box[3] = {64, (uint32_t)a.group, (uint32_t)tokens};
  return tc_encode_map(m, const_cast<__nv_bfloat16*>(a.q), 3, dims, strides, box, kTcMapBf16Sw128);
}

template <int D, bool F8>
int launch_all(const Args& a, cudaStream_t s) {
  using C = Cfg<D, F8>;
  const char* what = "moe_chunk_attention";
  static SmemLimit limit;
  CUtensorMap mk, mv, many, few;
  int r = make_map(a, a.kv.k, &mk);
  if (r == PMOE_OK) r = make_map(a, a.kv.v, &mv);
  if (r == PMOE_OK) r = make_q_map(a, a.tile_tokens, &many);
  if (r == PMOE_OK) r = make_q_map(a, a.few_tokens, &few);
  if (r == PMOE_OK) r = limit.set(reinterpret_cast<const void*>(chunk_kernel<D, F8>), C::kSmem, what);
  if (r == PMOE_OK) r = launch(what, clear_kernel, 1, 256, 0, s, true, 1, a.done, 2 * a.ctas);
  if (r == PMOE_OK) r = launch(what, chunk_kernel<D, F8>, a.ctas, C::kThreads, C::kSmem, s, true, 1, mk, mv, many, few, a);
  return r;
}

struct Layout {
  size_t ml, done, bytes;
};

// Fills what follows from the sizes alone.
int plan(const pmoe_kv_desc* kv, int T, int q_heads, int R, Args* a, Layout* l) {
  const int r = check_kv(kv);
  if (r != PMOE_OK) return r;
  if (T < 0 || R < 0 || R > (1 << 20) || q_heads < 1 || q_heads % kv->kv_heads != 0) return PMOE_EINVAL;
  if ((int64_t)T * q_heads >= (1 << 24)) return PMOE_EINVAL;
  a->kv = *kv;
  a->T = T;
  a->R = R;
  a->q_heads = q_heads;
  a->group = q_heads / kv->kv_heads;
  if (a->group > kMaxGroup) return PMOE_EUNSUPPORTED;
  a->group_magic = (uint32_t)((1ull << 32) / a->group + 1);
  if (T == 0 || R == 0) return PMOE_OK;
  a->ctas = sm_count();
  if (a->ctas == 0) return PMOE_ECUDA;
  a->tile_tokens = kRows / a->group;
  a->few_tokens = std::max(1, 16 / a->group);
  // in us with 2 / 3 / 4 / 6: a prompt of 8,192 tokens (32 / 4 heads of 128) 427 / 411 / 412 / 423, with e4m3
  // 691 / 589 / 508 / 478; 256 single tokens with a window of 4,096 314 / 316 / 318 / 319
  a->head = kv->dtype == PMOE_KV_E4M3 ? 5 : 3;
  a->few = R <= 32 && T / a->tile_tokens + std::min(R, T) <= 32;
  a->part_rows = std::min(kRows, T * a->group);
  const size_t parts = (size_t)a->ctas * 2 * a->part_rows;
  l->ml = parts * kv->head_dim * 4;
  l->done = l->ml + parts * 8;
  l->bytes = l->done + (size_t)a->ctas * 8;
  return PMOE_OK;
}

}  // namespace
}  // namespace chunk
}  // namespace pmoe

using namespace pmoe;

extern "C" size_t moe_chunk_attention_scratch_bytes(const pmoe_kv_desc* kv, int T, int q_heads, int R) {
  chunk::Args a{};
  chunk::Layout l{};
  return chunk::plan(kv, T, q_heads, R, &a, &l) == PMOE_OK ? l.bytes : 0;
}

extern "C" int moe_chunk_attention(const pmoe_kv_desc* kv, const void* q, int64_t q_stride, int T, int q_heads, float scale,
                                   const int32_t* q_start, const int32_t* kv_len, int R, const int32_t* page_table,
                                   int table_stride, int window, int sinks, void* out, float* lse, void* scratch,
                                   size_t scratch_bytes, int32_t* err_out, void* stream) {
  // arguments first: the plan asks the device for its size
  if (check_kv(kv) == PMOE_OK && T > 0 && R > 0) {
    auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (q == nullptr || out == nullptr || q == out || off(q, 16) || off(out, 16) || q_stride % 8 != 0 ||
        q_stride < (int64_t)q_heads * kv->head_dim || !(fabsf(scale) < INFINITY))
      return PMOE_EINVAL;
    if (q_start == nullptr || kv_len == nullptr || page_table == nullptr || off(q_start, 4) || off(kv_len, 4) ||
        off(page_table, 4) || table_stride < 1 || (int64_t)table_stride * kv->page_size > (1 << 30))
      return PMOE_EINVAL;
    if (off(lse, 4) || off(err_out, 4) || off(scratch, 16)) return PMOE_EINVAL;
  }
  if (window < 0 || sinks < 0) return PMOE_EINVAL;
  chunk::Args a{};
  chunk::Layout lay{};
  const int r = chunk::plan(kv, T, q_heads, R, &a, &lay);
  if (r != PMOE_OK || T == 0 || R == 0) return r;
  if (scratch == nullptr || scratch_bytes < lay.bytes) return PMOE_EINVAL;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.scale = scale * attn::kLog2e;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.table_stride = table_stride;
  // a request has 2^30 keys at most: a window or sinks of as many hide nothing
  a.window = window >= (1 << 30) || sinks >= (1 << 30) ? 0 : window;
  a.sinks = a.window > 0 ? sinks : 0;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = err_out;
  uint8_t* base = static_cast<uint8_t*>(scratch);
  a.o_part = reinterpret_cast<float*>(base);
  a.ml_part = reinterpret_cast<float2*>(base + lay.ml);
  a.done = reinterpret_cast<uint32_t*>(base + lay.done);
  cudaStream_t s = (cudaStream_t)stream;
  const bool f8 = kv->dtype == PMOE_KV_E4M3;
  if (kv->head_dim == 128) return f8 ? chunk::launch_all<128, true>(a, s) : chunk::launch_all<128, false>(a, s);
  return f8 ? chunk::launch_all<64, true>(a, s) : chunk::launch_all<64, false>(a, s);
}
