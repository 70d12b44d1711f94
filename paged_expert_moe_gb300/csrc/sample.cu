// moe_sample_tokens: temperature, top-k, top-p, min-p and the draw, one pass over the logits.
//
// A row's weights n_i = floor(exp((x_i - m) / temperature) * 2^31) are whole numbers and so
// are all their sums: atomics and reductions in any order give the same draw.
//
// Bound: HBM for many rows (each logit read once), the chain of dependent steps for few. A
// cluster of up to 8 CTAs takes a row; each CTA keeps its slice in shared memory and the
// CTAs exchange statistics through distributed shared memory, written to where they are read.
//   1. Load the slice; its largest logit, and those of its threads (or of four groups of each
//      thread's). For rows that are cut by
//      top-k or top-p a lower bound of the K-th largest logit (K = top_k, or 1,024): with K /
//      CTAs of the threads' largest logits at or above a bound in every CTA, K logits are at
//      or above the least of these bounds, and seldom many more.
//   2. These candidates go to the row's first CTA, which orders them, cuts them and draws.
//      Rows with more than 2,048 candidates, or whose candidates do not reach top_p, go on
//      with step 3.
//   3. A histogram of the logits by distance from the largest, count and weight, without those
//      that weigh too little to be at the top-p threshold; the bin that holds the top_k-th token
//      or in which the weight reaches top_p. Its logits (again up to 2,048; else four passes
//      over 8 bits of the ordered logit) give the threshold itself.
//   4. Sums of the kept tokens in id order (ties of the threshold in id order), the segment
//      that holds floor(S * u), and its token.
// Uncut rows take steps 1 and 4.
//
// Measured: a row of 32,000 fp32 logits with top_k 50 and top_p 0.9 7.2 us, uncut 5.0; 64 bf16
// rows of 131,072 of all kinds 28 to 36 us by what the slowest rows need; 256 fp32 rows of 160,001
// 94 to 102 us, 1.6 TB/s, where a read alone would take 24. What holds them up is the chain of a row: its some ten exchanges between
// the CTAs and passes of a few hundred cycles each, on the 36 clusters that find room at once.
#include "pmoe_internal.h"

#include <cooperative_groups.h>
#include <float.h>
#include <limits.h>
#include <math.h>

namespace cg = cooperative_groups;

namespace pmoe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;          // distance bins (one per thread)
constexpr float kBinsPerUnit = 16.f;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 262144;
constexpr int kMaxSmem = (kMaxVocab / kMaxCluster + 8) * 4;
constexpr int kMerged = 2048;       // candidates of a row
// Candidates: more of them decide more rows, but a list that overflows costs a pass for nothing.
// top_k up to which rows are cut by theirs (16 rows of 131,072 with top_k 1,000 12.8 us, 25.2 by
// step 3; 40 rows of 32,000 with 1,300 23.5 and 19.9), and, where only top-p cuts, K as a share
// of each CTA (64 rows of 131,072 with top_p 0.8 37.9 us with 48, 26.9 with 128; 40 rows of
// 32,000 11.9, 12.4, and 17.4 with 150).
constexpr int kMaxK = 1200;
constexpr int kCutP = 128;
constexpr int kPairs = 256;         // elements up to which all pairs are compared
constexpr int kSegs = kMaxCluster * kWarps;

typedef unsigned long long u64;

struct SampleArgs {
  const void* logits;
  int T, V;
  int64_t row_stride;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* ids;
  float* logprob;
  int slice;  // elements of a CTA's slice (a multiple of 8)
};

struct Histogram {        // weights as two 16-bit halves: a slice holds at most 40,968
  uint32_t cnt[kBins];    // elements, so that no half's sum leaves 32 bits
  uint32_t lo[kBins];
  uint32_t hi[kBins];
};

struct Threshold {        // kept: key > this key, and the first `ties` ids that have it
  uint32_t key, ties;
  u64 total;              // weight of the kept tokens
};

struct Pick {             // a bin found by a scan, weight and count above it (bin kBins: all)
  u64 above;
  uint32_t cnt;
  int bin;
};

struct alignas(16) Shared {
  Histogram hist;
  Histogram level;        // select's, and step 3's passes over the key's bits
  u64 merged[kMerged];    // in the row's first CTA: ~key << 32 | id of the candidates
  int listed;             // there: how many,
  u64 sum, list_sum;      // all weights of the row, and the candidates'
  int arg;                // and, of greedy rows, the lowest id that has the largest logit
  float best[kMaxCluster], bound[kMaxCluster];  // every CTA's largest logit, its bound of the K-th
  uint32_t bound_key;
  float top[kWarps];
  Threshold thr;
  int members;            // select: elements of the bin it looks into
  u64 sel, sel_upto;      // and what it found
  u64 scan[kWarps];
  uint32_t scan_cnt[kWarps];
  Pick pick;
  u64 seg_sum[kSegs];     // step 4: per warp segment of the row, weight above the threshold
  uint32_t seg_tie[kSegs];
};

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 -> +0: ties are ties
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ u64 share(u64 total, float part) {
  const u64 n = (u64)(part * 16777216.f);
  return (total >> 24) * n + (((total & 0xffffffull) * n) >> 24);
}

__device__ __forceinline__ u64 share_of(u64 total, float u) { return share(total, u > 0.f ? fminf(u, 0.99999994f) : 0.f); }

__device__ __forceinline__ u64 least_weight(u64 total, float top_p) {
  return max((u64)1, share(total, top_p > 0.f ? top_p : 0.f));
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 d = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += d;
  }
  return v;
}
// Inclusive scan over the block; *total: the sum. Two barriers.
__device__ __forceinline__ u64 block_scan(Shared& sh, u64 v, u64* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v, lane);
  if (lane == 31) sh.scan[warp] = v;
  __syncthreads();
  u64 before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    const u64 s = sh.scan[i];
    if (i < warp) before += s;
    all += s;
  }
  __syncthreads();
  *total = all;
  return v + before;
}

__device__ __forceinline__ float exp2_approx(float x) {  // 2 ulp; what it flushes to 0 is below 2^-126
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Row {
  float m, r;  // largest logit, log2(e) / temperature; both finite but for rows with +inf
  // With a largest logit of +inf, r is too: +inf weighs the most there is, everything else 0.
  __device__ __forceinline__ Row(float best, float temp)
      : m(fminf(best, FLT_MAX)), r(best == INFINITY ? INFINITY : fminf(1.44269504f / temp, FLT_MAX)) {}
  // log2 of a weight: four roundings of an argument of at most 31, where the weight is not 0,
  // change the weight by less than 2^-17 of it.
  __device__ __forceinline__ float log2w(float x) const { return (x - m) * r; }
  __device__ __forceinline__ float weight(float x) const { return exp2_approx(log2w(x)); }
  // NaN gives 0, as -inf does
  __device__ __forceinline__ static uint32_t units(float w) { return (uint32_t)(w * 2147483648.f); }
  __device__ __forceinline__ uint32_t units_of(float x) const { return units(weight(x)); }
  // Distance from the largest in bins; with an infinite largest one it is below 0.
  __device__ __forceinline__ float distance(float x) const { return (m - x) * kBinsPerUnit; }
  __device__ __forceinline__ int bin(float x) const {
    const float d = distance(x);
    return d < (float)(kBins - 1) ? (int)(uint32_t)d : kBins - 1;  // the conversion takes d < 0 to 0
  }
};

template <bool BF16>
struct Vec {
  static constexpr int N = BF16 ? 8 : 4;  // logits in 16 bytes
  float f[N];
  static __device__ __forceinline__ uint4 none() {  // -inf
    const uint32_t w = BF16 ? 0xff80ff80u : 0xff800000u;
    return make_uint4(w, w, w, w);
  }
  __device__ __forceinline__ explicit Vec(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (BF16) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        f[i] = __uint_as_float(w[i]);
      }
    }
  }
};

constexpr int kEach = kMerged / kThreads;  // sorted elements of a thread

// Sorts the block's kMerged elements ascending: thread t has elements t * kEach .. of `buf`
// on entry (read after a barrier) and of the sorted sequence in c on return. Bitonic: pairs
// within a thread, within a warp by shuffles, further apart through `buf`.
__device__ void sort_up(u64* buf, u64 (&c)[kEach]) {
  static_assert(kEach == 4, "element pairs below");
  const int t = threadIdx.x;
#pragma unroll
  for (int e = 0; e < kEach; ++e) c[e] = buf[t * kEach + e];
  auto order = [](u64& x, u64& y, bool up) {
    const u64 lo = min(x, y), hi = max(x, y);
    x = up ? lo : hi;
    y = up ? hi : lo;
  };
  for (int k = 2; k <= kMerged; k <<= 1) {
    for (int j = k >> 1; j >= kEach; j >>= 1) {
      const int d = j / kEach;  // the partner's distance in threads
      const bool low = ((t & d) == 0) == ((t * kEach & k) == 0);
      u64 o[kEach];
      if (d < 32) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) o[e] = __shfl_xor_sync(0xffffffffu, c[e], d);
      } else {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kEach; ++e) buf[e * kThreads + t] = c[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kEach; ++e) o[e] = buf[e * kThreads + (t ^ d)];
      }
#pragma unroll
      for (int e = 0; e < kEach; ++e) c[e] = low ? min(c[e], o[e]) : max(c[e], o[e]);
    }
    if (k == 2) {
      order(c[0], c[1], true);
      order(c[2], c[3], false);
    } else {
      const bool up = (t * kEach & k) == 0;
      order(c[0], c[2], up);
      order(c[1], c[3], up);
      order(c[0], c[1], up);
      order(c[2], c[3], up);
    }
  }
  __syncthreads();  // buf is free
}

// Room in the first CTA's list (`to`) for the `c` candidates of this thread: where they begin.
// One remote atomic a warp; all lanes call it.
__device__ __forceinline__ int reserve(Shared* to, int c) {
  const int lane = threadIdx.x & 31;
  int upto = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int d = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += d;
  }
  int at = 0;
  if (lane == 31 && upto > 0) at = atomicAdd(&to->listed, upto);
  return __shfl_sync(0xffffffffu, at, 31) + upto - c;
}
__device__ __forceinline__ void put(Shared* to, int at, float x, int id) {
  if (at < kMerged) to->merged[at] = ((u64)~key_of(x) << 32) | (uint32_t)id;
}

__device__ __forceinline__ int pow2_above(int n) { return n <= 64 ? 64 : 1 << (32 - __clz(n - 1)); }

// The first CTA adds up bin `threadIdx.x` of all CTAs' histograms (`h`: this CTA's) and finds
// the first bin, ascending, at which the running count (by_count) or weight reaches `target`
// (> 0). Every CTA of the cluster calls it, and has the result in sh.pick (bin kBins where it
// is not reached). Had each CTA read all histograms for itself, it would take 5,500 cycles.
__device__ void find_bin(cg::cluster_group& cluster, Shared& sh, Histogram* h, bool by_count, bool weights, u64 target) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nb = (int)cluster.num_blocks();
  cluster.sync();
  if (cluster.block_rank() == 0) {
    if (tid == 0) sh.listed = 0;  // every CTA has read it
    uint32_t v[kMaxCluster][3];  // all remote loads in flight at once
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i) {
      const Histogram* o = cluster.map_shared_rank(h, i < nb ? i : 0);
      v[i][0] = by_count ? o->cnt[tid] : 0;
      v[i][1] = weights ? o->lo[tid] : 0, v[i][2] = weights ? o->hi[tid] : 0;
    }
    uint32_t c = 0;
    u64 w = 0;
#pragma unroll
    for (int i = 0; i < kMaxCluster; ++i)
      if (i < nb) c += v[i][0], w += ((u64)v[i][2] << 16) + v[i][1];
    u64 wi = w;
    uint32_t ci = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const u64 a = __shfl_up_sync(0xffffffffu, wi, o);
      const uint32_t d = __shfl_up_sync(0xffffffffu, ci, o);
      if (lane >= o) wi += a, ci += d;
    }
    if (lane == 31) sh.scan[warp] = wi, sh.scan_cnt[warp] = ci;
    __syncthreads();
    u64 wb = 0, total = 0;
    uint32_t cb = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) wb += sh.scan[i], cb += sh.scan_cnt[i];
      total += sh.scan[i];
    }
    wi += wb, ci += cb;
    if (tid == 0) sh.pick = Pick{total, 0, kBins};
    __syncthreads();
    if (by_count ? (ci >= target && ci - c < target) : (wi >= target && wi - w < target))
      sh.pick = Pick{wi - w, ci - c, tid};
    __syncthreads();
    if (tid > 0 && tid < nb) cluster.map_shared_rank(&sh, tid)->pick = sh.pick;
  }
  cluster.sync();
}

// Sum over the G consecutive lanes that share a candidate.
__device__ __forceinline__ u64 group_sum(u64 v, int G) {
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// How many of a[0, n) are below x, and (WEIGHTS) the sums of their weights and of all; the G
// threads that share x take every G-th pair of elements each.
template <bool WEIGHTS>
__device__ __forceinline__ void count_below(const u64* a, const uint32_t* weights, int n, u64 x, int part, int G, u64* place,
                                            u64* before, u64* all) {
  uint32_t p = 0;
  u64 b = 0, s = 0;
  const int pairs = n >> 1;
#pragma unroll 4
  for (int j = part; j < pairs; j += G) {
    const ulonglong2 v = reinterpret_cast<const ulonglong2*>(a)[j];
    const bool f = v.x < x, g = v.y < x;
    p += f;
    p += g;
    if (WEIGHTS) {
      const uint2 w = reinterpret_cast<const uint2*>(weights)[j];
      b += f ? w.x : 0u;
      b += g ? w.y : 0u;
      s += w.x;
      s += w.y;
    }
  }
  if ((n & 1) && part == 0) {
    const bool f = a[n - 1] < x;
    const uint32_t w = WEIGHTS ? weights[n - 1] : 0u;
    p += f;
    b += f ? w : 0u;
    s += w;
  }
  for (int o = G / 2; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
  *place = p;
  if (WEIGHTS) *before = group_sum(b, G), *all = group_sum(s, G);
}

// Step 2's end for up to kPairs candidates, the n of sh.merged. A candidate's place and the
// weight before it come from comparing it with all others, twice: in the order of the logits
// for the cuts, in the order of the ids for the draw. kThreads / n2 threads share a candidate.
__device__ void compare_and_draw(Shared& sh, const SampleArgs& a, const Row& rw, int row, int n, int top_k, bool use_k,
                                 float top_p, bool use_p, float min_p, float uu, u64 all_weights) {
  const int tid = threadIdx.x, n2 = pow2_above(n), G = kThreads / n2, i = tid / G, part = tid % G;
  const bool own = part == 0 && i < n;
  uint32_t *weights = sh.level.cnt, *kept_weights = sh.level.lo;
  const u64 c = i < n ? sh.merged[i] : ~0ull;
  const float wt = rw.weight(of_key(~(uint32_t)(c >> 32)));
  const uint32_t w = i < n ? Row::units(wt) : 0;
  u64 place, before = 0, total = all_weights, unused;
  if (use_p) {
    if (own) weights[i] = w;
    __syncthreads();
    count_below<true>(sh.merged, weights, n, c, part, G, &place, &before, &unused);
  } else {
    count_below<false>(sh.merged, weights, n, c, part, G, &place, &before, &unused);
  }
  const bool in_k = i < n && (!use_k || place < (u64)top_k);
  if (use_k && use_p) {
    if (own && place + 1 == (u64)min(top_k, n)) sh.sel = before + w;  // the weight of the first top_k
    __syncthreads();
    total = sh.sel;
  }
  const u64 least = use_p ? least_weight(total, top_p) : ~0ull;
  const uint32_t kept = in_k && before < least && !(wt < min_p) ? w : 0;
  // by id: what was cut goes behind every id, with no weight
  const u64 by_id = kept > 0 ? c << 32 : ~0ull;
  u64* ids = sh.merged + kPairs;
  if (own) ids[i] = by_id, kept_weights[i] = kept;
  __syncthreads();
  u64 run, S;
  count_below<true>(ids, kept_weights, n, by_id, part, G, &place, &run, &S);
  const u64 target = share_of(S, uu);
  if (own && kept > 0 && run <= target && target < run + kept) {
    a.ids[row] = (int32_t)(uint32_t)c;
    if (a.logprob != nullptr) a.logprob[row] = logf((float)kept / (float)S);
  }
}

__device__ __forceinline__ float logit_of(u64 x) { return of_key(~(uint32_t)(x >> 32)); }

// kEach elements of a thread, ~0 for none; their bins, which keep their order, and weights.
struct Elements {
  u64 c[kEach];
  int bin[kEach];
  uint32_t w[kEach];
};

// Of the block's elements, in ascending order, finds the one at which the running count
// (by_count) or weight reaches `target`, into sh.sel; the running weight up to it goes to
// sh.sel_upto if `weigh` (set without by_count). by_id: elements are id << 32 | weight, not
// ~key << 32 | id. One histogram finds the bin, comparing all pairs inside it the element; a bin
// of more than kPairs elements is sorted instead. sh.level and sh.members are zero on entry and
// on return.
__device__ void select(Shared& sh, const Row rw, const Elements& x, bool by_count, bool weigh, bool by_id, u64 target) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* weights = reinterpret_cast<uint32_t*>(sh.merged + kPairs);
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (x.c[e] != ~0ull) {
      const int b = x.bin[e];
      if (by_count) atomicAdd(&sh.level.cnt[b], 1u);
      if (weigh) {
        atomicAdd(&sh.level.lo[b], x.w[e] & 0xffffu);
        atomicAdd(&sh.level.hi[b], x.w[e] >> 16);
      }
    }
  __syncthreads();
  const uint32_t own_c = sh.level.cnt[tid];
  const u64 own_w = ((u64)sh.level.hi[tid] << 16) + sh.level.lo[tid];
  uint32_t ci = own_c;
  u64 wi = own_w;
  if (by_count) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t d = __shfl_up_sync(0xffffffffu, ci, o);
      if (lane >= o) ci += d;
    }
    if (lane == 31) sh.scan_cnt[warp] = ci;
  }
  if (weigh) {
    wi = warp_scan(wi, lane);
    if (lane == 31) sh.scan[warp] = wi;
  }
  __syncthreads();
  sh.level.cnt[tid] = sh.level.lo[tid] = sh.level.hi[tid] = 0;
#pragma unroll 4
  for (int i = 0; i < warp; ++i) {
    if (by_count) ci += sh.scan_cnt[i];
    if (weigh) wi += sh.scan[i];
  }
  if (by_count ? (ci >= target && ci - own_c < target) : (wi >= target && wi - own_w < target)) {
    sh.pick = Pick{wi - own_w, ci - own_c, tid};
  }
  __syncthreads();
  const int pick = sh.pick.bin;
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (x.c[e] != ~0ull && x.bin[e] == pick) {
      const int at = atomicAdd(&sh.members, 1);
      if (at < kPairs) sh.merged[at] = x.c[e], weights[at] = x.w[e];
    }
  __syncthreads();
  const int m = sh.members;
  if (m <= kPairs) {
    const int n2 = pow2_above(m), G = kThreads / n2, i = tid / G, part = tid % G;
    const u64 one = i < m ? sh.merged[i] : ~0ull;
    u64 place, before, unused;
    count_below<true>(sh.merged, weights, m, one, part, G, &place, &before, &unused);
    place += sh.pick.cnt;
    before += sh.pick.above;
    const uint32_t w = i < m ? weights[i] : 0;
    if (part == 0 && i < m && (by_count ? place + 1 == target : before < target && target <= before + w)) {
      sh.sel = one;
      sh.sel_upto = before + w;
    }
    __syncthreads();
    if (tid == 0) sh.members = 0;
    return;
  }
  // every element is sorted, those of other bins too
  u64 s[kEach];
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kEach; ++e) sh.merged[tid * kEach + e] = x.c[e];
  __syncthreads();
  sort_up(sh.merged, s);
  uint32_t ws[kEach];
  u64 mine = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    ws[e] = s[e] == ~0ull ? 0 : by_id ? (uint32_t)s[e] : rw.units_of(logit_of(s[e]));
    mine += ws[e];
  }
  u64 total, run = block_scan(sh, mine, &total) - mine;
  if (tid == 0) sh.members = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (s[e] != ~0ull && (by_count ? (u64)(tid * kEach + e) + 1 == target : run < target && target <= run + ws[e])) {
      sh.sel = s[e];
      sh.sel_upto = run + ws[e];
    }
    run += ws[e];
  }
  __syncthreads();
}

// sh.merged's n elements to registers, and sh.level cleared; ends with a barrier.
__device__ __forceinline__ void take_merged(Shared& sh, int n, Elements& x) {
  sh.level.cnt[threadIdx.x] = sh.level.lo[threadIdx.x] = sh.level.hi[threadIdx.x] = 0;
  if (threadIdx.x == 0) sh.members = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * kThreads + threadIdx.x;
    x.c[e] = i < n ? sh.merged[i] : ~0ull;
  }
  __syncthreads();
}

// The same for more candidates: the cuts and the draw are selections.
__device__ void select_and_draw(Shared& sh, const SampleArgs& a, const Row rw, int row, int n, int top_k,
                                             bool use_k, float top_p, bool use_p, float min_p, float uu, u64 all_weights) {
  Elements x;
  take_merged(sh, n, x);
  u64 mine = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const float logit = logit_of(x.c[e]);
    x.bin[e] = rw.bin(logit);
    x.w[e] = x.c[e] == ~0ull ? 0 : rw.units_of(logit);
    mine += x.w[e];
  }
  u64 last = ~0ull - 1, total = all_weights;  // the last candidate that is kept
  if (use_k) {
    if (n > top_k) {
      select(sh, rw, x, true, use_p, false, (u64)top_k);
      last = sh.sel, total = sh.sel_upto;
    } else {
      block_scan(sh, mine, &total);
    }
  }
  if (use_p) {
    select(sh, rw, x, false, true, false, least_weight(total, top_p));
    last = min(last, sh.sel);
  }
  // in the order of the ids: id << 32 | weight
  const float bins_per_id = (float)kBins / (float)a.V;
  mine = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const bool cut = x.c[e] > last || rw.weight(logit_of(x.c[e])) < min_p;
    const uint32_t w = cut ? 0 : x.w[e], id = (uint32_t)x.c[e];
    x.c[e] = w > 0 ? ((u64)id << 32) | w : ~0ull;
    x.w[e] = w;
    x.bin[e] = min((int)((float)id * bins_per_id), kBins - 1);
    mine += w;
  }
  u64 S;
  block_scan(sh, mine, &S);
  select(sh, rw, x, false, true, true, share_of(S, uu) + 1);
  if (threadIdx.x == 0) {
    a.ids[row] = (int32_t)(sh.sel >> 32);
    if (a.logprob != nullptr) a.logprob[row] = logf((float)(uint32_t)sh.sel / (float)S);
  }
}

// Step 3's end, in the row's first CTA: sh.merged holds the n logits of bin `bin`; the one at
// which their running count (by_count) or weight reaches `target` is the threshold.
__device__ void find_in_bin(Shared& sh, const Row rw, int n, int bin, bool by_count, u64 target, u64 above) {
  const int tid = threadIdx.x;
  Elements x;
  take_merged(sh, n, x);
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    // the bin, cut into kBins again (the last one reaches to -inf)
    const float logit = logit_of(x.c[e]), d = (rw.distance(logit) - (float)bin) * (float)kBins;
    x.bin[e] = d < (float)(kBins - 1) ? max((int)d, 0) : kBins - 1;
    x.w[e] = rw.units_of(logit);
  }
  select(sh, rw, x, by_count, true, false, target);
  if (tid == 0) sh.thr.ties = 0;
  const u64 sel = sh.sel;
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (x.c[e] <= sel && x.c[e] >> 32 == sel >> 32) atomicAdd(&sh.thr.ties, 1u);
  if (tid == 0) sh.thr.key = ~(uint32_t)(sel >> 32), sh.thr.total = above + sh.sel_upto;
  __syncthreads();
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
  using V = Vec<BF16>;
  constexpr int N = V::N, EB = BF16 ? 2 : 4;
  extern __shared__ __align__(16) uint4 xs[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // waited for before the first remote access
  pdl_wait();  // the logits may come from the kernel ahead
  pdl_trigger();
  const int nb = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / nb;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  const float temp = a.temperature != nullptr ? a.temperature[row] : 1.f;
  const int top_k = a.top_k != nullptr ? a.top_k[row] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[row] : 1.f;
  const float min_p = a.min_p != nullptr ? fminf(a.min_p[row], 1.f) : 0.f;
  const float uu = a.u[row];
  // slices start where the row's 16-byte vectors do: `shift` elements before its first
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + (int64_t)row * a.row_stride * EB;
  const int shift = (int)((reinterpret_cast<uintptr_t>(base) & 15) / EB);
  const int first = rank * a.slice - shift;  // id of the slice's element 0
  const int n = max(0, min(a.slice, a.V - first));
  const int nv = (n + N - 1) / N;            // its vectors

  // ---- 1. load; elements outside the row are -inf
  for (int i = tid; i < nv; i += kThreads) {
    const int id = first + i * N;
    if (id >= 0 && (i + 1) * N <= n) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(xs + i)),
                   "l"(base + (int64_t)id * EB)
                   : "memory");
    } else {
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (BF16) {
          uint32_t h[2];
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int e = id + 2 * q + z;
            h[z] = e >= 0 && i * N + 2 * q + z < n ? reinterpret_cast<const uint16_t*>(base)[e] : 0xff80u;
          }
          w[q] = h[0] | (h[1] << 16);
        } else {
          w[q] = id + q >= 0 && i * N + q < n ? reinterpret_cast<const uint32_t*>(base)[id + q] : 0xff800000u;
        }
      }
      xs[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  sh.hist.cnt[tid] = 0;
  if (tid == 0) sh.arg = INT_MAX, sh.listed = 0, sh.sum = 0, sh.list_sum = 0;
  asm volatile("cp.async.wait_all;" ::: "memory");
  const bool use_k = top_k > 0 && top_k < a.V, use_p = top_p < 1.f;
  const bool listing = temp > 0.f && (use_k ? top_k <= kMaxK : use_p);
  const uint32_t want = use_k ? (top_k + nb - 1) / nb : kCutP;  // of a CTA, if `listing`
  // A bound that a fourth of the threads' largest logits or more shall reach is found from
  // those of four groups of each thread's instead: 256 bf16 rows of 8,000 with top_k 1,000 in
  // one CTA each overflow their lists otherwise. Other rows need not tell the groups apart.
  const bool fine = listing && want > kThreads / 4;
  float mine = -INFINITY;  // of the vectors this thread loaded; fmaxf leaves NaN out
  float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  if (fine) {
    for (int i = tid, k = 0; i < nv; i += kThreads, ++k) {
      const V x(xs[i]);
      float v[N / 4];
#pragma unroll
      for (int h = 0; h < N / 4; ++h) v[h] = fmaxf(fmaxf(x.f[4 * h], x.f[4 * h + 1]), fmaxf(x.f[4 * h + 2], x.f[4 * h + 3]));
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        constexpr int per = 16 / N;  // vectors until the groups come round again
        top4[g] = g / (N / 4) == k % per ? fmaxf(top4[g], v[g % (N / 4)]) : top4[g];
      }
    }
    mine = fmaxf(fmaxf(top4[0], top4[1]), fmaxf(top4[2], top4[3]));
  } else {
    for (int i = tid; i < nv; i += kThreads) {
      const V x(xs[i]);
#pragma unroll
      for (int q = 0; q < N; ++q) mine = fmaxf(mine, x.f[q]);
    }
  }
  float best = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) sh.top[warp] = best;
  __syncthreads();
  best = sh.top[lane % kWarps];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  const float cta_best = best;
  float bound = -FLT_MAX;  // fewer threads with a logit than that: every logit is a candidate
  if (listing) {
    // the bin of the largest logits, by distance from the CTA's, that holds the want-th; the
    // bound is the least of those in it or above it
    const Row by(best, 1.f);
    if (fine) {
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (top4[g] > -INFINITY) atomicAdd(&sh.hist.cnt[by.bin(top4[g])], 1u);
    } else if (mine > -INFINITY) {
      atomicAdd(&sh.hist.cnt[by.bin(mine)], 1u);
    }
    if (tid == 0) sh.pick.bin = kBins, sh.bound_key = 0xffffffffu;
    __syncthreads();
    uint32_t upto = sh.hist.cnt[tid];
    const uint32_t own = upto;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t d = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += d;
    }
    if (lane == 31) sh.scan_cnt[warp] = upto;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i)
      if (i < warp) upto += sh.scan_cnt[i];
    if (upto >= want && upto - own < want) sh.pick.bin = tid;
    __syncthreads();
    const int last = sh.pick.bin;
    if (fine) {
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (top4[g] > -INFINITY && by.bin(top4[g]) <= last) atomicMin(&sh.bound_key, key_of(top4[g]));
    } else if (mine > -INFINITY && by.bin(mine) <= last) {
      atomicMin(&sh.bound_key, key_of(mine));
    }
    __syncthreads();
    if (sh.pick.bin != kBins) bound = of_key(sh.bound_key);
  }
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the row has started
  if (tid < nb) {
    Shared* o = cluster.map_shared_rank(&sh, tid);
    o->best[rank] = cta_best, o->bound[rank] = bound;
  }
  cluster.sync();
#pragma unroll
  for (int i = 0; i < kMaxCluster; ++i)
    if (i < nb) best = fmaxf(best, sh.best[i]), bound = fminf(bound, sh.bound[i]);
  Shared* const head = cluster.map_shared_rank(&sh, 0);  // the row's first CTA

  const Row rw(best, temp);
  if (best == -INFINITY || !(temp > 0.f)) {  // the same for every CTA of the row
    if (best != -INFINITY && cta_best == best) {
      int low = INT_MAX;
      for (int i = tid; i < nv; i += kThreads) {
        const V x(xs[i]);
#pragma unroll
        for (int q = N - 1; q >= 0; --q)
          if (x.f[q] == best) low = min(low, first + i * N + q);
      }
      low = __reduce_min_sync(0xffffffffu, low);
      if (lane == 0 && low != INT_MAX) atomicMin(&head->arg, low);
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
      a.ids[row] = best == -INFINITY ? -1 : sh.arg;
      if (a.logprob != nullptr) a.logprob[row] = best == -INFINITY ? -INFINITY : 0.f;
    }
    return;
  }

  // ---- 2. candidates
  u64 total = 0;  // of all weights where only top-p cuts, then of what is kept
  if (listing) {
    int found = 0;
    if (use_k) {
      if (mine >= bound)
        for (int i = tid; i < nv; i += kThreads) {
          const V x(xs[i]);
#pragma unroll
          for (int q = 0; q < N; ++q) found += x.f[q] >= bound;
        }
    } else {
      u64 sum = 0, list_sum = 0;
      for (int i = tid; i < nv; i += kThreads) {
        const V x(xs[i]);
        uint32_t w[N];
#pragma unroll
        for (int q = 0; q < N; ++q) w[q] = rw.units_of(x.f[q]);
#pragma unroll
        for (int q = 0; q < N; ++q) {
          sum += w[q];
          if (x.f[q] >= bound) list_sum += w[q], ++found;
        }
      }
      sum = warp_sum(sum);
      list_sum = warp_sum(list_sum);
      if (lane == 0) atomicAdd(&head->sum, sum), atomicAdd(&head->list_sum, list_sum);
    }
    if (__any_sync(0xffffffffu, found > 0)) {
      int at = reserve(head, found);
      if (found > 0)
        for (int i = tid; i < nv; i += kThreads) {
          const V x(xs[i]);
#pragma unroll
          for (int q = 0; q < N; ++q)
            if (x.f[q] >= bound) put(head, at++, x.f[q], first + i * N + q);
        }
    }
    cluster.sync();
    const Shared& of = rank == 0 ? sh : *head;
    const int listed = of.listed;  // the same in every CTA
    total = of.sum;
    const u64 list_sum = of.list_sum;
    if (listed <= kMerged && (use_k || list_sum >= least_weight(total, top_p))) {
      asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // this CTA has read the first one's
      if (rank == 0) {
        if (listed <= kPairs)
          compare_and_draw(sh, a, rw, row, listed, top_k, use_k, top_p, use_p, min_p, uu, total);
        else
          select_and_draw(sh, a, rw, row, listed, top_k, use_k, top_p, use_p, min_p, uu, total);
        __syncthreads();
      }
      asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      return;
    }
  }

  // ---- 3. histogram over the distance from the largest
  uint32_t key_t = 0;            // kept: key > key_t, and the first `ties` ids of key == key_t
  uint32_t ties = 0xffffffffu;
  auto elements = [&](auto&& f) {
    for (int i = tid; i < nv; i += kThreads) {
      const V x(xs[i]);
#pragma unroll
      for (int q = 0; q < N; ++q)
        if (x.f[q] > -INFINITY) f(x.f[q]);
    }
  };
  auto add = [&](Histogram& h, int bin, float x, bool count, bool weigh) {
    if (count) atomicAdd(&h.cnt[bin], 1u);
    const uint32_t w = weigh ? rw.units_of(x) : 0;
    if (w) {
      atomicAdd(&h.lo[bin], w & 0xffffu);
      atomicAdd(&h.hi[bin], w >> 16);
    }
  };
  if (use_k || use_p) {
    sh.hist.cnt[tid] = sh.hist.lo[tid] = sh.hist.hi[tid] = 0;
    __syncthreads();
    if (use_k) {
      elements([&](float x) { add(sh.hist, rw.bin(x), x, true, use_p); });
    } else {
      // what weighs at most (total - target) / V cannot be where the target is reached: all of
      // it together weighs less than what may be cut. Half or more of the row's logits, as a rule.
      const uint32_t least = (uint32_t)((total - least_weight(total, top_p)) / (uint32_t)a.V);
      elements([&](float x) {
        const uint32_t w = rw.units_of(x);
        if (w > least) {
          const int b = rw.bin(x);
          atomicAdd(&sh.hist.lo[b], w & 0xffffu);
          atomicAdd(&sh.hist.hi[b], w >> 16);
        }
      });
    }
    for (int mode = use_k ? 0 : 1; mode <= (use_p ? 1 : 0); ++mode) {
      // mode 0: the top_k-th token; mode 1: the token at which the weight reaches top_p (the
      // total is step 2's, or mode 0's)
      const u64 target = mode == 0 ? (u64)top_k : least_weight(total, top_p);
      find_bin(cluster, sh, &sh.hist, mode == 0, use_p, target);
      const Pick pick = sh.pick;
      if (pick.bin == kBins) {  // top_k exceeds the logits above -inf: none is cut
        total = pick.above;
        continue;
      }
      const int bin = pick.bin;
      const u64 inside = target - (mode == 0 ? pick.cnt : pick.above);
      int found = 0;
      const float d_lo = bin == 0 ? -INFINITY : (float)bin, d_hi = bin == kBins - 1 ? NAN : (float)(bin + 1);
      auto inside_bin = [&](float x) {
        const float d = rw.distance(x);
        return d >= d_lo && !(d >= d_hi) && x > -INFINITY;
      };
      for (int i = tid; i < nv; i += kThreads) {
        const V x(xs[i]);
#pragma unroll
        for (int q = 0; q < N; ++q) found += inside_bin(x.f[q]);
      }
      if (__any_sync(0xffffffffu, found > 0)) {
        int at = reserve(head, found);
        if (found > 0)
          for (int i = tid; i < nv; i += kThreads) {
            const V x(xs[i]);
#pragma unroll
            for (int q = 0; q < N; ++q)
              if (inside_bin(x.f[q])) put(head, at++, x.f[q], first + i * N + q);
          }
      }
      cluster.sync();
      const int listed = head->listed;
      if (listed <= kMerged) {
        if (rank == 0) {
          find_in_bin(sh, rw, listed, bin, mode == 0, inside, pick.above);
          if (tid > 0 && tid < nb) cluster.map_shared_rank(&sh, tid)->thr = sh.thr;
        }
        cluster.sync();
        key_t = sh.thr.key, ties = sh.thr.ties;
        total = sh.thr.total;
        continue;
      }
      // inside the bin, 8 bits of the key at a time
      uint32_t prefix = 0;
      u64 over = pick.above;
      uint32_t over_cnt = pick.cnt;
      for (int level = 0; level < 4; ++level) {
        const int sft = 24 - 8 * level;
        sh.level.cnt[tid] = sh.level.lo[tid] = sh.level.hi[tid] = 0;
        __syncthreads();
        elements([&](float x) {
          if (rw.bin(x) != bin) return;
          const uint32_t k = key_of(x);
          if (level == 0 || (k >> (sft + 8)) == prefix) add(sh.level, 255 - ((k >> sft) & 255), x, true, use_p);  // descending
        });
        find_bin(cluster, sh, &sh.level, mode == 0, use_p, target - (mode == 0 ? over_cnt : over));
        over += sh.pick.above;
        over_cnt += sh.pick.cnt;
        prefix = (prefix << 8) | (255 - sh.pick.bin);
      }
      key_t = prefix;
      const u64 each = rw.units_of(of_key(key_t));
      ties = (uint32_t)(mode == 0 ? target - over_cnt : (target - over + each - 1) / each);
      total = over + each * ties;
    }
  }

  // ---- 4. sums in id order: warp w of CTA c owns segment c * kWarps + w
  const int per_warp = ((nv + kWarps - 1) / kWarps + 31) & ~31;
  const int s0 = min(nv, warp * per_warp), s1 = min(nv, s0 + per_warp);
  const bool all_keys = key_t == 0;
  const float x_t = all_keys ? -INFINITY : of_key(key_t);
  const uint32_t unit_t = all_keys ? 0u : rw.units_of(x_t);
  const bool tie_ok = !all_keys && !(rw.weight(x_t) < min_p);
  // an element's weight if it lies above the threshold (ties are counted apart)
  auto kept = [&](float x) -> uint32_t {
    const float w = rw.weight(x);
    return x > x_t && !(w < min_p) ? Row::units(w) : 0u;
  };
  u64 sum = 0;
  uint32_t nt = 0;
  if (all_keys && !(min_p > 0.f)) {
    for (int i = s0 + lane; i < s1; i += 32) {
      const V x(xs[i]);
      uint32_t w[N];
#pragma unroll
      for (int q = 0; q < N; ++q) w[q] = rw.units_of(x.f[q]);
#pragma unroll
      for (int q = 0; q < N; ++q) sum += w[q];
    }
  } else if (!(min_p > 0.f)) {
    for (int i = s0 + lane; i < s1; i += 32) {
      const V x(xs[i]);
      uint32_t w[N];
#pragma unroll
      for (int q = 0; q < N; ++q) {
        w[q] = rw.units_of(x.f[q]);
        nt += x.f[q] == x_t;
      }
#pragma unroll
      for (int q = 0; q < N; ++q) sum += x.f[q] > x_t ? w[q] : 0u;
    }
  } else {
    // A vector whose elements are all cut needs no weights: none at or above the threshold, or
    // all safely below min_p (by more than its logarithm, the weights and x_lo can be off).
    const float x_lo = fmaxf(x_t, rw.m + (log2f(min_p) - 0.01f) / rw.r - fabsf(rw.m) * 2.4e-7f);
    for (int i = s0 + lane; i < s1; i += 32) {
      const V x(xs[i]);
      float top = x.f[0];
#pragma unroll
      for (int q = 1; q < N; ++q) top = fmaxf(top, x.f[q]);
      if (top >= x_lo) {
#pragma unroll
        for (int q = 0; q < N; ++q) {
          nt += x.f[q] == x_t;
          sum += kept(x.f[q]);
        }
      }
    }
  }
  sum = warp_sum(sum);
  nt = (uint32_t)__reduce_add_sync(0xffffffffu, nt);
  if (lane < nb) {  // to every CTA
    Shared* o = cluster.map_shared_rank(&sh, lane);
    o->seg_sum[rank * kWarps + warp] = sum, o->seg_tie[rank * kWarps + warp] = nt;
  }
  cluster.sync();  // the last one: no CTA reads another's memory from here on
  // running ties and sums over the segments, kSegs / 32 in a row to a lane
  constexpr int R = kSegs / 32;
  const int segs = nb * kWarps, seg = rank * kWarps + warp;
  u64 sums[R], run_s = 0;
  uint32_t tied[R], run_t = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int s = lane * R + i;
    sums[i] = s < segs ? sh.seg_sum[s] : 0;
    tied[i] = s < segs ? sh.seg_tie[s] : 0;
    run_t += tied[i];
  }
  {
    const uint32_t own = run_t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t d = __shfl_up_sync(0xffffffffu, run_t, o);
      if (lane >= o) run_t += d;
    }
    run_t -= own;
  }
  uint32_t ties_before[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    ties_before[i] = run_t;
    const uint32_t in = run_t >= ties ? 0 : min(tied[i], ties - run_t);
    run_t += tied[i];
    if (tie_ok) sums[i] += (u64)in * unit_t;
    run_s += sums[i];
  }
  const u64 upto = warp_scan(run_s, lane);
  const u64 S = __shfl_sync(0xffffffffu, upto, 31);
  u64 lo = upto - run_s, hi = lo;
  uint32_t tb = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (i < seg % R) lo += sums[i];
    if (i <= seg % R) hi += sums[i];
    if (i == seg % R) tb = ties_before[i];
  }
  lo = __shfl_sync(0xffffffffu, lo, seg / R);
  hi = __shfl_sync(0xffffffffu, hi, seg / R);
  tb = __shfl_sync(0xffffffffu, tb, seg / R);
  const u64 target = share_of(S, uu);
  if (target >= lo && target < hi) {  // exactly one warp of the cluster
    u64 run = lo;
    for (int i0 = s0; i0 < s1; i0 += 32) {
      u64 w[N], v = 0;
      uint32_t t = 0;
      const int i = i0 + lane;
      const V x(i < s1 ? xs[i] : V::none());
#pragma unroll
      for (int q = 0; q < N; ++q) t += x.f[q] == x_t;
      uint32_t ti = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t d = __shfl_up_sync(0xffffffffu, ti, o);
        if (lane >= o) ti += d;
      }
      uint32_t before = tb + ti - t;
      tb += __shfl_sync(0xffffffffu, ti, 31);
#pragma unroll
      for (int q = 0; q < N; ++q) {
        w[q] = kept(x.f[q]);
        if (x.f[q] == x_t) {
          if (tie_ok && before < ties) w[q] = unit_t;
          ++before;
        }
        v += w[q];
      }
      const u64 vi = warp_scan(v, lane);
      const uint32_t over = __ballot_sync(0xffffffffu, run + vi > target);
      if (over) {
        if (lane == __ffs(over) - 1) {
          run += vi - v;
          bool found = false;
#pragma unroll
          for (int q = 0; q < N; ++q) {
            run += w[q];
            if (!found && run > target) {
              found = true;
              a.ids[row] = first + i * N + q;
              if (a.logprob != nullptr) a.logprob[row] = logf((float)w[q] / (float)S);
            }
          }
        }
        break;
      }
      run += __shfl_sync(0xffffffffu, vi, 31);
    }
  }
}

}  // namespace
}  // namespace pmoe

using namespace pmoe;

extern "C" int moe_sample_tokens(const void* logits, int is_bf16, int T, int V, int64_t row_stride,
                                 const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                                 const float* u, int32_t* ids_out, float* logprob_out, void* stream) {
  if (T < 0 || V < 1 || V > kMaxVocab || row_stride < V) return PMOE_EINVAL;
  if (T == 0) return PMOE_OK;
  if (logits == nullptr || u == nullptr || ids_out == nullptr) return PMOE_EINVAL;
  auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (off(logits, is_bf16 ? 2 : 4) || off(temperature, 4) || off(top_k, 4) || off(top_p, 4) || off(min_p, 4) || off(u, 4) ||
      off(ids_out, 4) || off(logprob_out, 4))
    return PMOE_EINVAL;
  // CTAs of a row: one up to 4,096 logits (a row of 3,000 8.5 us, 9.3 with 2), else slices of up
  // to 2,048, 8 CTAs at most (a row of 8,000 6.4 with 4, 6.9 with 2). With more than 200 CTAs
  // (clusters of 8 do not all find room) a CTA's fixed steps cost more than its share of the row:
  // slices of up to 8,192, and beyond 608 CTAs of up to 80 KB (two fit an SM). But a row that
  // needs step 3 takes the longer the fewer CTAs it has. In us, with settings of all kinds, 8 / 4 / 2 / 1 CTAs a row:
  // 30 rows of 32,000 16.5 / 16.3 / 23.4 / 29.6; 60 of 8,000 16.8 / 11.9 / 10.3 / 10.8; 150 of 5,000
  // 43.8 / 19.5 / 13.4 / 11.7; 256 of 32,000 62 / 43 / 36 / 40, of 50,001 72 / 51 / 56; bf16 rows of
  // 131,072: 256 of them 90 / 75, 64 of them 29.5 / 33.1.
  int cluster = 1;
  const int64_t rows = T, bytes = (int64_t)V * (is_bf16 ? 2 : 4);
  while (cluster < kMaxCluster && V > cluster * 2048 && V > 4096) cluster *= 2;
  while (cluster > 1 && rows * cluster > 200 && 2 * V <= cluster * 8192) cluster /= 2;
  while (cluster > 1 && rows * cluster > 608 && 2 * bytes <= (int64_t)cluster * 81920) cluster /= 2;
  if ((int64_t)T * cluster > INT32_MAX) return PMOE_EINVAL;
  SampleArgs a{logits, T, V, row_stride, temperature, top_k, top_p, min_p, u, ids_out, logprob_out, 0};
  // 7: the most elements by which a row can start after its first 16-byte vector
  a.slice = (((V + 7 + cluster - 1) / cluster) + 7) & ~7;
  const int smem = a.slice * (is_bf16 ? 2 : 4);
  const auto kernel = is_bf16 ? sample_kernel<true> : sample_kernel<false>;
  static SmemLimit limit[2];
  const int r = limit[is_bf16 ? 1 : 0].set(reinterpret_cast<const void*>(kernel), kMaxSmem, "moe_sample_tokens");
  if (r != PMOE_OK) return r;
  return launch("moe_sample_tokens", kernel, (unsigned)(T * cluster), kThreads, smem, (cudaStream_t)stream, true, cluster, a);
}
