// moe_router_select: the choice of experts by scores with a balance bias and expert groups.
//
// s_e = softmax or sigmoid of the logits; c_e = s_e + bias_e decides, s_e weighs. Of equal groups of
// neighbouring experts the best by the sum of their one or two largest c are kept, and in them the
// top_k largest c, ties to the lower id.
//
// Which expert is chosen must not hang on how an exponential is rounded, so the order is that of c in
// exact arithmetic: c is computed in fp32 to within a known bound, and where two that have to be told
// apart lie closer than that, the token is done again in fp64. Where there is no bias the order is
// the logits' own.
//
// Bound: issue slots, 0.65 of them in use: 16,384 tokens of 256 experts in 8 groups 21.9 us (sigmoid and bias, 852 instructions a
// token; their logits take 2.7 us to read), 4 tokens 3.4 us. Softmax with a bias 51 us, 56 with the groups: one token in a
// thousand is done in fp64, which takes 30 us. Where many c are equal, as with bf16 logits and no other bias than 0, every third token
// is: sigmoid 34 us, softmax 304 to 324. A warp a token, lane l with the logits l N .. l N + N - 1, so that a group of whole
// lanes is compared by shuffles, that of equal values the lowest lane's is the lowest id's, and a row is read
// in whole vectors; the bias stays in registers from token to token. The largest value of the warp is an
// integer maximum over keys that order like the floats.
#include "pmoe_internal.h"

#include <algorithm>
#include <math.h>

namespace pmoe {
namespace {

constexpr int kWarps = 8;  // tokens of a block

struct SelectArgs {
  const void* logits;
  int64_t row_stride;
  int T, E, top_k, sigmoid;
  const float* bias;
  int groups, top_groups, group_top, renorm;
  float scale;
  int32_t* ids;
  float* w;
  int size;   // experts of a group
  int lanes;  // of a group, where it is a power of two of whole lanes; else 0
  int shift;  // log2 of the lanes that work on a group
};

// Keys that order like the values; 0 stands below all of them.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);  // (-0 like 0)
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
__device__ __forceinline__ uint64_t key_of(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t k) { return __reduce_max_sync(0xffffffffu, k); }
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

// A row's logit: NaN counts as -inf.
template <bool BF16>
__device__ __forceinline__ float logit(const SelectArgs& a, int64_t row, int e) {
  float x;
  if constexpr (BF16)
    x = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(a.logits) + row + e) << 16);
  else
    x = __ldg(static_cast<const float*>(a.logits) + row + e);
  return x != x ? -INFINITY : x;
}

// One token in fp64, by one warp. choice: E values of this warp's in shared memory (where there are groups).
template <bool BF16>
__device__ __noinline__ void select_in_64_bits(const SelectArgs& a, int t, double* choice) {
  const int lane = threadIdx.x & 31;
  const int64_t row = t * a.row_stride;
  // lane l takes experts l + 32 i; their keys are worked out again for every pass, which is seldom
  float top = -INFINITY;
  for (int e = lane; e < a.E; e += 32) top = fmaxf(top, logit<BF16>(a, row, e));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  double sum = 0;
  if (!a.sigmoid) {
    for (int e = lane; e < a.E; e += 32) {
      const float x = logit<BF16>(a, row, e);
      sum += x == top ? 1. : exp((double)x - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  auto score = [&](float x) { return a.sigmoid ? 1. / (1. + exp(-(double)x)) : (x == top ? 1. : exp((double)x - top)) / sum; };
  for (int e = lane; e < a.E; e += 32) {
    const float x = logit<BF16>(a, row, e);
    double c = a.bias == nullptr && a.group_top == 1 ? x : score(x);
    if (a.bias != nullptr) c += a.bias[e];
    choice[e] = c != c ? -INFINITY : c;
  }
  __syncwarp();
  uint32_t kept = ~0u;
  const int size = a.E / a.groups;
  if (a.groups > 1) {
    double value = -INFINITY;  // lane g: of group g
    if (lane < a.groups) {
      double m1 = -INFINITY, m2 = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const double c = choice[lane * size + i];
        if (c > m1)
          m2 = m1, m1 = c;
        else if (c > m2)
          m2 = c;
      }
      value = a.group_top > 1 && size > 1 ? m1 + m2 : m1;
      if (value != value) value = -INFINITY;  // infinities of both signs
    }
    int rank = 0;
    for (int k = 0; k < a.groups; ++k) {
      const double other = __shfl_sync(0xffffffffu, value, k);
      if (other > value || (other == value && k < lane)) ++rank;
    }
    kept = __ballot_sync(0xffffffffu, lane < a.groups && rank < a.top_groups);
  }
  // (the logits themselves decide where there is no bias)
  auto key = [&](int e) -> uint64_t {
    if (a.groups > 1 && !(kept >> (e / size) & 1)) return 0;
    return key_of(a.bias != nullptr ? choice[e] : (double)logit<BF16>(a, row, e));
  };
  uint64_t bound = ~0ull;  // the last one taken: key and id
  int bound_id = -1, id = 0;
  for (int r = 0; r < a.top_k; ++r) {
    uint64_t best = 0;
    int at = 0x7fffffff;
    for (int e = lane; e < a.E; e += 32) {
      const uint64_t k = key(e);
      if (k > best && (k < bound || (k == bound && e > bound_id))) best = k, at = e;
    }
    const uint64_t all = warp_max(best);
    at = (int)__reduce_min_sync(0xffffffffu, (uint32_t)(best == all ? at : 0x7fffffff));
    bound = all, bound_id = at;
    if (lane == r) id = at;
  }
  const double s = lane < a.top_k ? score(logit<BF16>(a, row, id)) : 0.;
  double w = s;
  if (a.renorm) {
    double total = s;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    w = total > 0 ? s / total : 0.;
  }
  if (lane < a.top_k) {
    a.ids[(int64_t)t * a.top_k + lane] = id;
    a.w[(int64_t)t * a.top_k + lane] = (float)(w * a.scale);
  }
  __syncwarp();
}

// c of expert e in fp64, with sigmoid scores.
template <bool BF16>
__device__ __forceinline__ double exact_choice(const SelectArgs& a, int64_t row, int e) {
  double c = 1. / (1. + exp(-(double)logit<BF16>(a, row, e)));
  if (a.bias != nullptr) c += a.bias[e];
  return c != c ? -INFINITY : c;
}

// Batcher's odd-even merge sort: runs of P are merged, first by comparisons K apart. (By templates: nested
// loops are not unrolled for 16 values and more, and the keys then lie in local memory: 16,384 tokens of 512 experts
// 53.8 us, so 44.6; with the sums in a tree 32.8.)
template <int N, int P, int K>
__device__ __forceinline__ void merge_descending(uint32_t (&v)[N]) {
#pragma unroll
  for (int i = K % P; i + K < N; ++i)
    if ((i - K % P) / K % 2 == 0 && i / (2 * P) == (i + K) / (2 * P)) {
      const uint32_t x = v[i], y = v[i + K];
      v[i] = max(x, y);
      v[i + K] = min(x, y);
    }
  if constexpr (K > 1)
    merge_descending<N, P, K / 2>(v);
  else if constexpr (2 * P < N)
    merge_descending<N, 2 * P, 2 * P>(v);
}
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[N]) {
  if constexpr (N > 1) merge_descending<N, 1, 1>(v);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269504f;
// Sum in a tree, so that no term takes more than log2 N roundings.
template <int I, int N, int M>
__device__ __forceinline__ float sum_of(const float (&t)[M]) {
  if constexpr (N == 1)
    return t[I];
  else
    return sum_of<I, N / 2>(t) + sum_of<I + N / 2, N - N / 2>(t);
}

// N values of a row from element i on; beyond `n` and NaN: -inf. VEC: whole vectors.
template <int N, bool BF16, bool VEC>
__device__ __forceinline__ void load_row(const void* p, int64_t row, int i, int n, float (&x)[N]) {
  if constexpr (VEC && BF16 && N % 2 == 0) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p) + row + i);
    uint32_t v[N / 2];
    if constexpr (N % 8 == 0) {
#pragma unroll
      for (int k = 0; k < N / 8; ++k) *reinterpret_cast<uint4*>(v + 4 * k) = __ldg(reinterpret_cast<const uint4*>(w) + k);
    } else {
#pragma unroll
      for (int k = 0; k < N / 2; ++k) v[k] = __ldg(w + k);
    }
#pragma unroll
    for (int k = 0; k < N / 2; ++k) x[2 * k] = __uint_as_float(v[k] << 16), x[2 * k + 1] = __uint_as_float(v[k] & 0xffff0000u);
  } else if constexpr (VEC && !BF16 && N % 4 == 0) {
    const float4* w = reinterpret_cast<const float4*>(static_cast<const float*>(p) + row + i);
#pragma unroll
    for (int k = 0; k < N / 4; ++k) {
      const float4 f = __ldg(w + k);
      x[4 * k] = f.x, x[4 * k + 1] = f.y, x[4 * k + 2] = f.z, x[4 * k + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      x[k] = -INFINITY;
      if (i + k < n) {
        if constexpr (BF16)
          x[k] = __uint_as_float((uint32_t)__ldg(static_cast<const uint16_t*>(p) + row + i + k) << 16);
        else
          x[k] = __ldg(static_cast<const float*>(p) + row + i + k);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) x[k] = fmaxf(x[k], -INFINITY);  // (NaN: the other operand)
}

// One token in fp32 by one warp; false: not sure. bias: this lane's. choice [E] and lane_keys [32 N], one after the
// other in the same place, and list [33]: of this warp, in shared memory.
template <int N, bool BF16, bool VEC>
__device__ __forceinline__ bool select_token(const SelectArgs& a, int t, const float (&bias)[N], float* choice, uint32_t* lane_keys,
                                             uint2* list) {
  const int lane = threadIdx.x & 31;
  const int64_t row = t * a.row_stride;
  float x[N];
  load_row<N, BF16, VEC>(a.logits, row, lane * N, a.E, x);
  // softmax: the largest logit and 1 / the sum of the exponentials. Logits of +inf, or all of -inf, share the row.
  float top = 0.f, inv = 1.f;
  if (!a.sigmoid) {
    top = x[0];
#pragma unroll
    for (int k = 1; k < N; ++k) top = fmaxf(top, x[k]);
    top = value_of(warp_max(key_of(top)));
    float term[N];
#pragma unroll
    for (int k = 0; k < N; ++k) term[k] = lane * N + k >= a.E ? 0.f : x[k] == top ? 1.f : ex2((x[k] - top) * kLog2e);
    float sum = sum_of<0, N>(term);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv = 1.f / sum;
  }
  auto score = [&](float v) {
    if (a.sigmoid) return rcp(1.f + ex2(fmaxf(v, -200.f) * -kLog2e));
    return v == top ? inv : ex2((v - top) * kLog2e) * inv;
  };
  // The same for the weights, to within a few units in the last place of the exponential (and the sum's error):
  // `score` is off by 2^-23 |argument| of itself, 2^-17 where all logits of a row's choice are as low as -60.
  auto fine_score = [&](float v) {
    if (a.sigmoid) return __fdividef(1.f, 1.f + expf(-v));
    if (v == top) return inv;
    const float d = v - top, back = d - v, rest = (v - (d - back)) - (top + back);  // v - top = d + rest
    if (!(d > -104.f)) return 0.f;
    const float e = expf(d);
    return fmaf(e, rest, e) * inv;
  };
  // What a score may be off by, with u = 2^-24. Sigmoid: the exponential 4 u, its argument |x| 1.23 u, of which s (1 - s)
  // <= 1/4 and |x| s (1 - s) <= 0.23 reach s; sum and reciprocal 3 u: 5 u. Softmax: of the row's sum the terms 4 u, their
  // arguments 2.23 u times a mean of |x - top|, which is at most log(1024) = 7, and 10 u of adding in a tree; division, own
  // exponential and product 6 u: 36 u of the score, which is at most the largest one's, inv. It is the row's largest
  // that counts for all: an expert of a large score may stand among ones of small scores by its bias.
  const float score_error = a.sigmoid ? 3.5e-7f : 2.2e-6f * inv;
  // c and d, which two scores are in, may be the other way round (2^-24 of each by its own rounding)
  auto unsure = [&](float c, float d) { return !(c - d > 2.f * score_error + 1.1920929e-7f * (fabsf(c) + fabsf(d))); };

  // ---- what decides: c, or without a bias the logits themselves
  const bool by_logits = a.bias == nullptr, scored = !by_logits || (a.groups > 1 && a.group_top > 1);
  uint32_t key[N], group_key[N];
  auto there = [&](int k) { return VEC || lane * N + k < a.E; };
  if (!scored) {
#pragma unroll
    for (int k = 0; k < N; ++k) key[k] = group_key[k] = there(k) ? key_of(x[k]) : 0;
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) key[k] = group_key[k] = there(k) ? key_of(fmaxf(score(x[k]) + bias[k], -INFINITY)) : 0;
    if (by_logits) {
#pragma unroll
      for (int k = 0; k < N; ++k) key[k] = there(k) ? key_of(x[k]) : 0;
    }
  }

  // ---- the groups
  if (a.groups > 1) {
    const int size = a.size, per = 1 << a.shift, g = lane >> a.shift;  // this lane's group, lanes of a group
    uint32_t m1 = 0, m2 = 0;                                           // the two largest of a group
    if (a.lanes > 0) {  // groups of whole lanes, a power of two of them
#pragma unroll
      for (int k = 0; k < N; ++k) {
        m2 = max(m2, min(m1, group_key[k]));
        m1 = max(m1, group_key[k]);
      }
    } else {  // by way of shared memory
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (lane * N + k < a.E) choice[lane * N + k] = value_of(group_key[k]);
      __syncwarp();
      if (g < a.groups)
        for (int i = lane & (per - 1); i < size; i += per) {
          const uint32_t c = key_of(choice[g * size + i]);
          m2 = max(m2, min(m1, c));
          m1 = max(m1, c);
        }
      __syncwarp();
    }
    for (int o = 1; o < per; o <<= 1) {
      const uint32_t n1 = __shfl_xor_sync(0xffffffffu, m1, o), n2 = __shfl_xor_sync(0xffffffffu, m2, o);
      m2 = max(min(m1, n1), max(m2, n2));
      m1 = max(m1, n1);
    }
    const bool pairs = a.group_top > 1 && size > 1;
    float value = pairs ? value_of(m1) + value_of(m2) : value_of(m1);
    value = fmaxf(value, -INFINITY);  // (infinities of both signs)
    int rank = 0;  // of equal groups the first is better
    const uint32_t mark = key_of(value);
#pragma unroll 4
    for (int k = 0; k < a.groups; ++k) {
      const uint32_t other = __shfl_sync(0xffffffffu, mark, k << a.shift);
      rank += other >= mark + (k < g ? 0 : 1);
    }
    bool in = g < a.groups && rank < a.top_groups;
    if (scored) {
      // What each value may be off by: two scores, and 2^-24 of either c, of their sum and of
      // the bounds. The c of a group may cancel, so the sum says nothing of their own errors. All that is
      // kept has to lie above all that is not. (-inf is exact or below what fp32 holds.)
      const float spread = 2.f * score_error + 2.3841858e-7f * (fabsf(value_of(m1)) + (pairs ? fabsf(value_of(m2)) : 0.f));
      const float low = fmaxf(value - spread, -INFINITY), high = value == -INFINITY ? value : value + spread;
      const uint32_t worst = ~warp_max(in ? ~key_of(low) : 0u), best = warp_max(g < a.groups && !in ? key_of(high) : 0u);
      if (!(value_of(worst) > value_of(best))) {
        if (!a.sigmoid) return false;
        // each group's two largest in fp64: those that come near its second, one a lane
        const float near = value_of(m2) - 1.5e-6f - 2.5e-7f * fabsf(value_of(m2));
        int n = 0;
#pragma unroll 1
        for (int k = 0; k < N; ++k) {
          float c = 0.f;
          int group = -1;
          const int e = lane * N + k;
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (j == k) c = value_of(group_key[j]);
          if (e < a.E) group = e / size;
          const float bound = __shfl_sync(0xffffffffu, near, max(group, 0) << a.shift);
          const uint32_t takes = __ballot_sync(0xffffffffu, group >= 0 && !(c < bound));
          const int at = n + __popc(takes & ((1u << lane) - 1));
          if (takes >> lane & 1 && at < 32) list[at].y = e;
          n += __popc(takes);
        }
        __syncwarp();
        if (n > 32) return false;
        const int e = lane < n ? list[lane].y : 0, group = lane < n ? e / size : -1;
        const double c = exact_choice<BF16>(a, row, e);
        double d1 = -INFINITY, d2 = -INFINITY;  // lane i: of group i
#pragma unroll 1
        for (int k = 0; k < n; ++k) {
          const double other = __shfl_sync(0xffffffffu, c, k);
          if (__shfl_sync(0xffffffffu, group, k) == lane) {
            if (other > d1)
              d2 = d1, d1 = other;
            else if (other > d2)
              d2 = other;
          }
        }
        double sum = pairs ? d1 + d2 : d1;
        if (sum != sum) sum = -INFINITY;
        int place = 0;
#pragma unroll 1
        for (int k = 0; k < a.groups; ++k) {
          const double other = __shfl_sync(0xffffffffu, sum, k);
          place += other > sum || (other == sum && k < lane);
        }
        const uint32_t best_groups = __ballot_sync(0xffffffffu, lane < a.groups && place < a.top_groups);
        in = g < a.groups && (best_groups >> g & 1);
        __syncwarp();
      }
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, in);
    if (a.lanes > 0) {
      if (!in) {
#pragma unroll
        for (int k = 0; k < N; ++k) key[k] = 0;
      }
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (lane * N + k < a.E && !(kept >> ((lane * N + k) / size * per) & 1)) key[k] = 0;
    }
  }

  // ---- the top_k largest, and with scores one more to see how sure the last is
  const bool check = !by_logits;
  const int rounds = a.top_k + (check ? 1 : 0);
  // a lane's keys in descending order, its largest against the other lanes'; which expert a key is of is
  // looked up at the end
#pragma unroll
  for (int k = 0; k < N; ++k) lane_keys[lane * N + k] = key[k];
  sort_descending<N>(key);
  uint32_t last = 0;
  int n = 0;  // of the list
  auto take = [&]() {
    last = warp_max(key[0]);
    const int from = __ffs(__ballot_sync(0xffffffffu, key[0] == last)) - 1;  // (of equal ones the lowest lane)
    if (lane == from) {
      list[n] = make_uint2(last, lane);
#pragma unroll
      for (int k = 0; k + 1 < N; ++k) key[k] = key[k + 1];
      key[N - 1] = 0;
    }
    ++n;
  };
#pragma unroll 1
  while (n < rounds) take();
  uint2 mine;
  float s, c;
  int id;
  auto look = [&]() {  // lane i: the i-th of the list
    __syncwarp();
    mine = lane < n ? list[lane] : make_uint2(0, lane);
    // of equal keys of one lane the first is the lower id's
    const uint32_t same = __match_any_sync(0xffffffffu, (uint64_t)mine.y << 32 | mine.x);
    int skip = __popc(same & ((1u << lane) - 1));
    id = 0;
    const uint32_t* keys = lane_keys + mine.y * N;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const bool hit = keys[k] == mine.x;
      if (hit && skip-- == 0) id = mine.y * N + k;
    }
    s = mine.x != 0 ? fine_score(logit<BF16>(a, row, id)) : 0.f;
    c = value_of(mine.x);
  };
  look();
  if (check) {
    // neighbours in the order, the last against the one after it
    float d = __shfl_down_sync(0xffffffffu, c, 1);
    if (lane == 31) d = value_of(last);  // (of 33)
    const bool pair = lane + 1 < a.top_k || (lane + 1 == a.top_k && last != 0);
    if (__any_sync(0xffffffffu, pair && unsure(c, d))) {
      if (!a.sigmoid || a.top_k > 30) return false;
      // the list in fp64, and with it all that come near its end; one a lane, sorted by rank
      float end = __shfl_sync(0xffffffffu, c, a.top_k - 1);
      end -= 1.5e-6f + 2.5e-7f * fabsf(end);
      while (n < 32 && last != 0 && !(value_of(last) < end)) take();
      if (n == 32) return false;
      look();
      const bool there = mine.x != 0;
      const double exact = there ? exact_choice<BF16>(a, row, id) : 0.;
      int place = 0;
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const double other = __shfl_sync(0xffffffffu, exact, k);
        const int other_id = __shfl_sync(0xffffffffu, id, k), other_there = __shfl_sync(0xffffffffu, (int)there, k);
        place += other_there && (other > exact || (other == exact && other_id < id));
      }
      __syncwarp();
      if (there && place < a.top_k) list[place] = make_uint2(__float_as_uint(s), id);
      __syncwarp();
      if (lane < a.top_k) s = __uint_as_float(list[lane].x), id = list[lane].y;
    }
  }
  __syncwarp();  // list may be written for the next token
  float w = s;
  if (a.renorm) {
    float sum = lane < a.top_k ? s : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (sum < 1e-30f) return false;  // scores that fp32 does not hold
    w = __fdividef(s, sum);
  }
  if (lane < a.top_k) {
    a.ids[(int64_t)t * a.top_k + lane] = id;
    a.w[(int64_t)t * a.top_k + lane] = w * a.scale;
  }
  return true;
}

template <int N, bool BF16, bool VEC>
__global__ void __launch_bounds__(kWarps * 32) select_kernel(const SelectArgs a) {
  extern __shared__ double choices[];  // [kWarps][32 N]
  __shared__ uint2 lists[kWarps][kMaxTopK + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  float bias[N];
#pragma unroll
  for (int k = 0; k < N; ++k) bias[k] = a.bias != nullptr && lane * N + k < a.E ? __ldg(a.bias + lane * N + k) : 0.f;
  double* mine = choices + (size_t)warp * 32 * N;
  for (int t = blockIdx.x * kWarps + warp; t < a.T; t += gridDim.x * kWarps)
    if (!select_token<N, BF16, VEC>(a, t, bias, reinterpret_cast<float*>(mine), reinterpret_cast<uint32_t*>(mine),
                                     lists[warp])) select_in_64_bits<BF16>(a, t, mine);
}

template <int N, bool BF16, bool VEC>
int launch_one(SelectArgs a, cudaStream_t s) {
  const char* what = "moe_router_select";
  static SmemLimit limit;
  a.size = a.E / a.groups;
  a.lanes = a.size % N == 0 && (a.size / N & (a.size / N - 1)) == 0 ? a.size / N : 0;
  a.shift = 0;
  while (a.lanes > 0 ? 1 << a.shift < a.lanes : a.groups << (a.shift + 1) <= 32) ++a.shift;
  const auto kernel = select_kernel<N, BF16, VEC>;
  const int r = limit.set(reinterpret_cast<const void*>(kernel), kWarps * N * 32 * 8, what);
  // one wave of blocks on the GB300's 152 SMs: four an SM by registers, two with 16 keys a lane (16,384 tokens of 512
  // experts 32.8 us, 35.6 with four)
  const unsigned blocks = (unsigned)std::min((a.T + kWarps - 1) / kWarps, 152 * (N < 16 ? 4 : 2));
  return r != PMOE_OK ? r : launch(what, kernel, blocks, kWarps * 32, kWarps * N * 32 * 8, s, true, 1, a);
}

// A lane takes 2^n experts; of 96, 160, 192 and 384 experts, in rows that are aligned for it, exactly E / 32: fewer keys to
// sort, and of 160 experts in 8 groups four lanes hold a group, while of 8 a lane no whole ones do. 16,384 tokens, so and with
// 2^n: 96 experts 15.2 and 16.3 us, 160 21.2 and 29.3, 192 18.2 and 18.3, 384 20.5 and 33.4. Other multiples of 32 take 2^n.
template <bool BF16>
int launch_select(SelectArgs a, cudaStream_t s) {
  if (reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.row_stride * (BF16 ? 2 : 4) % 16 == 0) {
    switch (a.E) {
      case 32: return launch_one<1, BF16, true>(a, s);
      case 64: return launch_one<2, BF16, true>(a, s);
      case 96: return launch_one<3, BF16, true>(a, s);
      case 128: return launch_one<4, BF16, true>(a, s);
      case 160: return launch_one<5, BF16, true>(a, s);
      case 192: return launch_one<6, BF16, true>(a, s);
      case 256: return launch_one<8, BF16, true>(a, s);
      case 384: return launch_one<12, BF16, true>(a, s);
      case 512: return launch_one<16, BF16, true>(a, s);
      case 1024: return launch_one<32, BF16, true>(a, s);
    }
  }
  const int npl = (a.E + 31) / 32;
  if (npl <= 1) return launch_one<1, BF16, false>(a, s);
  if (npl <= 2) return launch_one<2, BF16, false>(a, s);
  if (npl <= 4) return launch_one<4, BF16, false>(a, s);
  if (npl <= 8) return launch_one<8, BF16, false>(a, s);
  if (npl <= 16) return launch_one<16, BF16, false>(a, s);
  return launch_one<32, BF16, false>(a, s);
}

}  // namespace
}  // namespace pmoe

using namespace pmoe;

extern "C" int moe_router_select(const void* logits, int is_bf16, int T, int E, int64_t row_stride, int top_k, int scoring,
                                 const float* bias, int groups, int top_groups, int group_top, int renormalize, float scale,
                                 int32_t* ids_out, float* w_out, void* stream) {
  if (T < 0 || E < 1 || E > kMaxExperts || top_k < 1 || top_k > kMaxTopK || top_k > E || row_stride < E) return PMOE_EINVAL;
  if (scoring != PMOE_SCORE_SOFTMAX && scoring != PMOE_SCORE_SIGMOID) return PMOE_EINVAL;
  if (groups < 1 || groups > 32 || E % groups != 0 || top_groups < 1 || top_groups > groups || group_top < 1 || group_top > 2 ||
      top_k > E / groups * top_groups || !(fabsf(scale) < INFINITY))
    return PMOE_EINVAL;
  if (T == 0) return PMOE_OK;
  auto off = [](const void* p, size_t n) { return p == nullptr || reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (off(logits, is_bf16 ? 2 : 4) || (bias != nullptr && off(bias, 4)) || off(ids_out, 4) || off(w_out, 4)) return PMOE_EINVAL;
  const bool grouped = groups > 1 && top_groups < groups;  // all groups kept: no choice among them
  const SelectArgs a{logits, row_stride, T, E, top_k, scoring == PMOE_SCORE_SIGMOID, bias, grouped ? groups : 1,
                     grouped ? top_groups : 1, E / groups > 1 ? group_top : 1, renormalize != 0, scale, ids_out, w_out, 0, 0, 0};
  return is_bf16 ? launch_select<true>(a, (cudaStream_t)stream) : launch_select<false>(a, (cudaStream_t)stream);
}
