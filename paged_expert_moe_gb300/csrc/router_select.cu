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
// Bound: issue slots; a warp a token, its logits in registers, lane l experts l + 32 i. The largest
// of the warp is found by integer maxima over keys that order like the floats.
#include "pmoe_internal.h"

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

// e^x within 2^-21 of its value, x <= 88; below -87: 0
__device__ __forceinline__ float exp_of(float x) {
  constexpr float kL = 1.44269504088896f, kRest = 1.92596299e-8f;  // log2(e) and what its float leaves
  const float y = x * kL, rest = fmaf(x, kRest, fmaf(x, kL, -y));
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return x < -87.f ? 0.f : fmaf(r, rest * 0.693147181f, r);
}
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

__device__ __forceinline__ float sigmoid(float x) { return x < -87.f ? 0.f : 1.f / (1.f + exp_of(fmaxf(-x, -88.f))); }
__device__ __forceinline__ double sigmoid(double x) { return 1. / (1. + exp(-x)); }

template <class F>
struct KeyOf;
template <>
struct KeyOf<float> {
  using T = uint32_t;
};
template <>
struct KeyOf<double> {
  using T = uint64_t;
};

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

// Whether c, of score s, may be no larger than d, of score t, given what both may be off by in fp32:
// sigmoid: 2^-20 of the scores (the exponential 2^-21.5, its sum with 1 and the division 2^-24 each);
// softmax: 2^-18 (a sum of up to 32 values a lane and 5 exchanges, 2^-24 each); and the sum with the
// bias, 2^-24 of c and of d.
__device__ __forceinline__ bool unsure(const SelectArgs& a, float c, float s, float d, float t) {
  return !(c - d > (a.sigmoid ? 9.5367432e-7f : 3.8146973e-6f) * (s + t) + 1.1920929e-7f * (fabsf(c) + fabsf(d)));
}

// One token by one warp, in arithmetic F. False: done again in fp64. choice: E values of this warp's
// in shared memory (groups > 1 only).
template <class F, int NPL, bool BF16>
__device__ __forceinline__ bool select_token(const SelectArgs& a, int t, F* choice) {
  using Key = typename KeyOf<F>::T;
  const int lane = threadIdx.x & 31;
  const int64_t row = t * a.row_stride;
  float x[NPL];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 32 * i;
    x[i] = e < a.E ? logit<BF16>(a, row, e) : -INFINITY;
    top = fmaxf(top, x[i]);
  }
  F inv = 1;  // softmax: 1 / sum
  if (!a.sigmoid) {
    top = value_of(warp_max(key_of(top)));
    F sum = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)  // (logits of +inf, or all of -inf, share the row)
      if (lane + 32 * i < a.E) sum += x[i] == top ? (F)1 : exp_of((F)x[i] - (F)top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    inv = (F)1 / sum;
  }
  auto score = [&](float v) -> F {
    if (a.sigmoid) return sigmoid((F)v);
    return v == top ? inv : exp_of((F)v - (F)top) * inv;
  };

  // ---- what decides: c, or the logits themselves
  const bool by_logits = a.bias == nullptr;
  Key key[NPL];
  if (!by_logits || (a.groups > 1 && a.group_top > 1)) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      key[i] = 0;
      if (e < a.E) {
        F c = score(x[i]);
        if (!by_logits) {
          const float bias = __ldg(a.bias + e);
          c += bias;
          if (c != c) c = -INFINITY;
        }
        key[i] = key_of(by_logits ? (F)x[i] : c);
        if (a.groups > 1) choice[e] = c;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      key[i] = e < a.E ? key_of((F)x[i]) : 0;
      if (a.groups > 1 && e < a.E) choice[e] = x[i];
    }
  }

  // ---- the groups: 32 / 2^ceil(log2 groups) lanes each
  if (a.groups > 1) {
    __syncwarp();
    int per = 32;
    while (per * a.groups > 32) per >>= 1;
    const int g = lane / per, size = a.E / a.groups;
    F m1 = -INFINITY, m2 = -INFINITY;  // the group's largest two
    bool one = false;
    if (g < a.groups) {
      one = size == 1;
      for (int i = lane % per; i < size; i += per) {
        const F c = choice[g * size + i];
        if (c > m1)
          m2 = m1, m1 = c;
        else if (c > m2)
          m2 = c;
      }
    }
    for (int o = 1; o < per; o <<= 1) {
      const F n1 = __shfl_xor_sync(0xffffffffu, m1, o), n2 = __shfl_xor_sync(0xffffffffu, m2, o);
      m2 = fmax(fmin(m1, n1), fmax(m2, n2));
      m1 = fmax(m1, n1);
    }
    F value = a.group_top > 1 && !one ? m1 + m2 : m1;
    if (value != value) value = -INFINITY;  // infinities of both signs
    // its rank among the groups; of equal ones the first is better
    int rank = 0;
    for (int k = 0; k < a.groups; ++k) {
      const F other = __shfl_sync(0xffffffffu, value, k * per);
      if (other > value || (other == value && k < g)) ++rank;
    }
    const bool in = g < a.groups && rank < a.top_groups;
    if (sizeof(F) == 4 && !(by_logits && a.group_top == 1)) {
      // the worst that is kept against the best that is not, as sums of two scores of at most 1
      const uint32_t worst = ~warp_max(in ? ~key_of((float)value) : 0u);
      const uint32_t best = warp_max(g < a.groups && !in ? key_of((float)value) : 0u);
      if (best != 0) {
        if (unsure(a, value_of(worst), 2.f, value_of(best), 2.f)) return false;
      }
    }
    const uint32_t kept = __ballot_sync(0xffffffffu, in);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && !(kept >> (e / size * per) & 1)) key[i] = 0;
    }
    __syncwarp();  // choice may be written for the next token
  }

  // ---- the top_k largest, one more to see how sure the last is; lane r keeps the r-th
  Key mine = 0;
  int id = 0;
  const bool check = sizeof(F) == 4 && !by_logits;
  const int rounds = a.top_k + (check ? 1 : 0);
  Key last = 0;
  for (int r = 0; r < rounds; ++r) {
    Key best = 0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) best = key[i] > best ? key[i] : best;
    const Key all = warp_max(best);
    int e = 0x7fffffff;
    if (best == all) {
#pragma unroll
      for (int i = NPL - 1; i >= 0; --i)
        if (key[i] == all) e = lane + 32 * i;
    }
    e = (int)__reduce_min_sync(0xffffffffu, (uint32_t)e);
    if ((e & 31) == lane) {
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if (e == lane + 32 * i) key[i] = 0;
    }
    if (lane == r) mine = all, id = e;
    last = all;
  }
  const F s = lane < rounds && mine != 0 ? score(logit<BF16>(a, row, id)) : (F)0;
  if (check) {
    // neighbours in the order, the last against the one after it
    const float c = value_of((uint32_t)mine);
    float d = __shfl_down_sync(0xffffffffu, c, 1), u = __shfl_down_sync(0xffffffffu, (float)s, 1);
    if (lane == 31) d = value_of((uint32_t)last), u = 1.f;  // (of 33; some score)
    const bool pair = lane + 1 < a.top_k || (lane + 1 == a.top_k && last != 0);
    if (__any_sync(0xffffffffu, pair && unsure(a, c, (float)s, d, u))) return false;
  }
  F w = s;
  if (a.renorm) {
    F sum = lane < a.top_k ? s : (F)0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (sizeof(F) == 4 && sum < 1e-30f) return false;  // scores that fp32 does not hold
    w = sum > 0 ? s / sum : (F)0;
  }
  if (lane < a.top_k) {
    a.ids[(int64_t)t * a.top_k + lane] = id;
    a.w[(int64_t)t * a.top_k + lane] = (float)(w * (F)a.scale);
  }
  return true;
}

template <int NPL, bool BF16>
__device__ __noinline__ void select_in_64_bits(const SelectArgs& a, int t, double* choice) {
  select_token<double, NPL, BF16>(a, t, choice);
}

template <int NPL, bool BF16>
__global__ void __launch_bounds__(kWarps * 32) select_kernel(const SelectArgs a) {
  extern __shared__ double choices[];  // [kWarps][E] where there are groups
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kWarps + warp;
  if (t >= a.T) return;
  double* mine = choices + (size_t)warp * a.E;
  if (!select_token<float, NPL, BF16>(a, t, reinterpret_cast<float*>(mine))) select_in_64_bits<NPL, BF16>(a, t, mine);
}

template <bool BF16>
int launch_select(const SelectArgs& a, cudaStream_t s) {
  const int npl = (a.E + 31) / 32;
  const unsigned blocks = (unsigned)((a.T + kWarps - 1) / kWarps);
  const size_t smem = a.groups > 1 ? (size_t)kWarps * a.E * 8 : 0;
#define PMOE_SELECT_CASE(N)                                                                                             \
  do {                                                                                                                  \
    static SmemLimit limit;                                                                                             \
    const int r = limit.set(reinterpret_cast<const void*>(select_kernel<N, BF16>), kWarps * N * 32 * 8, "moe_router_select"); \
    return r != PMOE_OK ? r                                                                                             \
                        : launch("moe_router_select", select_kernel<N, BF16>, blocks, kWarps * 32, smem, s, true, 1, a); \
  } while (0)
  if (npl <= 1) PMOE_SELECT_CASE(1);
  if (npl <= 2) PMOE_SELECT_CASE(2);
  if (npl <= 4) PMOE_SELECT_CASE(4);
  if (npl <= 8) PMOE_SELECT_CASE(8);
  if (npl <= 16) PMOE_SELECT_CASE(16);
  PMOE_SELECT_CASE(32);
#undef PMOE_SELECT_CASE
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
                     grouped ? top_groups : 1, group_top, renormalize != 0, scale, ids_out, w_out};
  return is_bf16 ? launch_select<true>(a, (cudaStream_t)stream) : launch_select<false>(a, (cudaStream_t)stream);
}
