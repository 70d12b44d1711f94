// moe_adjust_logits: penalties for repeated tokens, biases and grammar masks on logits.
//
// A row's history touches few of its V logits. Which, and how often each occurs, is counted in shared
// memory: a CTA takes a slice of the ids of one row, one word an id, and looks at the row's whole history,
// of which it counts what falls into its slice. Then the slice's logits go by once, four a thread with their
// four words. The counts are whole numbers, so their order does not matter.
//
// Bound: HBM, the logits read and written once, and the history's counting, in which a CTA waits for its
// atomics. The first logits and mask words are on their way meanwhile. 256 fp32 rows of 160,001 with 2,000 ids of
// history at most 70 us (50 without; a plain copy 56), 64 bf16 rows of 131,072 to fp32 with 4,000 20 us (10
// without; a copy 17, cold caches 27), one row 3.5 us. In place 62, 23 (a four that changes is read and written where it
// lies, after its counts are known, so nothing is on its way before) and 3.5 us.
#include "pmoe_internal.h"

#include <math.h>

namespace pmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kPerSM = 5;
constexpr int kInFlight = 4;  // fours of logits of a thread
constexpr int kMaxSlice = 2 * 4 * kInFlight * kThreads;
// A word of the table: times in the output (19 bits), in the prompt (1 bit), 1 + index of the bias (12 bits).
constexpr uint32_t kPrompt = 1u << 19, kCount = kPrompt - 1;
constexpr int kBiasShift = 20, kMaxBiases = 4095;

struct AdjustArgs {
  const void* logits;
  void* out;
  int64_t row_stride, out_stride;
  int T, V, in_place;
  const int32_t* history;
  int64_t history_stride;
  int max_history;
  const int32_t *prompt_len, *history_len;
  const float *repetition, *frequency, *presence;
  const int32_t* bias_ids;
  const float* bias;
  int biases;
  const uint32_t* mask;
  int64_t mask_stride;
  int32_t* err;
  int slice, slices;
};

template <bool BF16>
__device__ __forceinline__ float load1(const void* p, int64_t i) {
  if constexpr (BF16) return __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  return static_cast<const float*>(p)[i];
}
template <bool BF16>
__device__ __forceinline__ void store1(void* p, int64_t i, float v) {
  if constexpr (BF16)
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[i] = v;
}
// Four values as they lie in memory.
template <bool BF16>
struct Quad;
template <>
struct Quad<true> {
  uint2 u;
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = __uint_as_float(u.x << 16), v[1] = __uint_as_float(u.x & 0xffff0000u);
    v[2] = __uint_as_float(u.y << 16), v[3] = __uint_as_float(u.y & 0xffff0000u);
  }
};
template <>
struct Quad<false> {
  float4 f;
  __device__ __forceinline__ void get(float (&v)[4]) const { v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w; }
};
template <bool BF16>
__device__ __forceinline__ Quad<BF16> load4(const void* p, int64_t i) {
  if constexpr (BF16)
    return {*reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i)};
  else
    return {*reinterpret_cast<const float4*>(static_cast<const float*>(p) + i)};
}
template <bool BF16>
__device__ __forceinline__ void store4(void* p, int64_t i, const float (&v)[4]) {
  if constexpr (BF16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + i) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(p) + i) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// BI, BO: logits, out in bf16
template <bool BI, bool BO>
__global__ void __launch_bounds__(kThreads, kPerSM) adjust_kernel(const AdjustArgs a) {
  extern __shared__ __align__(16) uint32_t table[];  // [slice]
  pdl_wait();
  pdl_trigger();
  const int t = blockIdx.x / a.slices, part = blockIdx.x - t * a.slices, tid = threadIdx.x;
  const int v0 = part * a.slice, v1 = min(a.V, v0 + a.slice), n = v1 - v0;
  const int64_t in = t * a.row_stride, out = t * a.out_stride;
  const uint32_t* mask = a.mask != nullptr ? a.mask + t * a.mask_stride : nullptr;
  auto complain = [&](int32_t what) {
    if (a.err != nullptr && part == 0) atomicOr(a.err, what);
  };
  const float kOff = -INFINITY;
  const bool sparse = a.max_history > 0 || a.biases > 0;
  const float rep = a.repetition != nullptr ? a.repetition[t] : 1.f, freq = a.frequency != nullptr ? a.frequency[t] : 0.f,
              pres = a.presence != nullptr ? a.presence[t] : 0.f;
  auto adjusted = [&](float x, uint32_t e) {
    const uint32_t times = e & kCount;
    if (e & (kCount | kPrompt)) x = x > 0.f ? x / rep : x * rep;
    if (times > 0) x = x - freq * (float)times - pres;
    if (e >> kBiasShift) x += a.bias[(int64_t)t * a.biases + (e >> kBiasShift) - 1];
    return x;
  };
  // 4 logits at a time from where both rows are aligned; one by one where they are not alike
  const int ai = (int)((reinterpret_cast<uintptr_t>(a.logits) / (BI ? 2 : 4) + in) & 3);
  const int ao = (int)((reinterpret_cast<uintptr_t>(a.out) / (BO ? 2 : 4) + out) & 3);
  const int b0 = ai == ao ? min(v1, v0 + (int)((4 - ((ai + v0) & 3)) & 3)) : v1, quads = (v1 - b0) >> 2, b1 = b0 + 4 * quads;
  const int word0 = (4 - (b0 - v0)) & 3;  // of the slice's first id in the table, so that the four's words are aligned
  constexpr int U = kInFlight;
  Quad<BI> x[U];
  uint32_t bits[U];
  const bool whole = (b0 & 3) == 0;  // four logits' bits lie in one word
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads, v = b0 + 4 * i;
      bits[u] = ~0u;
      if (i >= quads) continue;
      if (!a.in_place) x[u] = load4<BI>(a.logits, in + v);
      if (mask != nullptr) bits[u] = mask[v >> 5];
    }
  };
  load(tid);

  // ---- the table
  if (sparse) {
    for (int i = tid; i < (n + word0 + 3) / 4; i += kThreads) reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int j = tid; j < a.biases; j += kThreads) {
      const int id = a.bias_ids[(int64_t)t * a.biases + j];
      if ((unsigned)(id - v0) < (unsigned)n)
        atomicMax(&table[id - v0 + word0], (uint32_t)(j + 1) << kBiasShift);
      else if (id < -1 || id >= a.V)
        complain(kErrBadToken);
    }
    __syncthreads();
    if (a.max_history > 0) {
      const int len = a.history_len[t], all = min(max(len, 0), a.max_history);
      const int prompt = a.prompt_len != nullptr ? a.prompt_len[t] : 0, made = min(max(prompt, 0), all);
      if (tid == 0 && (len != all || prompt != made)) complain(kErrBadLength);
      const int32_t* history = a.history + t * a.history_stride;
      uint32_t* mine = table + word0;
      auto count = [&](int j, int id) {
        if ((unsigned)(id - v0) < (unsigned)n) {
          if (j < made)
            atomicOr(&mine[id - v0], kPrompt);
          else
            atomicAdd(&mine[id - v0], 1u);
        }
      };
      // 4 at a time from where the row is aligned, in as few instructions an id as can be: every slice looks
      // at them all
      const int j0 = min(all, (int)((4 - (reinterpret_cast<uintptr_t>(history) >> 2)) & 3)), fours = (all - j0) >> 2;
      if (tid < j0) count(tid, history[tid]);
      if (tid < all - j0 - 4 * fours) count(j0 + 4 * fours + tid, history[j0 + 4 * fours + tid]);
#pragma unroll 2
      for (int i = tid; i < fours; i += kThreads) {
        const int4 id = *reinterpret_cast<const int4*>(history + j0 + 4 * i);
        count(j0 + 4 * i, id.x), count(j0 + 4 * i + 1, id.y), count(j0 + 4 * i + 2, id.z), count(j0 + 4 * i + 3, id.w);
      }
      // ids outside the vocabulary: each slice looks through a part of them
      bool bad = false;
      for (int j = part * kThreads + tid; j < all; j += a.slices * kThreads) bad |= (unsigned)history[j] >= (unsigned)a.V;
      if (bad && a.err != nullptr) atomicOr(a.err, kErrBadToken);
    }
    __syncthreads();
  }

  // ---- the logits
  auto one = [&](int v) {
    const bool on = mask == nullptr || (mask[v >> 5] >> (v & 31) & 1);
    const uint32_t e = sparse ? table[v - v0 + word0] : 0;
    if (on && a.in_place && e == 0) return;
    store1<BO>(a.out, out + v, on ? adjusted(load1<BI>(a.logits, in + v), e) : kOff);
  };
  if (ai != ao) {
#pragma unroll 4
    for (int v = v0 + tid; v < v1; v += kThreads) one(v);
    return;
  }
  if (tid < b0 - v0) one(v0 + tid);
  if (tid < v1 - b1) one(b1 + tid);
  const uint4* words = reinterpret_cast<const uint4*>(table + word0 + b0 - v0);
  for (int i0 = tid; i0 < quads; i0 += U * kThreads) {
    if (i0 != tid) load(i0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kThreads, v = b0 + 4 * i;
      if (i >= quads) break;
      uint32_t on = __funnelshift_r(bits[u], bits[u], v);  // (by v mod 32)
      if (!whole && mask != nullptr && (v & 31) > 28) on = __funnelshift_r(bits[u], mask[(v >> 5) + 1], v);
      on &= 15;
      const uint4 e = sparse ? words[i] : make_uint4(0, 0, 0, 0);
      const bool touched = (e.x | e.y | e.z | e.w) != 0;
      if (a.in_place) {
        if (on == 15 && !touched) continue;
        x[u] = load4<BI>(a.logits, in + v);
      }
      float f[4];
      x[u].get(f);
      if (touched) {
        if (e.x) f[0] = adjusted(f[0], e.x);
        if (e.y) f[1] = adjusted(f[1], e.y);
        if (e.z) f[2] = adjusted(f[2], e.z);
        if (e.w) f[3] = adjusted(f[3], e.w);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (!(on >> k & 1)) f[k] = kOff;
      store4<BO>(a.out, out + v, f);
    }
  }
}

}  // namespace
}  // namespace pmoe

using namespace pmoe;

extern "C" int moe_adjust_logits(const void* logits, int is_bf16, int T, int V, int64_t row_stride, const int32_t* history,
                                 int64_t history_stride, int max_history, const int32_t* prompt_len,
                                 const int32_t* history_len, const float* repetition, const float* frequency,
                                 const float* presence, const int32_t* bias_ids, const float* bias, int biases,
                                 const uint32_t* mask, int64_t mask_stride, void* out, int out_is_bf16, int64_t out_stride,
                                 int32_t* err_out, void* stream) {
  if (T < 0 || V < 1 || V > 262144 || row_stride < V || out_stride < V || max_history < 0 || max_history > (int)kCount ||
      biases < 0 || biases > kMaxBiases)
    return PMOE_EINVAL;
  if (T == 0) return PMOE_OK;
  auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
  if (logits == nullptr || out == nullptr || off(logits, is_bf16 ? 2 : 4) || off(out, out_is_bf16 ? 2 : 4)) return PMOE_EINVAL;
  if (max_history > 0 && (history == nullptr || history_len == nullptr || history_stride < max_history)) return PMOE_EINVAL;
  if (biases > 0 && (bias_ids == nullptr || bias == nullptr)) return PMOE_EINVAL;
  if (mask != nullptr && mask_stride < (V + 31) / 32) return PMOE_EINVAL;
  const void* words[] = {history, prompt_len, history_len, repetition, frequency, presence, bias_ids, bias, mask, err_out};
  for (const void* p : words)
    if (off(p, 4)) return PMOE_EINVAL;
  const bool in_place = logits == out;
  if (in_place && ((is_bf16 != 0) != (out_is_bf16 != 0) || (T > 1 && row_stride != out_stride))) return PMOE_EINVAL;
  AdjustArgs a{logits,    out,        row_stride, out_stride, T,      V,    in_place, history, history_stride, max_history,
               prompt_len, history_len, repetition, frequency,  presence, bias_ids, bias,     biases,  mask,           mask_stride,
               err_out,   0,          0};
  // Each slice looks at its row's whole history, so they are as large as leaves every SM (of 152) its share, and no
  // larger than two turns of the logits in flight: 256 rows of 160,001 in slices of 16,384, 8,192, 4,096 89, 76, 97 us.
  a.slice = kMaxSlice;
  while (a.slice > 1024 && (int64_t)T * ((V + a.slice - 1) / a.slice) < 152 * kPerSM) a.slice /= 2;
  a.slices = (V + a.slice - 1) / a.slice;
  a.slice = ((V + a.slices - 1) / a.slices + 3) / 4 * 4;  // all alike
  if ((int64_t)T * a.slices > INT32_MAX) return PMOE_EINVAL;
  static SmemLimit limits[4];
  const size_t smem = max_history > 0 || biases > 0 ? (size_t)a.slice * 4 + 16 : 0;
  cudaStream_t s = (cudaStream_t)stream;
  const char* what = "moe_adjust_logits";
  const unsigned blocks = (unsigned)(T * a.slices);
  const auto kernel = is_bf16 ? (out_is_bf16 ? adjust_kernel<true, true> : adjust_kernel<true, false>)
                              : (out_is_bf16 ? adjust_kernel<false, true> : adjust_kernel<false, false>);
  const int r = limits[(is_bf16 ? 2 : 0) + (out_is_bf16 ? 1 : 0)].set(reinterpret_cast<const void*>(kernel), kMaxSlice * 4 + 16, what);
  return r != PMOE_OK ? r : launch(what, kernel, blocks, kThreads, smem, s, true, 1, a);
}
