// moe_adjust_logits: penalties for repeated tokens, biases and grammar masks on logits.
//
// A row's history touches few of its V logits, so the row is copied as it is (or left in place) with
// the masked ones set to -inf, and the touched ones are worked out after that. Which those are, and
// how often each occurs, is counted in shared memory: a CTA takes a slice of the ids of one row, one
// word an id, and reads the row's whole history, of which it counts what falls into its slice. The
// counts are whole numbers, so their order does not matter.
//
// Bound: HBM, the logits read and written once.
#include "pmoe_internal.h"

#include <math.h>

namespace pmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxSlice = 8192;
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
__global__ void __launch_bounds__(kThreads) adjust_kernel(const AdjustArgs a) {
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
  // ---- all of them as they are, or -inf
  const float kOff = -INFINITY;
  if (!a.in_place || mask != nullptr) {
    auto one = [&](int v) {
      const bool on = mask == nullptr || (mask[v >> 5] >> (v & 31) & 1);
      if (on && a.in_place) return;
      store1<BO>(a.out, out + v, on ? load1<BI>(a.logits, in + v) : kOff);
    };
    // 4 at a time from where both rows are aligned
    const int ai = (int)((reinterpret_cast<uintptr_t>(a.logits) / (BI ? 2 : 4) + in) & 3);
    const int ao = (int)((reinterpret_cast<uintptr_t>(a.out) / (BO ? 2 : 4) + out) & 3);
    if (ai == ao) {
      const int b0 = min(v1, v0 + (int)((4 - ((ai + v0) & 3)) & 3)), quads = (v1 - b0) >> 2, b1 = b0 + 4 * quads;
      if (tid < b0 - v0) one(v0 + tid);
      if (tid < v1 - b1) one(b1 + tid);
      constexpr int U = 8;  // in flight
      for (int i0 = tid; i0 < quads; i0 += U * kThreads) {
        uint32_t on[U];
        Quad<BI> x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * kThreads, v = b0 + 4 * i;
          on[u] = 15;
          if (mask != nullptr && i < quads) {
            // 4 bits from v on, of one word or two
            const int w = v >> 5, s = v & 31;
            on[u] = mask[w] >> s;
            if (s > 28) on[u] |= mask[w + 1] << (32 - s);
            on[u] &= 15;
          }
          if (i >= quads) on[u] = 16;  // none
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (on[u] - 1 < (a.in_place ? 14u : 15u)) x[u] = load4<BI>(a.logits, in + b0 + 4 * (i0 + u * kThreads));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (on[u] == 16 || (on[u] == 15 && a.in_place)) continue;
          float f[4] = {kOff, kOff, kOff, kOff};
          if (on[u] != 0) x[u].get(f);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!(on[u] >> k & 1)) f[k] = kOff;
          store4<BO>(a.out, out + b0 + 4 * (i0 + u * kThreads), f);
        }
      }
    } else {
#pragma unroll 8
      for (int v = v0 + tid; v < v1; v += kThreads) one(v);
    }
  }
  // ---- the touched ones: first which
  const bool sparse = a.max_history > 0 || a.biases > 0;
  if (!sparse) return;
  for (int i = tid; i < (n + 3) / 4; i += kThreads) reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  for (int j = tid; j < a.biases; j += kThreads) {
    const int id = a.bias_ids[(int64_t)t * a.biases + j];
    if ((unsigned)(id - v0) < (unsigned)n)
      atomicMax(&table[id - v0], (uint32_t)(j + 1) << kBiasShift);
    else if (id < -1 || id >= a.V)
      complain(kErrBadToken);
  }
  __syncthreads();
  if (a.max_history > 0) {
    const int len = a.history_len[t], all = min(max(len, 0), a.max_history);
    const int prompt = a.prompt_len != nullptr ? a.prompt_len[t] : 0, made = min(max(prompt, 0), all);
    if (tid == 0 && (len != all || prompt != made)) complain(kErrBadLength);
    const int32_t* history = a.history + t * a.history_stride;
#pragma unroll 8
    for (int j = tid; j < all; j += kThreads) {
      const int id = history[j];
      if ((unsigned)(id - v0) < (unsigned)n) {
        if (j < made)
          atomicOr(&table[id - v0], kPrompt);
        else
          atomicAdd(&table[id - v0], 1u);
      } else if (id < 0 || id >= a.V) {
        complain(kErrBadToken);
      }
    }
  }
  __syncthreads();

  // ---- then what they become
  const float rep = a.repetition != nullptr ? a.repetition[t] : 1.f, freq = a.frequency != nullptr ? a.frequency[t] : 0.f,
              pres = a.presence != nullptr ? a.presence[t] : 0.f;
  for (int i4 = tid; i4 < (n + 3) / 4; i4 += kThreads) {
    const uint4 four = reinterpret_cast<const uint4*>(table)[i4];
    if ((four.x | four.y | four.z | four.w) == 0) continue;
    const uint32_t es[4] = {four.x, four.y, four.z, four.w};
    const int v = v0 + 4 * i4;
    bool on[4];
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      on[k] = es[k] != 0 && (mask == nullptr || (mask[(v + k) >> 5] >> ((v + k) & 31) & 1));
      if (on[k]) x[k] = load1<BI>(a.logits, in + v + k);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!on[k]) continue;
      const uint32_t times = es[k] & kCount;
      float y = x[k];
      if (es[k] & (kCount | kPrompt)) y = y > 0.f ? y / rep : y * rep;
      if (times > 0) y = y - freq * (float)times - pres;
      if (es[k] >> kBiasShift) y += a.bias[(int64_t)t * a.biases + (es[k] >> kBiasShift) - 1];
      store1<BO>(a.out, out + v + k, y);
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
  // a slice an SM four times over, where the rows give that much
  a.slice = kMaxSlice;
  while (a.slice > 1024 && (int64_t)T * ((V + a.slice - 1) / a.slice) < 608) a.slice /= 2;
  a.slices = (V + a.slice - 1) / a.slice;
  if ((int64_t)T * a.slices > INT32_MAX) return PMOE_EINVAL;
  const size_t smem = max_history > 0 || biases > 0 ? (size_t)a.slice * 4 : 0;
  cudaStream_t s = (cudaStream_t)stream;
  const char* what = "moe_adjust_logits";
  const unsigned blocks = (unsigned)(T * a.slices);
  if (is_bf16)
    return out_is_bf16 ? launch(what, adjust_kernel<true, true>, blocks, kThreads, smem, s, true, 1, a)
                       : launch(what, adjust_kernel<true, false>, blocks, kThreads, smem, s, true, 1, a);
  return out_is_bf16 ? launch(what, adjust_kernel<false, true>, blocks, kThreads, smem, s, true, 1, a)
                     : launch(what, adjust_kernel<false, false>, blocks, kThreads, smem, s, true, 1, a);
}
