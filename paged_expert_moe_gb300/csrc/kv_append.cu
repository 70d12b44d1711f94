// moe_kv_append: head norm, rotary positions and the append to a paged cache, in one pass.
//
// For token t and head h of q and k (x the head's D values):
//   x <- x * rsqrt(mean(x^2) + eps) * norm_w            (where a norm weight is given)
//   (a, b) <- (a cos - b sin, b cos + a sin)             for each of the R/2 rotated pairs,
//   angle_i = positions[axis(i)][t] * inv_freq[i]
// then q -> q_out (bf16) and k, v -> the cache row that slots[t] names (bf16, or e4m3 of
// x / scale[kv head]). All of it is fp32 with one rounding at the end.
//
// The angle keeps what its floats round off, of the position (beyond 2^24) and of the product
// (one fma): at position 10^5 the latter alone would be up to 4e-3 rad, more than a bf16 output's
// own rounding. The sine and cosine of the rounded angle are turned by it.
//
// Bound: HBM (every input read once, every output written once); one token is launch
// latency. A block takes a few tokens, computes their sines and cosines once into shared
// memory while the first heads' values are in flight, and gives each head D/16 threads of
// 16 elements, arranged so that a thread holds both halves of its 8 pairs: no exchange
// between threads but the norm's sum.
//
// Measured (32 + 4 + 4 heads of 128, bf16): 8,192 tokens 30.9 us, 5.4 TB/s of the 6.8 a copy
// reaches, with the issue slots 67% busy; 4,099 tokens of 48 heads of 64 11.4 us, 4.4 TB/s; one
// token 3.0 us, a launch.
#include "pmoe_internal.h"

#include <algorithm>
#include <cuda_fp8.h>
#include <math.h>

namespace pmoe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTok = 16;    // tokens of a block
constexpr int kMaxPairs = 64;  // R / 2 <= D / 2
// Up to this angle its rounding is at most 2^-7, and the second-order correction off by 2^-23.5.
constexpr float kFarAngle = 131072.f;

struct AppendArgs {
  pmoe_kv_desc kv;
  const __nv_bfloat16 *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int T, q_heads;
  const int32_t* positions;
  int axes;
  const int32_t* pair_axis;
  const float* inv_freq;
  int rot, interleaved;
  const __nv_bfloat16 *q_norm, *k_norm;
  float eps;
  const int32_t* slots;
  __nv_bfloat16* q_out;
  int32_t* err;
};

__device__ __forceinline__ void unpack8(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 values as e4m3 of f / s: round to nearest even, saturating at +-448 (NaN stays NaN)
__device__ __forceinline__ uint2 pack8_e4m3(const float* f, float s) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] / s, f[4 * i + 1] / s), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] / s, f[4 * i + 3] / s), __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

// Sine and cosine of pos * f beyond kFarAngle, or of a position that a float does not hold (above
// 2^24): by the sum of the rounded product and of what was rounded off, of both. Out of line
// it costs 8,192 tokens at ordinary positions 0.2 us (30.9), in line 0.4.
__device__ __noinline__ void far_angle(int pos, float f, float* s, float* c) {
  const float p = (float)pos, rest = (float)((long long)pos - (long long)p);
  const float hi = p * f, lo = fmaf(rest, f, fmaf(p, f, -hi));
  float sh, ch, sl, cl;
  sincosf(hi, &sh, &ch);
  sincosf(lo, &sl, &cl);
  *s = sh * cl + ch * sl;
  *c = ch * cl - sh * sl;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a, int tok) {
  constexpr int LPH = D / 16;              // threads of a head
  constexpr int UNITS = kThreads / LPH;    // heads at once
  __shared__ __align__(16) float cs[kMaxTok][2][kMaxPairs];
  pdl_wait();  // the caches and inputs may come from the kernel ahead
  pdl_trigger();
  const int t0 = blockIdx.x * tok;
  const int nt = min(tok, a.T - t0);
  const int hk = a.kv.kv_heads, heads = a.q_heads + 2 * hk;
  const int j = threadIdx.x % LPH;
  // the two 8-element runs of this thread: for half-split pairs one in each half of the
  // rotated part, else the 16 elements from 16 j on
  const int half = a.rot >> 1;
  const bool split = !a.interleaved && j * 16 < a.rot;
  const int e0 = split ? j * 8 : j * 16, e1 = split ? half + j * 8 : j * 16 + 8;
  const bool turn = j * 16 < a.rot;
  const int psh = 31 - __clz(a.kv.page_size);

  // unit u is head u % heads of token t0 + u / heads; (t, h) walks it without divisions
  struct At {
    int t, h;
  };
  uint4 x0 = make_uint4(0, 0, 0, 0), x1 = x0, y0 = x0, y1 = x0;
  auto load = [&](const At& at, uint4& v0, uint4& v1) {
    const int64_t t = t0 + at.t;
    const __nv_bfloat16* p = at.h < a.q_heads        ? a.q + t * a.q_stride + at.h * D
                             : at.h < a.q_heads + hk ? a.k + t * a.k_stride + (at.h - a.q_heads) * D
                                                     : a.v + t * a.v_stride + (at.h - a.q_heads - hk) * D;
    v0 = __ldg(reinterpret_cast<const uint4*>(p + e0));
    v1 = __ldg(reinterpret_cast<const uint4*>(p + e1));
  };
  auto step = [&](At at) {
    at.h += UNITS;
    while (at.h >= heads) at.h -= heads, ++at.t;
    return at;
  };
  const int total = nt * heads;
  At at{0, (int)threadIdx.x / LPH};
  while (at.h >= heads) at.h -= heads, ++at.t;
  if (at.t < nt) load(at, x0, x1);
  At ahead = step(at);
  if (ahead.t < nt) load(ahead, y0, y1);

  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int tt = i / half, pr = i - tt * half;
    int ax = 0;
    if (a.pair_axis != nullptr) {
      ax = a.pair_axis[pr];
      if ((unsigned)ax >= (unsigned)a.axes) {
        if (a.err != nullptr) atomicOr(a.err, kErrBadAxis);
        ax = 0;
      }
    }
    const int pos = a.positions[(size_t)ax * a.T + t0 + tt];
    const float p = (float)pos, f = a.inv_freq[pr];
    const float hi = p * f, lo = fmaf(p, f, -hi);
    float s, c;
    if (fmaxf(fabsf(hi), fabsf(p) * 0.0078125f) > kFarAngle) {
      far_angle(pos, f, &s, &c);
      cs[tt][0][pr] = c;
      cs[tt][1][pr] = s;
    } else {
      sincosf(hi, &s, &c);
      const float l2 = 0.5f * lo * lo;
      cs[tt][0][pr] = c - lo * s - l2 * c;
      cs[tt][1][pr] = s + lo * c - l2 * s;
    }
  }
  __syncthreads();

  // The loop count is the same for all threads of a warp: the norm's shuffles need them. Two
  // units' loads are in flight while one is worked on.
  for (int base = 0; base < total; base += UNITS) {
    const bool live = at.t < nt;
    const int tt = live ? at.t : 0, t = t0 + tt, h = live ? at.h : 0;
    float f[16];
    unpack8(x0, f);
    unpack8(x1, f + 8);
    x0 = y0, x1 = y1;
    at = ahead;
    ahead = step(ahead);
    if (ahead.t < nt) load(ahead, y0, y1);
    const bool is_q = h < a.q_heads, is_k = !is_q && h < a.q_heads + hk;
    const __nv_bfloat16* nw = is_q ? a.q_norm : is_k ? a.k_norm : nullptr;
    if (a.q_norm != nullptr || a.k_norm != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
      for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (nw != nullptr) {
        const float r = rsqrtf(ss * (1.0f / D) + a.eps);
        float w[16];
        unpack8(__ldg(reinterpret_cast<const uint4*>(nw + e0)), w);
        unpack8(__ldg(reinterpret_cast<const uint4*>(nw + e1)), w + 8);
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = f[i] * r * w[i];
      }
    }
    if (turn && (is_q || is_k)) {
      const float* c = &cs[tt][0][j * 8];
      const float* s = &cs[tt][1][j * 8];
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = f[2 * i], y = f[2 * i + 1];
          f[2 * i] = x * c[i] - y * s[i];
          f[2 * i + 1] = y * c[i] + x * s[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = f[i], y = f[i + 8];
          f[i] = x * c[i] - y * s[i];
          f[i + 8] = y * c[i] + x * s[i];
        }
      }
    }
    if (live && is_q) {
      __nv_bfloat16* p = a.q_out + ((size_t)t * a.q_heads + h) * D;
      *reinterpret_cast<uint4*>(p + e0) = pack8(f);
      *reinterpret_cast<uint4*>(p + e1) = pack8(f + 8);
    } else if (live) {
      const int kh = h - a.q_heads - (is_k ? 0 : hk);
      const int slot = a.slots[t];
      const int page = slot >> psh;
      if (slot >= 0 && page < a.kv.num_pages) {
        const size_t row = (size_t)page * a.kv.page_stride +
                           ((size_t)kh * a.kv.page_size + (slot & (a.kv.page_size - 1))) * D;
        void* cache = is_k ? a.kv.k : a.kv.v;
        if (a.kv.dtype == PMOE_KV_BF16) {
          __nv_bfloat16* p = static_cast<__nv_bfloat16*>(cache) + row;
          *reinterpret_cast<uint4*>(p + e0) = pack8(f);
          *reinterpret_cast<uint4*>(p + e1) = pack8(f + 8);
        } else {
          uint8_t* p = static_cast<uint8_t*>(cache) + row;
          const float sc = (is_k ? a.kv.k_scale : a.kv.v_scale)[kh];
          *reinterpret_cast<uint2*>(p + e0) = pack8_e4m3(f, sc);
          *reinterpret_cast<uint2*>(p + e1) = pack8_e4m3(f + 8, sc);
        }
      } else if (slot != -1 && j == 0 && a.err != nullptr) {
        atomicOr(a.err, kErrBadSlot);
      }
    }
  }
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

int check_kv(const pmoe_kv_desc* kv) {
  if (kv == nullptr || kv->k == nullptr || kv->v == nullptr) return PMOE_EINVAL;
  if (kv->dtype != PMOE_KV_BF16 && kv->dtype != PMOE_KV_E4M3) return PMOE_EUNSUPPORTED;
  if (kv->head_dim != 64 && kv->head_dim != 128) return PMOE_EUNSUPPORTED;
  if (kv->page_size < 16 || kv->page_size > 256 || (kv->page_size & (kv->page_size - 1)) != 0) return PMOE_EUNSUPPORTED;
  if (kv->num_pages < 1 || kv->kv_heads < 1 || kv->kv_heads > 1024) return PMOE_EINVAL;
  if ((int64_t)kv->num_pages * kv->page_size > INT32_MAX) return PMOE_EINVAL;
  if (kv->dtype == PMOE_KV_E4M3 && (kv->k_scale == nullptr || kv->v_scale == nullptr || !aligned(kv->k_scale, 4) ||
                                    !aligned(kv->v_scale, 4)))
    return PMOE_EINVAL;
  const int64_t eb = kv->dtype == PMOE_KV_BF16 ? 2 : 1;
  if (kv->page_stride < (int64_t)kv->kv_heads * kv->page_size * kv->head_dim || kv->page_stride * eb % 16 != 0)
    return PMOE_EINVAL;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return PMOE_EINVAL;
  return PMOE_OK;
}

}  // namespace pmoe

using namespace pmoe;

extern "C" int moe_kv_append(const pmoe_kv_desc* kv, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                             const void* v, int64_t v_stride, int T, int q_heads, const int32_t* positions, int axes,
                             const int32_t* pair_axis, const float* inv_freq, int rotary_dim, int interleaved,
                             const void* q_norm, const void* k_norm, float eps, const int32_t* slots, void* q_out,
                             int32_t* err_out, void* stream) {
  const int r = check_kv(kv);
  if (r != PMOE_OK) return r;
  const int D = kv->head_dim, hk = kv->kv_heads;
  if (T < 0 || q_heads < 1 || q_heads > 1024) return PMOE_EINVAL;
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0) return PMOE_EINVAL;
  if (axes < 1 || axes > 8 || (axes > 1 && rotary_dim > 0 && pair_axis == nullptr)) return PMOE_EINVAL;
  if (!(eps >= 0.f)) return PMOE_EINVAL;
  if (q_stride < (int64_t)q_heads * D || k_stride < (int64_t)hk * D || v_stride < (int64_t)hk * D) return PMOE_EINVAL;
  if (T == 0) return PMOE_OK;
  if (q == nullptr || k == nullptr || v == nullptr || slots == nullptr || q_out == nullptr ||
      q == q_out)
    return PMOE_EINVAL;
  if (rotary_dim > 0 && (positions == nullptr || inv_freq == nullptr)) return PMOE_EINVAL;
  // heads move in 16-byte vectors
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || q_stride % 8 != 0 ||
      k_stride % 8 != 0 || v_stride % 8 != 0 || (q_norm != nullptr && !aligned(q_norm, 16)) ||
      (k_norm != nullptr && !aligned(k_norm, 16)))
    return PMOE_EINVAL;
  if (!aligned(positions, 4) || !aligned(pair_axis, 4) || !aligned(inv_freq, 4) || !aligned(slots, 4) ||
      !aligned(err_out, 4))
    return PMOE_EINVAL;
  const AppendArgs a{*kv,       static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
                     static_cast<const __nv_bfloat16*>(v), q_stride, k_stride, v_stride, T, q_heads, positions, axes,
                     pair_axis, inv_freq, rotary_dim, interleaved != 0, static_cast<const __nv_bfloat16*>(q_norm),
                     static_cast<const __nv_bfloat16*>(k_norm), eps, slots, static_cast<__nv_bfloat16*>(q_out), err_out};
  // A block's fixed steps cost more than a token's heads, and blocks beyond the four that an
  // SM holds are another wave: 4,099 tokens of 48 heads of 64 take 11.7 us with 7 tokens a
  // block (586 blocks), 13.8 with 6 (684); 8,192 of 40 of 128 take 51.9 with 1, 31.0 with 14.
  const int tok = std::min(kMaxTok, (T + 607) / 608);
  const int blocks = (T + tok - 1) / tok;
  cudaStream_t s = (cudaStream_t)stream;
  return launch("moe_kv_append", D == 128 ? kv_append_kernel<128> : kv_append_kernel<64>, blocks, kThreads, 0, s, true, 1, a,
                tok);
}
