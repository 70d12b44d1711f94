// moe_sample_tokens: temperature, top-k, top-p, min-p and the draw, one pass over the logits.
//
// A row's weights n_i = floor(exp((x_i - m) / temperature) * 2^31) are whole numbers and so
// are all their sums: atomics and reductions in any order give the same draw.
//
// Bound: HBM for many rows (each logit read once), the chain of dependent steps for few. A
// cluster of up to 8 CTAs takes a row; each CTA keeps its slice in shared memory, and the
// CTAs exchange statistics through distributed shared memory, every CTA making the same
// decisions for itself from all CTAs' figures:
//   1. load the slice; the row's largest (logit, lowest id);
//   2. histogram of the logits' distance from the largest, 512 bins of 1/16: count and
//      weight per bin; the bin in which the k-th token lies, and the one in which the
//      weight reaches top_p;
//   3. inside such a bin, four passes over 8 bits of the ordered logit each find the
//      threshold itself;
//   4. sums of the kept tokens in id order (ties of the threshold in id order), the segment
//      that holds floor(S * u), and its token.
#include "pmoe_internal.h"

#include <cooperative_groups.h>
#include <math.h>

namespace cg = cooperative_groups;

namespace pmoe {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kBins = 512;          // distance bins of step 2 (one per thread)
constexpr float kBinsPerUnit = 16.f;
constexpr int kMaxCluster = 8;
constexpr int kMaxVocab = 262144;

typedef unsigned long long u64;

struct SampleArgs {
  const void* logits;
  int is_bf16, T, V;
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

struct Shared {
  u64 best;               // this CTA's largest (key, ~id)
  u64 scan[kWarps];
  u64 pick_above;         // the bin found by a scan: weight above it,
  uint32_t pick_cnt;      // count above it,
  int pick_bin;           // and the bin
  uint32_t scan_cnt[kWarps];
  uint32_t cnt[2][kBins]; // histograms; weights as two 16-bit halves (a slice holds at most
  uint32_t lo[2][kBins];  // 32,768 elements: no half's sum leaves 32 bits)
  uint32_t hi[2][kBins];
  u64 seg_sum[kWarps];    // step 4: per warp segment, weight above the threshold
  uint32_t seg_tie[kWarps];
  u64 all_sum[kMaxCluster * kWarps];
  u64 base_sum;
  int pick_seg;
  uint32_t pick_tie;      // ties before the picked segment
};

__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

// NaN -> -inf, -0 -> +0 (ties are ties)
__device__ __forceinline__ float clean(float x) { return x == x ? x + 0.f : -INFINITY; }

__device__ __forceinline__ u64 share(u64 total, float part) {
  const u64 n = (u64)(part * 16777216.f);
  return (total >> 24) * n + (((total & 0xffffffull) * n) >> 24);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Row {
  float m, r;  // largest logit, 1 / temperature
  __device__ float weight(float x) const { return x == m ? 1.f : expf((x - m) * r); }
  __device__ static uint32_t units(float w) { return (uint32_t)(w * 2147483648.f); }
  __device__ int bin(float x) const {
    const float d = (m - x) * kBinsPerUnit;  // NaN (inf - inf): bin 0
    return d < (float)(kBins - 1) ? (int)d : (x == m ? 0 : kBins - 1);
  }
};

// Adds up bin `threadIdx.x` of all CTAs' histogram `b`; finds the first bin, ascending, at
// which the running count (by_count) or weight reaches `target` (> 0, at most the total).
// Every CTA of the cluster calls it; the result is in sh.pick_*. Returns the total weight.
__device__ u64 find_bin(cg::cluster_group& cluster, Shared& sh, int b, bool by_count, u64 target, u64* total_out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster.sync();
  uint32_t c = 0;
  u64 w = 0;
  for (unsigned i = 0; i < cluster.num_blocks(); ++i) {
    const Shared* o = cluster.map_shared_rank(&sh, i);
    c += o->cnt[b][tid];
    w += ((u64)o->hi[b][tid] << 16) + o->lo[b][tid];
  }
  u64 wi = w;
  uint32_t ci = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 a = __shfl_up_sync(0xffffffffu, wi, o);
    const uint32_t d = __shfl_up_sync(0xffffffffu, ci, o);
    if (lane >= o) wi += a, ci += d;
  }
  if (lane == 31) sh.scan[warp] = wi, sh.scan_cnt[warp] = ci;
  if (tid == 0) sh.pick_bin = kBins;
  __syncthreads();
  u64 wb = 0, total = 0;
  uint32_t cb = 0;
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) wb += sh.scan[i], cb += sh.scan_cnt[i];
    total += sh.scan[i];
  }
  wi += wb, ci += cb;
  if (total_out != nullptr) *total_out = total;
  if (by_count ? (ci >= target && ci - c < target) : (wi >= target && wi - w < target)) {
    sh.pick_bin = tid;
    sh.pick_cnt = ci - c;
    sh.pick_above = wi - w;
  }
  __syncthreads();
  return total;
}

__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  extern __shared__ __align__(16) float xs[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int nb = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / nb;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // slices start where the row's 16-byte vectors do: `shift` elements before its first
  const int eb = a.is_bf16 ? 2 : 4, per = 16 / eb;
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + (int64_t)row * a.row_stride * eb;
  const int shift = (int)((reinterpret_cast<uintptr_t>(base) & 15) / eb);
  const int first = rank * a.slice - shift;  // id of the slice's element 0
  const int n = max(0, min(a.slice, a.V - first));

  // ---- 1. load, largest
  u64 best = 0;
  auto put = [&](int i, float x) {
    xs[i] = x = clean(x);
    const u64 c = ((u64)key_of(x) << 32) | (uint32_t)~(first + i);
    best = max(best, c);
  };
  for (int i = tid * per; i < n; i += kThreads * per) {
    if (first + i >= 0 && i + per <= n) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(base + (int64_t)(first + i) * eb));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      if (a.is_bf16) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          put(i + 2 * q, __uint_as_float(w[q] << 16));
          put(i + 2 * q + 1, __uint_as_float(w[q] & 0xffff0000u));
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) put(i + q, __uint_as_float(w[q]));
      }
    } else {
      for (int q = i; q < min(i + per, n); ++q) {
        float x = -INFINITY;
        if (first + q >= 0)
          x = a.is_bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(base)[first + q] << 16)
                        : reinterpret_cast<const float*>(base)[first + q];
        if (first + q >= 0)
          put(q, x);
        else
          xs[q] = x;
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) sh.scan[warp] = best;
  for (int i = tid; i < kBins; i += kThreads) sh.cnt[0][i] = sh.lo[0][i] = sh.hi[0][i] = 0;
  __syncthreads();
  if (tid == 0) {
    for (int i = 0; i < kWarps; ++i) best = max(best, sh.scan[i]);
    sh.best = best;
  }
  cluster.sync();
  best = 0;
  for (int i = 0; i < nb; ++i) best = max(best, cluster.map_shared_rank(&sh, i)->best);

  const float temp = a.temperature != nullptr ? a.temperature[row] : 1.f;
  Row rw;
  rw.m = of_key((uint32_t)(best >> 32));
  rw.r = 1.f / temp;
  const bool none = rw.m == -INFINITY || best == 0;
  if (none || !(temp > 0.f)) {  // the same for every CTA of the row
    if (rank == 0 && tid == 0) {
      a.ids[row] = none ? -1 : (int32_t)~(uint32_t)best;
      if (a.logprob != nullptr) a.logprob[row] = none ? -INFINITY : 0.f;
    }
    cluster.sync();
    return;
  }

  // ---- 2. histogram over the distance from the largest
  const int top_k = a.top_k != nullptr ? a.top_k[row] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[row] : 1.f;
  const float min_p = a.min_p != nullptr ? fminf(a.min_p[row], 1.f) : 0.f;
  const bool use_k = top_k > 0 && top_k < a.V, use_p = top_p < 1.f;
  uint32_t key_t = 0;            // kept: key > key_t, and the first `ties` ids of key == key_t
  uint32_t ties = 0xffffffffu;
  if (use_k || use_p) {
    for (int i = tid; i < n; i += kThreads) {
      if (first + i < 0) continue;
      const float x = xs[i];
      const int b = rw.bin(x);
      const uint32_t w = Row::units(rw.weight(x));
      atomicAdd(&sh.cnt[0][b], 1u);
      if (w) {
        atomicAdd(&sh.lo[0][b], w & 0xffffu);
        atomicAdd(&sh.hi[0][b], w >> 16);
      }
    }
    __syncthreads();
    u64 total = 0, least = 0;
    for (int mode = use_k ? 0 : 1; mode <= (use_p ? 1 : 0); ++mode) {
      // mode 0: the top_k-th token; mode 1: the token at which the weight reaches top_p
      u64 target;
      if (mode == 0) {
        target = (u64)top_k;
      } else {
        if (!use_k) find_bin(cluster, sh, 0, false, 1, &total);
        least = max((u64)1, share(total, top_p > 0.f ? top_p : 0.f));
        target = least;
      }
      find_bin(cluster, sh, 0, mode == 0, target, nullptr);
      const int bin = sh.pick_bin;
      u64 above = sh.pick_above;
      uint32_t above_cnt = sh.pick_cnt;
      // ---- 3. the threshold inside the bin, 8 bits of the key at a time
      uint32_t prefix = 0;
      for (int level = 0; level < 4; ++level) {
        const int sft = 24 - 8 * level;
        __syncthreads();
        cluster.sync();  // every CTA has read histogram 1 of the level before
        for (int i = tid; i < kBins; i += kThreads) sh.cnt[1][i] = sh.lo[1][i] = sh.hi[1][i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
          if (first + i < 0) continue;
          const float x = xs[i];
          if (rw.bin(x) != bin) continue;
          const uint32_t k = key_of(x);
          if (level > 0 && (k >> (sft + 8)) != prefix) continue;
          const int d = 255 - ((k >> sft) & 255);  // descending
          const uint32_t w = Row::units(rw.weight(x));
          atomicAdd(&sh.cnt[1][d], 1u);
          atomicAdd(&sh.lo[1][d], w & 0xffffu);
          atomicAdd(&sh.hi[1][d], w >> 16);
        }
        __syncthreads();
        find_bin(cluster, sh, 1, mode == 0, mode == 0 ? target - above_cnt : target - above, nullptr);
        above += sh.pick_above;
        above_cnt += sh.pick_cnt;
        prefix = (prefix << 8) | (255 - sh.pick_bin);
      }
      key_t = prefix;
      const u64 each = Row::units(rw.weight(of_key(key_t)));
      if (mode == 0) {
        ties = (uint32_t)(target - above_cnt);
        total = above + each * ties;
      } else {
        ties = (uint32_t)((target - above + each - 1) / each);
      }
    }
  }

  // ---- 4. sums in id order: warp w of CTA c owns segment c * kWarps + w
  const int per_warp = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int s0 = min(n, warp * per_warp), s1 = min(n, s0 + per_warp);
  const uint32_t unit_t = Row::units(rw.weight(of_key(key_t)));
  const bool tie_ok = rw.weight(of_key(key_t)) >= min_p || !(min_p > 0.f);
  // weight of the element if it lies above the threshold; *tie: it lies on it
  auto kept = [&](int i, bool* tie) -> uint32_t {
    *tie = false;
    if (i >= s1 || first + i < 0) return 0;
    const float x = xs[i];
    const uint32_t k = key_of(x);
    if (k < key_t) return 0;
    if (k == key_t) {
      *tie = true;
      return 0;
    }
    const float w = rw.weight(x);
    return (w >= min_p || !(min_p > 0.f)) ? Row::units(w) : 0;
  };
  u64 sum = 0;
  uint32_t nt = 0;
  for (int i = s0 + lane; i < s1; i += 32) {
    bool tie;
    sum += kept(i, &tie);
    nt += tie;
  }
  sum = warp_sum(sum);
  nt = (uint32_t)warp_sum(nt);
  if (lane == 0) sh.seg_sum[warp] = sum, sh.seg_tie[warp] = nt;
  cluster.sync();
  const int segs = nb * kWarps;
  if (warp == 0) {
    // every CTA: running ties and sums over all segments
    u64 run = 0;
    uint32_t run_t = 0;
    for (int s = lane; s < ((segs + 31) & ~31); s += 32) {
      u64 v = 0;
      uint32_t t = 0;
      if (s < segs) {
        const Shared* o = cluster.map_shared_rank(&sh, s / kWarps);
        v = o->seg_sum[s % kWarps];
        t = o->seg_tie[s % kWarps];
      }
      uint32_t ti = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t d = __shfl_up_sync(0xffffffffu, ti, o);
        if (lane >= o) ti += d;
      }
      const uint32_t before = run_t + ti - t;
      run_t += __shfl_sync(0xffffffffu, ti, 31);
      const uint32_t in = before >= ties ? 0 : min(t, ties - before);
      if (tie_ok) v += (u64)in * unit_t;
      u64 vi = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 d = __shfl_up_sync(0xffffffffu, vi, o);
        if (lane >= o) vi += d;
      }
      vi += run;
      run = __shfl_sync(0xffffffffu, vi, 31);
      if (s < segs) sh.all_sum[s] = vi;
      if (s >= rank * kWarps && s < (rank + 1) * kWarps) sh.scan_cnt[s - rank * kWarps] = before;
    }
    if (lane == 0) sh.base_sum = run;
  }
  __syncthreads();
  const u64 S = sh.base_sum;
  const float uu = a.u[row];
  const u64 target = share(S, uu > 0.f ? fminf(uu, 0.99999994f) : 0.f);
  const int seg = rank * kWarps + warp;
  const u64 lo = seg == 0 ? 0 : sh.all_sum[seg - 1], hi = sh.all_sum[seg];
  if (target >= lo && target < hi) {  // exactly one warp of the cluster
    u64 run = lo;
    uint32_t tb = sh.scan_cnt[warp];
    for (int i0 = s0; i0 < s1; i0 += 32) {
      bool tie;
      u64 v = kept(i0 + lane, &tie);
      const uint32_t tm = __ballot_sync(0xffffffffu, tie);
      if (tie && tie_ok && tb + __popc(tm & ((1u << lane) - 1)) < ties) v = unit_t;
      tb += __popc(tm);
      u64 vi = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const u64 d = __shfl_up_sync(0xffffffffu, vi, o);
        if (lane >= o) vi += d;
      }
      const uint32_t over = __ballot_sync(0xffffffffu, run + vi > target);
      if (over) {
        const int l = __ffs(over) - 1;
        if (lane == l) {
          a.ids[row] = first + i0 + l;
          if (a.logprob != nullptr) a.logprob[row] = logf((float)v / (float)S);
        }
        break;
      }
      run += __shfl_sync(0xffffffffu, vi, 31);
    }
  }
  cluster.sync();  // no CTA leaves while another reads its shared memory
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
  int cluster = 1;
  while (cluster < kMaxCluster && V > cluster * 2048) cluster *= 2;
  if ((int64_t)T * cluster > INT32_MAX) return PMOE_EINVAL;
  SampleArgs a{logits, is_bf16 != 0, T, V, row_stride, temperature, top_k, top_p, min_p, u, ids_out, logprob_out, 0};
  // 7: the most elements by which a row can start after its first 16-byte vector
  a.slice = (((V + 7 + cluster - 1) / cluster) + 7) & ~7;
  const int smem = a.slice * 4;
  int r = cuda_status(cudaFuncSetAttribute(sample_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem),
                      "moe_sample_tokens");
  if (r != PMOE_OK) return r;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(T * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, sample_kernel, a), "moe_sample_tokens");
}
