// moe_sample_tokens: temperature, top-k, top-p, min-p and the draw, one pass over the logits.
//
// A row's weights n_i = floor(exp((x_i - m) / temperature) * 2^31) are whole numbers and so
// are all their sums: atomics and reductions in any order give the same draw.
//
// Bound: HBM for many rows (each logit read once), the chain of dependent steps for few. A
// cluster of up to 8 CTAs takes a row; each CTA keeps its slice in shared memory and the
// CTAs exchange statistics through distributed shared memory.
//   1. Load the slice; the largest logit of the row and of each thread.
//   2. Rows that are cut by top-k or top-p: of the threads' largest logits, the bin (1/16
//      wide, by distance from the row's largest) that holds the K-th, K = top_k or 512. At
//      least K logits lie in it or above it, and seldom many more: these candidates go to
//      the row's first CTA, which sorts them, cuts them and draws. Rows with more than 2,048
//      candidates, or whose candidates do not reach top_p, go on with step 3.
//   3. A histogram of all logits over the same bins, count and weight; the bin that holds
//      the top_k-th token or in which the weight reaches top_p; inside it four passes over
//      8 bits of the ordered logit find the threshold itself.
//   4. Sums of the kept tokens in id order (ties of the threshold in id order), the segment
//      that holds floor(S * u), and its token.
// Uncut rows take steps 1 and 4.
#include "pmoe_internal.h"

#include <cooperative_groups.h>
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
constexpr int kList = 1024;         // candidates of a CTA
constexpr int kMerged = 2048;       // and of a row
constexpr int kMaxK = 1200;         // top_k up to which rows are cut by their candidates
constexpr int kCutP = 512;          // K for rows that only top-p cuts
// exp(z) 2^31 < 1 for z below -21.487...
constexpr float kZeroBelow = -21.6f;

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

struct Histogram {        // weights as two 16-bit halves: a slice holds at most 32,776
  uint32_t cnt[kBins];    // elements, so that no half's sum leaves 32 bits
  uint32_t lo[kBins];
  uint32_t hi[kBins];
};

struct Shared {
  union {
    Histogram hist[2];
    struct {
      u64 merged[kMerged];
      u64 list[kList];
    };
  };
  float best;             // this CTA's largest logit
  int arg;                // and, for greedy rows, the lowest id that has it
  int listed;             // candidates found
  int done;               // the row's first CTA has drawn
  u64 sum;                // all weights of the slice
  u64 scan[kWarps];
  uint32_t scan_cnt[kWarps];
  u64 pick_above;         // the bin found by a scan: weight above it,
  uint32_t pick_cnt;      // count above it,
  int pick_bin;           // and the bin
  u64 seg_sum[kWarps];    // step 4: per warp segment, weight above the threshold
  uint32_t seg_tie[kWarps];
  u64 all_sum[kMaxCluster * kWarps];
  u64 base_sum;
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

struct Row {
  float m, r;  // largest logit, 1 / temperature
  __device__ __forceinline__ float weight(float x) const { return x == m ? 1.f : expf((x - m) * r); }
  // NaN gives 0, as -inf does
  __device__ __forceinline__ static uint32_t units(float w) { return (uint32_t)(w * 2147483648.f); }
  __device__ __forceinline__ uint32_t units_of(float x) const {
    const float z = (x - m) * r;
    return x == m ? 0x80000000u : z > kZeroBelow ? units(expf(z)) : 0u;
  }
  __device__ __forceinline__ int bin(float x) const {
    const float d = (m - x) * kBinsPerUnit;
    return d < (float)(kBins - 1) ? (int)d : (x == m ? 0 : kBins - 1);
  }
};

template <bool BF16>
struct Vec {
  static constexpr int N = BF16 ? 8 : 4;  // logits in 16 bytes
  float f[N];
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

// Sorts a[0, n) ascending, n a power of two from 64 to kMerged. A barrier is only needed
// where a pair lies further apart than the 64 elements that a warp covers.
__device__ void sort_up(u64* a, int n) {
  for (int k = 2; k <= n; k <<= 1)
    for (int j = k >> 1; j > 0; j >>= 1) {
      for (int t = threadIdx.x; t < n / 2; t += kThreads) {
        const int i = 2 * t - (t & (j - 1));
        const u64 x = a[i], y = a[i + j];
        if ((x > y) == ((i & k) == 0)) a[i] = y, a[i + j] = x;
      }
      if (j > 32 || (j == 1 && 2 * k > 64))
        __syncthreads();
      else
        __syncwarp();
    }
}

__device__ __forceinline__ int pow2_above(int n) { return n <= 64 ? 64 : 1 << (32 - __clz(n - 1)); }

// Adds up bin `threadIdx.x` of all CTAs' histogram `b`; finds the first bin, ascending, at
// which the running count (by_count) or weight reaches `target` (> 0). Every CTA of the
// cluster calls it; the result is in sh.pick_* (bin kBins where it is not reached).
// Returns the total weight.
__device__ u64 find_bin(cg::cluster_group& cluster, Shared& sh, int b, bool by_count, u64 target) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  cluster.sync();
  uint32_t c = 0;
  u64 w = 0;
  for (unsigned i = 0; i < cluster.num_blocks(); ++i) {
    const Histogram& o = cluster.map_shared_rank(&sh, i)->hist[b];
    c += o.cnt[tid];
    if (!by_count || b == 1) w += ((u64)o.hi[tid] << 16) + o.lo[tid];
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
  if (by_count ? (ci >= target && ci - c < target) : (wi >= target && wi - w < target)) {
    sh.pick_bin = tid;
    sh.pick_cnt = ci - c;
    sh.pick_above = wi - w;
  }
  __syncthreads();
  return total;
}

// Step 2's end, in the row's first CTA: sh.merged holds n candidates as (~key << 32 | id).
// false: the kept tokens are not all among them.
__device__ bool cut_and_draw(Shared& sh, const SampleArgs& a, const Row& rw, int row, int n, int top_k, bool use_k,
                             float top_p, bool use_p, float min_p, u64 all_weights) {
  const int tid = threadIdx.x;
  constexpr int E = kMerged / kThreads;
  int n2 = pow2_above(n);
  for (int i = n + tid; i < n2; i += kThreads) sh.merged[i] = ~0ull;
  __syncthreads();
  sort_up(sh.merged, n2);
  __syncthreads();
  // thread t takes candidates t * e .. t * e + e - 1
  const int e = n2 <= kThreads ? 1 : n2 / kThreads;
  u64 c[E], w[E], mine = 0;
  float wt[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int at = tid * e + i;
    w[i] = 0;
    if (i < e && at < n && (!use_k || at < top_k)) {
      c[i] = sh.merged[at];
      wt[i] = rw.weight(of_key(~(uint32_t)(c[i] >> 32)));
      w[i] = Row::units(wt[i]);
      mine += w[i];
    }
  }
  u64 total;
  u64 run = block_scan(sh, mine, &total) - mine;
  u64 least = ~0ull;
  if (use_p) {
    least = max((u64)1, share(use_k ? total : all_weights, top_p > 0.f ? top_p : 0.f));
    if (total < least) return false;
  }
  u64 kept = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const bool k = w[i] > 0 && run < least && !(wt[i] < min_p);
    run += w[i];
    if (!k) w[i] = 0;
    kept += k;
  }
  u64 r;
  block_scan(sh, kept, &r);  // the kept tokens are the first r
  n2 = pow2_above((int)r);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int at = tid * e + i;
    if (i < e && at < n2) sh.merged[at] = w[i] > 0 ? (c[i] << 32) | w[i] : ~0ull;
  }
  for (int i = kThreads * e + tid; i < n2; i += kThreads) sh.merged[i] = ~0ull;
  __syncthreads();
  sort_up(sh.merged, n2);
  __syncthreads();
  const int e2 = n2 <= kThreads ? 1 : n2 / kThreads;
  mine = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int at = tid * e2 + i;
    w[i] = 0;
    if (i < e2 && at < (int)r) {
      c[i] = sh.merged[at];
      w[i] = c[i] & 0xffffffffull;
      mine += w[i];
    }
  }
  run = block_scan(sh, mine, &total) - mine;
  const float uu = a.u[row];
  const u64 target = share(total, uu > 0.f ? fminf(uu, 0.99999994f) : 0.f);
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if (run <= target && target < run + w[i]) {
      a.ids[row] = (int32_t)(c[i] >> 32);
      if (a.logprob != nullptr) a.logprob[row] = logf((float)w[i] / (float)total);
    }
    run += w[i];
  }
  return true;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) sample_kernel(const SampleArgs a) {
  using V = Vec<BF16>;
  constexpr int N = V::N, EB = BF16 ? 2 : 4;
  extern __shared__ __align__(16) uint4 xs[];
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int nb = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int row = blockIdx.x / nb;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  // slices start where the row's 16-byte vectors do: `shift` elements before its first
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + (int64_t)row * a.row_stride * EB;
  const int shift = (int)((reinterpret_cast<uintptr_t>(base) & 15) / EB);
  const int first = rank * a.slice - shift;  // id of the slice's element 0
  const int n = max(0, min(a.slice, a.V - first));
  const int nv = (n + N - 1) / N;            // its vectors

  // ---- 1. load; elements outside the row are -inf
  float mine = -INFINITY;  // fmaxf leaves NaN out
  {
    constexpr int U = 4;
    for (int i0 = tid; i0 < nv; i0 += kThreads * U) {
      uint4 v[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * kThreads, id = first + i * N;
        if (i < nv && id >= 0 && (i + 1) * N <= n) {
          v[k] = __ldg(reinterpret_cast<const uint4*>(base + (int64_t)id * EB));
        } else {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (BF16) {
              uint32_t h[2];
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const int e = id + 2 * q + z;
                h[z] = i < nv && e >= 0 && e < a.V && i * N + 2 * q + z < n ? reinterpret_cast<const uint16_t*>(base)[e] : 0xff80u;
              }
              w[q] = h[0] | (h[1] << 16);
            } else {
              const int e = id + q;
              w[q] = i < nv && e >= 0 && e < a.V && i * N + q < n ? reinterpret_cast<const uint32_t*>(base)[e] : 0xff800000u;
            }
          }
          v[k] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * kThreads;
        if (i < nv) xs[i] = v[k];
        const V x(v[k]);
#pragma unroll
        for (int q = 0; q < N; ++q) mine = fmaxf(mine, x.f[q]);
      }
    }
  }
  float best = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
  if (lane == 0) sh.seg_sum[warp] = __float_as_uint(best);
  sh.hist[0].cnt[tid] = 0;
  if (tid == 0) sh.arg = INT_MAX, sh.listed = 0, sh.done = 0;
  __syncthreads();
  if (tid == 0) {
    for (int i = 0; i < kWarps; ++i) best = fmaxf(best, __uint_as_float((uint32_t)sh.seg_sum[i]));
    sh.best = best;
  }
  cluster.sync();
  best = -INFINITY;
  for (int i = 0; i < nb; ++i) best = fmaxf(best, cluster.map_shared_rank(&sh, i)->best);

  const float temp = a.temperature != nullptr ? a.temperature[row] : 1.f;
  const Row rw{best, 1.f / temp};
  if (best == -INFINITY || !(temp > 0.f)) {  // the same for every CTA of the row
    if (best != -INFINITY && sh.best == best) {
      int low = INT_MAX;
      for (int i = tid; i < nv; i += kThreads) {
        const V x(xs[i]);
#pragma unroll
        for (int q = N - 1; q >= 0; --q)
          if (x.f[q] == best) low = min(low, first + i * N + q);
      }
      low = __reduce_min_sync(0xffffffffu, low);
      if (lane == 0) atomicMin(&sh.arg, low);
    }
    cluster.sync();
    if (rank == 0 && tid == 0) {
      int low = INT_MAX;
      for (int i = 0; i < nb; ++i) low = min(low, cluster.map_shared_rank(&sh, i)->arg);
      a.ids[row] = best == -INFINITY ? -1 : low;
      if (a.logprob != nullptr) a.logprob[row] = best == -INFINITY ? -INFINITY : 0.f;
    }
    cluster.sync();
    return;
  }

  const int top_k = a.top_k != nullptr ? a.top_k[row] : 0;
  const float top_p = a.top_p != nullptr ? a.top_p[row] : 1.f;
  const float min_p = a.min_p != nullptr ? fminf(a.min_p[row], 1.f) : 0.f;
  const bool use_k = top_k > 0 && top_k < a.V, use_p = top_p < 1.f;

  // ---- 2. candidates
  if ((use_k && top_k <= kMaxK) || (!use_k && use_p)) {
    if (mine > -INFINITY) atomicAdd(&sh.hist[0].cnt[rw.bin(mine)], 1u);
    __syncthreads();
    find_bin(cluster, sh, 0, true, use_k ? (u64)top_k : (u64)kCutP);
    // candidates: bin at most pick_bin; everything where the threads are fewer than K
    const float below = sh.pick_bin >= kBins - 1 ? INFINITY : (float)(sh.pick_bin + 1);
    cluster.sync();  // every CTA has read the counts: the list may take their place
    u64 sum = 0;
    const bool totals = !use_k;
    for (int i = tid; i < nv; i += kThreads) {
      const V x(xs[i]);
#pragma unroll
      for (int q = 0; q < N; ++q) {
        if (totals) sum += rw.units_of(x.f[q]);
        if ((rw.m - x.f[q]) * kBinsPerUnit < below || x.f[q] == rw.m) {
          const int at = atomicAdd(&sh.listed, 1);
          if (at < kList) sh.list[at] = ((u64)~key_of(x.f[q]) << 32) | (uint32_t)(first + i * N + q);
        }
      }
    }
    if (totals) {
      sum = warp_sum(sum);
      if (lane == 0) sh.seg_sum[warp] = sum;
      __syncthreads();
      if (tid == 0) {
        for (int i = 1; i < kWarps; ++i) sum += sh.seg_sum[i];
        sh.sum = sum;
      }
    }
    cluster.sync();
    if (rank == 0) {
      int total = 0;
      bool fits = true;
      u64 weights = 0;
      for (int i = 0; i < nb; ++i) {
        const Shared* o = cluster.map_shared_rank(&sh, i);
        const int c = o->listed;
        fits = fits && c <= kList && total + c <= kMerged;
        if (fits)
          for (int k = tid; k < c; k += kThreads) sh.merged[total + k] = o->list[k];
        total += c;
        if (totals) weights += o->sum;
      }
      __syncthreads();
      if (fits && cut_and_draw(sh, a, rw, row, total, top_k, use_k, top_p, use_p, min_p, weights) && tid == 0) sh.done = 1;
    }
    cluster.sync();
    const bool done = cluster.map_shared_rank(&sh, 0)->done != 0;
    cluster.sync();
    if (done) return;
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
  auto add = [&](int b, int bin, float x) {
    const uint32_t w = rw.units_of(x);
    atomicAdd(&sh.hist[b].cnt[bin], 1u);
    if (w) {
      atomicAdd(&sh.hist[b].lo[bin], w & 0xffffu);
      atomicAdd(&sh.hist[b].hi[bin], w >> 16);
    }
  };
  if (use_k || use_p) {
    sh.hist[0].cnt[tid] = sh.hist[0].lo[tid] = sh.hist[0].hi[tid] = 0;
    __syncthreads();
    elements([&](float x) { add(0, rw.bin(x), x); });
    __syncthreads();
    u64 total = 0;
    for (int mode = use_k ? 0 : 1; mode <= (use_p ? 1 : 0); ++mode) {
      // mode 0: the top_k-th token; mode 1: the token at which the weight reaches top_p
      u64 target;
      if (mode == 0) {
        target = (u64)top_k;
      } else {
        if (!use_k) total = find_bin(cluster, sh, 0, false, 1);
        target = max((u64)1, share(total, top_p > 0.f ? top_p : 0.f));
      }
      const u64 all = find_bin(cluster, sh, 0, false, mode == 0 ? 1 : target);
      if (mode == 0) find_bin(cluster, sh, 0, true, target);
      if (sh.pick_bin == kBins) {  // top_k exceeds the logits above -inf: none is cut
        total = all;
        continue;
      }
      const int bin = sh.pick_bin;
      u64 above = 0;
      uint32_t above_cnt = sh.pick_cnt;
      if (mode == 1) above = sh.pick_above;
      // inside the bin, 8 bits of the key at a time
      uint32_t prefix = 0;
      for (int level = 0; level < 4; ++level) {
        const int sft = 24 - 8 * level;
        __syncthreads();
        cluster.sync();  // every CTA has read histogram 1 of the level before
        sh.hist[1].cnt[tid] = sh.hist[1].lo[tid] = sh.hist[1].hi[tid] = 0;
        __syncthreads();
        elements([&](float x) {
          if (rw.bin(x) != bin) return;
          const uint32_t k = key_of(x);
          if (level == 0 || (k >> (sft + 8)) == prefix) add(1, 255 - ((k >> sft) & 255), x);  // descending
        });
        __syncthreads();
        find_bin(cluster, sh, 1, mode == 0, mode == 0 ? target - above_cnt : target - above);
        above += sh.pick_above;
        above_cnt += sh.pick_cnt;
        prefix = (prefix << 8) | (255 - sh.pick_bin);
      }
      key_t = prefix;
      const u64 each = rw.units_of(of_key(key_t));
      if (mode == 0) {
        ties = (uint32_t)(target - above_cnt);
        // the weight above the bin, which the search by count does not add up
        __syncthreads();
        cluster.sync();
        u64 w = 0;
        if (tid < bin)
          for (int i = 0; i < nb; ++i) {
            const Histogram& o = cluster.map_shared_rank(&sh, i)->hist[0];
            w += ((u64)o.hi[tid] << 16) + o.lo[tid];
          }
        block_scan(sh, w, &total);
        total += above + each * ties;
      } else {
        ties = (uint32_t)((target - above + each - 1) / each);
      }
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
    const float z = (x - rw.m) * rw.r;
    if (x == rw.m) return x > x_t ? 0x80000000u : 0u;
    if (!(x > x_t && z > kZeroBelow)) return 0;
    const float w = expf(z);
    return w < min_p ? 0u : Row::units(w);
  };
  u64 sum = 0;
  uint32_t nt = 0;
  for (int i = s0 + lane; i < s1; i += 32) {
    const V x(xs[i]);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      sum += kept(x.f[q]);
      nt += x.f[q] == x_t;  // -inf where nothing is cut: tie_ok is false then
    }
  }
  sum = warp_sum(sum);
  nt = (uint32_t)__reduce_add_sync(0xffffffffu, nt);
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
      const u64 vi = warp_scan(v, lane) + run;
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
      u64 w[N], v = 0;
      uint32_t t = 0;
      const int i = i0 + lane;
      const V x(i < s1 ? xs[i] : BF16 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                                      : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u));
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
  SampleArgs a{logits, T, V, row_stride, temperature, top_k, top_p, min_p, u, ids_out, logprob_out, 0};
  // 7: the most elements by which a row can start after its first 16-byte vector
  a.slice = (((V + 7 + cluster - 1) / cluster) + 7) & ~7;
  const int smem = a.slice * (is_bf16 ? 2 : 4);
  const auto kernel = is_bf16 ? sample_kernel<true> : sample_kernel<false>;
  static SmemLimit limit[2];
  const int r = limit[is_bf16 ? 1 : 0].set(reinterpret_cast<const void*>(kernel), kMaxSmem, "moe_sample_tokens");
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
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, a), "moe_sample_tokens");
}
