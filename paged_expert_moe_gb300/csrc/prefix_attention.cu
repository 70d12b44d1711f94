// moe_prefix_attention: attention over a paged cache for a batch that shares a prefix.
//
// Three kernels. The prefix is read once for all rows of a kv head: on the tensor cores as
// two matrix products a tile (prefix_tc.cu). The stream kernel here takes each row's own
// keys, and the prefix too where few rows share it; the combine kernel joins the parts.
//
// The stream kernel is bound by HBM: a key and its value are used by the at most 16 query
// heads of an item only, 4 to 16 operations a byte. Every warp runs for itself, without a
// barrier of the block: a ring of 16-key tiles of its own that TMA fills (a tile lies inside
// one page; one box for K, one for V), mma.sync on 16 query rows, softmax in registers. The
// (item, tile) units of all items, in order, are cut into equal runs, one a warp of every
// SM; a warp whose run ends inside an item leaves a part of it. An item counts for kHead units
// more than its tiles: short ones cost more than their keys. So that an item has few parts, whose
// room is planned on the host, a run is at least a fraction of max_suffix: where that is far above
// the lengths, few warps have work (256 rows of 1..1,024 own keys on 32,768 shared ones: 147 us with
// a bound of 1,024, 206 with 8,192, 1,356 with 131,072). Calls of few and short items take a CTA or
// a cluster an item instead, which joins its warps' parts itself (4 rows of 564 keys 7.8 us, 1 of
// 2,064 9.1). Measured, with the combine: 256 rows of 1..1,024 keys (4 kv heads of 128, bf16) 59 us;
// 64 rows of 1,000..16,000 172 us, 6.4 TB/s, 0.95 of a copy; 2 rows on 100,003 shared and 256 own
// keys 45 us, 4.6 TB/s.
#include "attn.cuh"
#include "attn_plan.h"
#include "tc_gemm.h"
#include "tc_ptx.cuh"

#include <algorithm>
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

namespace pmoe {
namespace attn {
namespace {

using namespace tc;

constexpr int kTile = 16;       // keys of a unit
constexpr int kHead = 2;        // empty units at the start of an item
constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void lds128(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// D[16 x 8] += A[16 x 16] B[16 x 8]: bf16 operands, or fp16 with an e4m3 cache
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// What a warp has to know of a unit, noted in shared memory beside its stage.
struct Unit {
  int tile, tiles;  // of the item
  int valid;        // keys of this tile that the item sees, up to kTile
  int h;            // kv head
  int t;            // token; < 0: the prefix, whose rows are all T * group of them
  int row0;         // first query row of the item, in the token's group or in all rows
};

template <int D, bool F8>
struct StreamCfg {
  static constexpr int kTileBytes = kTile * D * (F8 ? 1 : 2);  // of K, and of V
  static constexpr int kStage = 2 * kTileBytes;
  // 16 KB a warp and 128 KB an SM in flight; what HBM delivers an SM within its latency is 50
  // KB, and 24 KB a warp is slower (52 against 50.6 us for 256 rows of 1..1,024 keys)
  static constexpr int kFit = 16384 / kStage, kStages = kFit < 8 ? kFit : 8;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kSmem = 1024 /* alignment */ + kRing + kWarps * kStages * (8 + (int)sizeof(Unit)) +
                               (kRowBlock + 1) * 8 + kRowBlock * 4 + 64 * 8;
  // Where 16-byte chunk c of row r lies in a K or V tile (as the TMA swizzle puts it)
  static __device__ __forceinline__ uint32_t place(int r, int c) {
    if (!F8) return (uint32_t)((c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
    if (D == 128) return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4));
    return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
  }
  // The key row of column j of an 8-key group. With e4m3 rows of 128 bytes a phase of a
  // 16-byte access covers rows 2i and 2i + 1: the order lets them differ in bit 2, which the
  // swizzle turns into distinct banks.
  static __device__ __forceinline__ int key_row(int j) { return F8 && D == 128 ? (j >> 1) | ((j & 1) << 2) : j; }
};

// Units of a row's suffix, and the share of a warp.
__device__ __forceinline__ int64_t row_units(const Args& a, int keys) {
  return keys > 0 ? (int64_t)((keys + kTile - 1) / kTile + kHead) * a.head_items : 0;
}
// The first unit with keys of an item, `origin` the first of its row's (or the prefix's) units.
__device__ __forceinline__ int64_t first_unit(int64_t origin, int item, int tiles) {
  return origin + (int64_t)item * (tiles + kHead) + kHead;
}
__device__ __forceinline__ int64_t share_of(const Args& a, int64_t units) {
  return max((int64_t)a.min_share, (units + a.warps - 1) / a.warps);
}

// WHOLE: a CTA, or a cluster of up to 8, takes all keys of one item, shared and own, its warps a
// run of tiles each, and writes the output itself.
template <int D, bool F8, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 1)
    stream_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Args a,
                  int block) {
  using C = StreamCfg<D, F8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + C::kRing);
  int64_t* base = reinterpret_cast<int64_t*>(bars + kWarps * C::kStages);  // [nrows + 1]
  int64_t* sums = base + kRowBlock + 1;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sums + kWarps);
  int32_t* keys = reinterpret_cast<int32_t*>(sums + 64);  // [nrows]
  Unit* notes = reinterpret_cast<Unit*>(keys + kRowBlock);
  float2* ml = reinterpret_cast<float2*>(base);  // WHOLE, which has no rows to plan: [kWarps][16]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int t0 = block * kRowBlock, nrows = a.max_suffix > 0 ? min(kRowBlock, a.T - t0) : 0;
  const int64_t pre = block == 0 && a.pre_tiles > 0 ? (int64_t)a.pre_items * (a.pre_tiles + kHead) : 0;
  // Behind the prefix kernel, which began after all that came before the call, this one starts
  // at once and waits at its end; else it is the call's first and waits here.
  if (a.tc_ctas == 0) pdl_wait();
  pdl_trigger();

  if (tid == 0) *abort_flag = 0;
  if (lane == 0) {
    for (int i = 0; i < C::kStages; ++i) mbar_init(&bars[warp * C::kStages + i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    if (warp == 0) prefetch_map(&map_k), prefetch_map(&map_v);
  }
  int64_t share = 0, w = 0, u0, u1;  // this warp's run of units; of a whole item: of its tiles
  Unit mine_item{};                  // WHOLE: the CTA's item, its shared tiles and own keys
  int shared_tiles = 0, own_keys = 0, rank = 0;
  if constexpr (WHOLE) {
    const int block_item = blockIdx.x / a.whole, rts = a.head_items / a.kv.kv_heads;
    const int t = block_item / a.head_items, item = block_item - t * a.head_items;
    rank = blockIdx.x - block_item * a.whole;
    mine_item.t = t, mine_item.h = item / rts, mine_item.row0 = (item - mine_item.h * rts) * 16;
    mine_item.tiles = INT_MAX;  // the run ends it
    shared_tiles = (a.prefix_len + kTile - 1) / kTile;
    own_keys = a.max_suffix > 0 ? suffix_keys(a, t) : 0;
    const int tiles = shared_tiles + (own_keys + kTile - 1) / kTile;
    share = (tiles + a.whole * kWarps - 1) / (a.whole * kWarps);
    u0 = min((int64_t)tiles, (rank * kWarps + warp) * share), u1 = min((int64_t)tiles, u0 + share);
    __syncthreads();
  } else {
    // ---- the first unit of every row: thread i sums 8 rows
    int64_t mine[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = tid * 8 + i;
      const int n = r < nrows ? suffix_keys(a, t0 + r) : 0;
      if (r < nrows) keys[r] = n;
      mine[i] = row_units(a, n);
      sum += mine[i];
    }
    int64_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t d = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += d;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    int64_t at = pre + upto - sum, units = pre;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) at += sums[i];
      units += sums[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = tid * 8 + i;
      if (r < nrows) {
        base[r] = at;
        if (blockIdx.x == 0) a.base[(int64_t)block * (kRowBlock + 1) + r] = at;  // for the combine kernel
      }
      at += mine[i];
    }
    if (tid == 0) {
      base[nrows] = units;
      if (blockIdx.x == 0) a.base[(int64_t)block * (kRowBlock + 1) + nrows] = units;
    }
    __syncthreads();

    // ---- this warp's run of units; neighbouring runs on different SMs
    share = share_of(a, units);
    w = (int64_t)warp * gridDim.x + blockIdx.x;
    u0 = w * share, u1 = min(units, u0 + share);
  }
  const int psh = 31 - __clz(a.kv.page_size);
  uint8_t* mystage = ring + warp * C::kStages * C::kStage;
  uint64_t* bar = bars + warp * C::kStages;

  Unit* note = notes + warp * C::kStages;

  // the pages of row t's own keys; none for a table row out of range, whose keys read as zeros
  auto own_pages = [&](int t) -> const int32_t* {
    const int seq = a.row_seq != nullptr ? a.row_seq[t] : t;
    if ((unsigned)seq < (unsigned)a.sequences) return a.page_table + (int64_t)seq * a.table_stride;
    return nullptr;
  };
  // ---- the loading side: lane i works out unit `batch` + i of the run, with its page id
  int64_t batch = u0 - 32;
  Unit mu{};
  int id = 0, row = 0, loaded = 0;
  uint32_t todo = 0;  // lanes whose units are still to be loaded
  auto load = [&]() {
    while (todo == 0) {
      batch += 32;
      if (batch >= u1) return;
      const int64_t v = batch + lane;
      bool live = v < u1;
      if (live) {
        int whole_tile = 0;
        int64_t r;  // unit of its row, or of the prefix
        const int32_t* pages;
        int n;
        if constexpr (WHOLE) {
          mu = mine_item;
          const bool shared = v < shared_tiles;
          r = v - (shared ? 0 : shared_tiles);
          n = shared ? a.prefix_len : own_keys;
          pages = shared ? a.prefix_pages : own_pages(mu.t);
        } else if (v < pre) {
          r = v;
          n = a.prefix_len;
          pages = a.prefix_pages;
          mu.t = -1;
        } else {
          int lo = 0, hi = nrows;  // base[lo] <= v < base[hi]
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (base[mid] <= v)
              lo = mid;
            else
              hi = mid;
          }
          r = v - base[lo];
          n = keys[lo];
          mu.t = t0 + lo;
          pages = own_pages(mu.t);
        }
        if constexpr (WHOLE) {
          whole_tile = (int)r;
        } else {
          mu.tiles = (n + kTile - 1) / kTile;
          const int span = mu.tiles + kHead;
          const int item = r >> 32 ? (int)(r / span) : (int)((uint32_t)r / (uint32_t)span);
          mu.tile = (int)(r - (int64_t)item * span) - kHead;
          live = mu.tile >= 0;
          if (mu.t < 0) {
            const int rt = item / a.kv.kv_heads;
            mu.h = item - rt * a.kv.kv_heads;
            mu.row0 = rt * 16;
          } else {
            const int rts = a.head_items / a.kv.kv_heads;
            mu.h = item / rts;
            mu.row0 = (item - mu.h * rts) * 16;
          }
        }
        if (live) {
          const int key = (WHOLE ? whole_tile : mu.tile) * kTile;
          mu.valid = min(kTile, n - key);
          row = key & (a.kv.page_size - 1);
          id = pages != nullptr ? __ldg(pages + (key >> psh)) : -1;
          if ((unsigned)id >= (unsigned)a.kv.num_pages) {
            if (a.err != nullptr) atomicOr(a.err, kErrBadPage);
            id = a.kv.num_pages;  // out of the map's range: reads as zeros
          }
        }
      }
      todo = __ballot_sync(0xffffffffu, live);
    }
    const int s = loaded % C::kStages;
    if (lane == __ffs(todo) - 1) {
      note[s] = mu;
      mbar_arrive_expect_tx(&bar[s], C::kStage);
      tma_load_5d(mystage + s * C::kStage, &map_k, &bar[s], 0, row, 0, mu.h, id);
      tma_load_5d(mystage + s * C::kStage + C::kTileBytes, &map_v, &bar[s], 0, row, 0, mu.h, id);
    }
    todo &= todo - 1;
    ++loaded;
    __syncwarp();
  };
#pragma unroll 1
  for (int i = 0; i < C::kStages; ++i) load();

  bool ok = true;
  int used = 0;  // units
  while (used < loaded && ok) {
    const Unit it = note[used % C::kStages];  // the first unit of an item, or of this warp's part of it
    const int rows = it.t < 0 ? min(16, a.T * a.group - it.row0) : min(16, a.group - it.row0);
    // ---- query fragments; rows beyond the last are zero
    uint32_t qf[D / 16][4];
    float qmul[2];  // what a score of rows g and g + 8 is multiplied by
    int64_t rowhead[2];
    bool live[2];
    {
      const __nv_bfloat16* qp[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = g + 8 * e;
        live[e] = i < rows;
        const int r = it.row0 + (live[e] ? i : 0), tok = it.t < 0 ? row_token(a, r) : it.t;
        const int head = it.h * a.group + (it.t < 0 ? r - tok * a.group : r);
        qp[e] = a.q + (int64_t)tok * a.q_stride + head * D;
        rowhead[e] = (int64_t)tok * a.q_heads + head;
        qmul[e] = a.scale;
      }
      if constexpr (!F8) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            qf[k][e] = live[e] ? __ldg(reinterpret_cast<const uint32_t*>(qp[e] + k * 16 + 2 * c)) : 0;
            qf[k][2 + e] = live[e] ? __ldg(reinterpret_cast<const uint32_t*>(qp[e] + k * 16 + 2 * c + 8)) : 0;
          }
      } else {
        // Slots of step k = 4 i + s hold elements 64 i + 16 c + 4 s + .. (the order in which a
        // thread reads 16 key bytes at once). q goes to fp16 divided by the power of two of
        // its row's largest element.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint2 raw[D / 16];
          float mx = 0.f;
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            raw[k] = live[e] ? __ldg(reinterpret_cast<const uint2*>(qp[e] + (k >> 2) * 64 + 16 * c + (k & 3) * 4))
                             : make_uint2(0, 0);
            const uint32_t v[2] = {raw[k].x, raw[k].y};
#pragma unroll
            for (int i = 0; i < 2; ++i)
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(v[i] << 16)), fabsf(__uint_as_float(v[i] & 0xffff0000u))));
          }
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          const int ex = row_exponent(mx);
          const float down = pow2(-ex);
          qmul[e] = a.scale * a.kv.k_scale[it.h] * pow2(ex);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t v[2] = {raw[k].x, raw[k].y};
#pragma unroll
            for (int i = 0; i < 2; ++i)
              qf[k][2 * i + e] = pack2<true>(__uint_as_float(v[i] << 16) * down, __uint_as_float(v[i] & 0xffff0000u) * down);
          }
        }
      }
    }

    float o[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    // m: what the exponents of the weights count from; it moves only when a score exceeds it
    // by 2^8 (any base gives the same quotient), so the sums are seldom rescaled
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    // until the item's last tile, or the run's
    for (bool more = true; more;) {
      const int s = used % C::kStages, tile = note[s].tile, valid = note[s].valid;
      if (!__all_sync(0xffffffffu, mbar_wait(&bar[s], (used / C::kStages) & 1, abort_flag, a.err))) {
        ok = false;
        break;
      }
      const uint32_t ks = smem_u32(mystage + s * C::kStage), vs = ks + C::kTileBytes;
      if (valid < kTile) {
        // values beyond the last key may be anything, and 0 x NaN is NaN
        constexpr int CH = C::kTileBytes / kTile / 16;  // 16-byte chunks of a row
        for (int i = valid * CH + lane; i < kTile * CH; i += 32)
          *reinterpret_cast<uint4*>(mystage + s * C::kStage + C::kTileBytes + C::place(i / CH, i % CH)) = make_uint4(0, 0, 0, 0);
        fence_async();
        __syncwarp();
      }
      float sc[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        sc[j][0] = sc[j][1] = sc[j][2] = sc[j][3] = 0.f;
        if constexpr (!F8) {
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            uint32_t b[4];
            ldsm4(b, ks + C::place(j * 8 + (lane & 7), k * 4 + (lane >> 3)));
            mma<false>(sc[j], qf[2 * k], b[0], b[1]);
            mma<false>(sc[j], qf[2 * k + 1], b[2], b[3]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            uint32_t b[4];
            lds128(b, ks + C::place(j * 8 + C::key_row(g), i * 4 + c));
#pragma unroll
            for (int k = 0; k < 4; ++k) mma<true>(sc[j], qf[4 * i + k], e4m3x2(b[k] & 0xffffu), e4m3x2(b[k] >> 16));
          }
        }
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sc[j][i] = j * 8 + C::key_row(2 * c + (i & 1)) < valid ? sc[j][i] * qmul[i >> 1] : -INFINITY;
          mx[i >> 1] = fmaxf(mx[i >> 1], sc[j][i]);
        }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] + 8.f || mx[1] > m[1] + 8.f)) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool grow = mx[e] > m[e] + 8.f;
          const float f = grow ? ex2(m[e] - mx[e]) : 1.f;
          if (grow) m[e] = mx[e];
          l[e] *= f;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) o[i][2 * e] *= f, o[i][2 * e + 1] *= f;
        }
      }
      uint32_t pf[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = ex2(sc[j][i] - (m[i >> 1] == -INFINITY ? 0.f : m[i >> 1]));
          l[i >> 1] += p[i];
        }
        pf[j * 2] = pack2<F8>(p[0], p[1]);
        pf[j * 2 + 1] = pack2<F8>(p[2], p[3]);
      }
      const int r = (lane & 8) | C::key_row(lane & 7);
      if constexpr (!F8) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t b[4];
          ldsm4t(b, vs + C::place(r, i * 2 + (lane >> 4)));
          mma<false>(o[2 * i], pf, b[0], b[1]);
          mma<false>(o[2 * i + 1], pf, b[2], b[3]);
        }
      } else {
        // a 16-bit element of the transposed load is 2 values of one key: the even and the
        // odd elements of 16 form an 8-column tile each
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t b[4];
          ldsm4t(b, vs + C::place(r, i * 2 + (lane >> 4)));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma<true>(o[4 * i + 2 * j], pf, e4m3x2(__byte_perm(b[2 * j], 0, 0x4420)),
                      e4m3x2(__byte_perm(b[2 * j + 1], 0, 0x4420)));
            mma<true>(o[4 * i + 2 * j + 1], pf, e4m3x2(__byte_perm(b[2 * j], 0, 0x4431)),
                      e4m3x2(__byte_perm(b[2 * j + 1], 0, 0x4431)));
          }
        }
      }
      __syncwarp();  // every lane has read the stage and its note
      ++used;
      load();
      more = tile + 1 < it.tiles && used < loaded;
    }
    if (!ok) break;

    if constexpr (WHOLE) {
      // the warp's ring is done with: it takes the warp's part
      float* mine_o = reinterpret_cast<float*>(mystage);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
        l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        float* dst = mine_o + (g + 8 * e) * D;
        if constexpr (!F8) {
#pragma unroll
          for (int k = 0; k < D / 8; ++k) *reinterpret_cast<float2*>(dst + k * 8 + 2 * c) = make_float2(o[k][2 * e], o[k][2 * e + 1]);
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            *reinterpret_cast<float4*>(dst + k * 16 + 4 * c) =
                make_float4(o[2 * k][2 * e], o[2 * k + 1][2 * e], o[2 * k][2 * e + 1], o[2 * k + 1][2 * e + 1]);
        }
        if (c == 0) ml[warp * 16 + g + 8 * e] = make_float2(m[e], l[e]);
      }
      break;
    }
    // ---- the part
    const int64_t origin = it.t < 0 ? 0 : base[it.t - t0];
    const int item = it.t < 0 ? it.row0 / 16 * a.kv.kv_heads + it.h : it.h * (a.head_items / a.kv.kv_heads) + it.row0 / 16;
    const int part = (int)(w - first_unit(origin, item, it.tiles) / share) + (it.t < 0 ? 0 : a.prefix_parts);
    const float vscale = F8 ? a.kv.v_scale[it.h] : 1.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      if (!live[e]) continue;
      const int64_t i = (int64_t)part * a.T * a.q_heads + rowhead[e];
      float* dst = a.o_part + i * D;
      if constexpr (!F8) {
#pragma unroll
        for (int k = 0; k < D / 8; ++k) *reinterpret_cast<float2*>(dst + k * 8 + 2 * c) = make_float2(o[k][2 * e], o[k][2 * e + 1]);
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          *reinterpret_cast<float4*>(dst + k * 16 + 4 * c) =
              make_float4(o[2 * k][2 * e] * vscale, o[2 * k + 1][2 * e] * vscale, o[2 * k][2 * e + 1] * vscale,
                          o[2 * k + 1][2 * e + 1] * vscale);
      }
      if (c == 0) a.ml_part[i] = make_float2(m[e], l[e]);
    }
  }
  // copies in flight land before the CTA leaves, even after a wait that gave up
  if (!ok)
    for (int i = used; i < loaded; ++i) {
      const long long c0 = clock64();
      while (!mbar_try_wait(&bar[i % C::kStages], (i / C::kStages) & 1) && clock64() - c0 < kWaitLimit) {
      }
    }
  if constexpr (WHOLE) {
    namespace cg = cooperative_groups;
    cg::cluster_group cluster = cg::this_cluster();
    if (a.whole > 1)
      cluster.sync();  // the first CTA's rings are done with too
    else
      __syncthreads();
    // 16 threads a row, D / 16 columns each; what the warps hold counts from their own bases
    const int i = tid >> 4, col = (tid & 15) * (D / 16);
    const int all = share > 0 ? (shared_tiles + (own_keys + kTile - 1) / kTile + (int)share - 1) / (int)share : 0;
    const int parts = max(0, min(kWarps, all - rank * kWarps));  // warps with tiles: of this CTA, of all
    float m = -INFINITY, l = 0.f, acc[D / 16];
    for (int k = 0; k < parts; ++k) m = fmaxf(m, ml[k * 16 + i].x);
#pragma unroll
    for (int d = 0; d < D / 16; ++d) acc[d] = 0.f;
    for (int k = 0; k < parts; ++k) {
      const float2 part = ml[k * 16 + i];
      const float f = ex2(part.x - (m == -INFINITY ? 0.f : m));
      l = fmaf(part.y, f, l);
      const float4* src =
          reinterpret_cast<const float4*>(reinterpret_cast<const float*>(ring + k * C::kStages * C::kStage) + i * D + col);
#pragma unroll
      for (int d = 0; d < D / 64; ++d) {
        const float4 x = src[d];
        acc[4 * d] = fmaf(x.x, f, acc[4 * d]), acc[4 * d + 1] = fmaf(x.y, f, acc[4 * d + 1]);
        acc[4 * d + 2] = fmaf(x.z, f, acc[4 * d + 2]), acc[4 * d + 3] = fmaf(x.w, f, acc[4 * d + 3]);
      }
    }
    if (a.whole > 1) {
      // the CTAs' parts meet in the first one's memory, in the halves of its rings that its own
      // warps' parts leave free
      constexpr int kHalf = C::kStages * C::kStage / 2;
      static_assert(16 * D * 4 <= kHalf, "a part in half a ring");
      if (rank > 0 && parts > 0) {
        float4* dst = reinterpret_cast<float4*>(cluster.map_shared_rank(ring, 0) + rank * 2 * kHalf + kHalf + (i * D + col) * 4);
#pragma unroll
        for (int d = 0; d < D / 64; ++d) dst[d] = make_float4(acc[4 * d], acc[4 * d + 1], acc[4 * d + 2], acc[4 * d + 3]);
        if ((tid & 15) == 0) cluster.map_shared_rank(ml, 0)[(kWarps + rank) * 16 + i] = make_float2(m, l);
      }
      cluster.sync();
      const int ctas = (all + kWarps - 1) / kWarps;
      float top = m;
      for (int k = 1; k < ctas; ++k) top = fmaxf(top, ml[(kWarps + k) * 16 + i].x);
      const float own = ex2(m - (top == -INFINITY ? 0.f : top));
      l *= own;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) acc[d] *= own;
      for (int k = 1; k < ctas && rank == 0; ++k) {
        const float2 part = ml[(kWarps + k) * 16 + i];
        const float f = ex2(part.x - (top == -INFINITY ? 0.f : top));
        l = fmaf(part.y, f, l);
        const float4* src = reinterpret_cast<const float4*>(ring + k * 2 * kHalf + kHalf + (i * D + col) * 4);
#pragma unroll
        for (int d = 0; d < D / 64; ++d) {
          const float4 x = src[d];
          acc[4 * d] = fmaf(x.x, f, acc[4 * d]), acc[4 * d + 1] = fmaf(x.y, f, acc[4 * d + 1]);
          acc[4 * d + 2] = fmaf(x.z, f, acc[4 * d + 2]), acc[4 * d + 3] = fmaf(x.w, f, acc[4 * d + 3]);
        }
      }
      m = top;
    }
    if (rank == 0 && mine_item.row0 + i < a.group) {
      const int64_t rh = (int64_t)mine_item.t * a.q_heads + mine_item.h * a.group + mine_item.row0 + i;
      const float inv = all == 0 ? 0.f : (F8 ? a.kv.v_scale[mine_item.h] : 1.f) / l;
#pragma unroll
      for (int d = 0; d < D / 16; d += 2)
        *reinterpret_cast<__nv_bfloat162*>(a.out + rh * D + col + d) = __floats2bfloat162_rn(acc[d] * inv, acc[d + 1] * inv);
      if (a.lse != nullptr && (tid & 15) == 0) a.lse[rh] = all == 0 ? -INFINITY : m * kLn2 + logf(l);
    }
  }
  pdl_wait();  // the combine kernel follows this one only: the tensor-core kernel is done then too
}

// Joins the parts of one row-head: W warps share its parts.
template <int D, int W>
__global__ void __launch_bounds__(W * 32 < 128 ? 128 : W * 32) combine_kernel(const Args a) {
  constexpr int kRowHeads = W < 4 ? 4 / W : 1, V = D / 32;
  __shared__ float red[W > 1 ? W : 1][D];
  const int64_t rh = (int64_t)a.T * a.q_heads;
  const int lane = threadIdx.x & 31, w = (threadIdx.x >> 5) % W;
  const int64_t i = (int64_t)blockIdx.x * kRowHeads + (threadIdx.x >> 5) / W;
  pdl_wait();
  pdl_trigger();
  if (W == 1 && i >= rh) return;
  const int t = (int)(i / a.q_heads), hq = (int)(i % a.q_heads), h = hq / a.group, r = hq - h * a.group;
  // the row's parts of the prefix, then those of its own keys
  int pre = 0, suf = 0;
  if (a.tc_ctas > 0) pre = tc_parts(a, t * a.group + r, h);
  const int64_t* base = a.base + (int64_t)(t / kRowBlock) * (kRowBlock + 1);
  if (a.pre_tiles > 0) {
    const int64_t share = share_of(a, a.base[a.max_suffix > 0 ? min(kRowBlock, a.T) : 0]);
    const int64_t f = first_unit(0, (t * a.group + r) / 16 * a.kv.kv_heads + h, a.pre_tiles);
    pre = (int)((f + a.pre_tiles - 1) / share - f / share) + 1;
  }
  if (a.max_suffix > 0) {
    const int nt = (suffix_keys(a, t) + kTile - 1) / kTile;
    if (nt > 0) {
      const int64_t share = share_of(a, base[min(kRowBlock, a.T - t / kRowBlock * kRowBlock)]);
      const int64_t f = first_unit(base[t % kRowBlock], h * (a.head_items / a.kv.kv_heads) + r / 16, nt);
      suf = (int)((f + nt - 1) / share - f / share) + 1;
    }
  }
  const int parts = pre + suf, skip = a.prefix_parts - pre;
  auto slot = [&](int p) { return (int64_t)(p < pre ? p : p + skip) * rh + i; };

  // warp w takes parts w, w + W, ..: lane i looks at the i-th of them
  __shared__ float tops[W];
  float2 ml = make_float2(-INFINITY, 0.f);
  float m = -INFINITY;
  for (int p = w + lane * W; p < parts; p += 32 * W) {
    const float2 x = a.ml_part[slot(p)];
    if (p < 32 * W) ml = x;
    m = fmaxf(m, x.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if constexpr (W > 1) {
    if (lane == 0) tops[w] = m;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < W; ++k) m = fmaxf(m, tops[k]);
  }
  const float top = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[V];
#pragma unroll
  for (int d = 0; d < V; ++d) acc[d] = 0.f;
  for (int p0 = 0; p0 < parts; p0 += 32 * W) {
    if (p0 > 0) ml = p0 + w + lane * W < parts ? a.ml_part[slot(p0 + w + lane * W)] : make_float2(-INFINITY, 0.f);
    const float f = ex2(ml.x - top);
    l = fmaf(ml.y, f, l);
    const int n = min(32, (parts - p0 - w + W - 1) / W);  // of this warp
    constexpr int U = W == 16 ? 8 : 4;  // parts in flight
    for (int j0 = 0; j0 < n; j0 += U) {
      float v[U][V];
#pragma unroll
      for (int k = 0; k < U; ++k) {
#pragma unroll
        for (int d = 0; d < V; ++d) v[k][d] = 0.f;
        if (j0 + k < n) {
          const float* src = a.o_part + slot(p0 + w + (j0 + k) * W) * D + lane * V;
          if constexpr (V == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[k][0] = x.x, v[k][1] = x.y;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float fj = __shfl_sync(0xffffffffu, f, j0 + k < n ? j0 + k : 0);
        if (j0 + k < n) {
#pragma unroll
          for (int d = 0; d < V; ++d) acc[d] = fmaf(v[k][d], fj, acc[d]);
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if constexpr (W > 1) {
    __syncthreads();  // tops is free
#pragma unroll
    for (int d = 0; d < V; ++d) red[w][lane * V + d] = acc[d];
    if (lane == 0) tops[w] = l;
    __syncthreads();
    if (w != 0) return;
    l = 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) l += tops[k];
#pragma unroll
    for (int d = 0; d < V; ++d) {
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) x += red[k][lane * V + d];
      acc[d] = x;
    }
  }
  const float inv = parts == 0 ? 0.f : 1.f / l;
#pragma unroll
  for (int d = 0; d < V; d += 2)
    *reinterpret_cast<__nv_bfloat162*>(a.out + i * D + lane * V + d) = __floats2bfloat162_rn(acc[d] * inv, acc[d + 1] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[i] = parts == 0 ? -INFINITY : m * kLn2 + logf(l);
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
  const uint64_t eb = f8 ? 1 : 2, row = a.kv.head_dim * eb, page = a.kv.page_size;
  const uint64_t inner = f8 ? a.kv.head_dim : 64, blocks = a.kv.head_dim / inner;  // elements of a swizzled row
  const uint64_t dims[5] = {inner, page, blocks, (uint64_t)a.kv.kv_heads, (uint64_t)a.kv.num_pages};
  const uint64_t strides[4] = {row, inner * eb, page * row, (uint64_t)a.kv.page_stride * eb};
  const uint32_t box[5] = {(uint32_t)inner, kTile, (uint32_t)blocks, 1, 1};
  return tc_encode_map(m, base, 5, dims, strides, box,
                       !f8 ? kTcMapBf16Sw128 : a.kv.head_dim == 128 ? kTcMapBytesSw128 : kTcMapBytesSw64);
}

// Warps of a row-head in the combine kernel: one where there are enough of them to fill the GPU,
// more where one would read many parts in turn. The whole call in us with 1 / 4 / 16: 128
// row-heads of 11 parts 11.3 / 10.6 / 11.4, 64 of 304 72.0 / 49.5 / 44.7, 512 of 40 32.6 / 26.6 /
// 34.7, 2,048 of 20 27.2 / 27.7 / 66, 8,192 of 5 23.6 / 37.4 / 174.
int join_warps(const Args& a) {
  const int parts = a.prefix_parts + a.suffix_parts;
  if (parts <= 32 && (int64_t)a.T * a.q_heads >= 1536) return 1;
  return parts <= 64 ? 4 : 16;
}

template <int D, bool F8>
int launch_all(const Args& a, cudaStream_t s) {
  using C = StreamCfg<D, F8>;
  int r = a.tc_ctas > 0 ? launch_prefix_tc(a, s) : PMOE_OK;
  if (r != PMOE_OK) return r;
  const char* what = "moe_prefix_attention";
  if (a.whole || a.pre_tiles > 0 || a.max_suffix > 0) {
    static SmemLimit limit[2];
    CUtensorMap mk, mv;
    const auto kernel = a.whole ? stream_kernel<D, F8, true> : stream_kernel<D, F8, false>;
    r = limit[a.whole > 0].set(reinterpret_cast<const void*>(kernel), C::kSmem, what);
    if (r == PMOE_OK) r = make_map(a, a.kv.k, &mk);
    if (r == PMOE_OK) r = make_map(a, a.kv.v, &mv);
    if (r != PMOE_OK) return r;
    if (a.whole)
      return launch(what, kernel, (unsigned)(a.T * a.head_items * a.whole), kThreads, C::kSmem, s, true, a.whole, mk, mv, a, 0);
    const int blocks = a.max_suffix > 0 ? (a.T + kRowBlock - 1) / kRowBlock : 1;
    for (int b = 0; b < blocks; ++b) {
      // a later block's launch does not overtake the one before it, which the combine kernel
      // would not wait for
      r = launch(what, kernel, a.warps / kWarps, kThreads, C::kSmem, s, b == 0, 1, mk, mv, a, b);
      if (r != PMOE_OK) return r;
    }
  }
  const unsigned rh = (unsigned)(a.T * a.q_heads);
  const int w = join_warps(a);
  if (w == 1) return launch(what, combine_kernel<D, 1>, (rh + 3) / 4, 128, 0, s, true, 1, a);
  if (w == 4) return launch(what, combine_kernel<D, 4>, rh, 128, 0, s, true, 1, a);
  return launch(what, combine_kernel<D, 16>, rh, 512, 0, s, true, 1, a);
}

struct Layout {
  size_t ml, base, bytes;
};
Layout scratch_layout(const Args& a) {
  const size_t n = (size_t)(a.prefix_parts + a.suffix_parts) * a.T * a.q_heads;
  Layout l;
  l.ml = n * a.kv.head_dim * 4;
  l.base = l.ml + n * 8;
  l.bytes = l.base + (size_t)((a.T + kRowBlock - 1) / kRowBlock) * (kRowBlock + 1) * 8;
  return l;
}

// What a call and every smaller one (in T, prefix_len and max_suffix) need at most: fewer rows
// may be cut into more parts, so the size of a call itself is no bound. R row-heads have
//   - of the prefix, in the stream kernel at most R (warps / items + 2) parts, where an item has
//     16 row-heads or fewer: 16 x 8 x SMs + 2 R; in the tensor-core kernel R (CTAs / groups + 2),
//     of groups of 256: 256 x SMs + 2 R;
//   - of their own keys R (most + 1), most <= max(4, 4 x warps / items);
//   - of neither more than one in 4 tiles of 16 keys, and 2.
size_t scratch_bound(const Args& a, int sms) {
  const int64_t R = (int64_t)a.T * a.q_heads;
  auto by_keys = [&](int keys) { return R * (((int64_t)keys + kTile - 1) / kTile / 4 + 2); };
  int64_t n = 0;
  if (a.prefix_len > 0) n += std::min<int64_t>(by_keys(a.prefix_len), 2 * R + 256ll * sms);
  if (a.max_suffix > 0) {
    const int64_t split = (4ll * kWarps * sms * a.q_heads + a.head_items - 1) / a.head_items;
    n += std::min<int64_t>(by_keys(a.max_suffix), R + std::max<int64_t>(4 * R, split));
  }
  return (size_t)n * (a.kv.head_dim * 4 + 8) + (size_t)((a.T + kRowBlock - 1) / kRowBlock) * (kRowBlock + 1) * 8;
}

// Plans the tensor-core prefix and returns the CTAs of the stream kernel. The one is bound by
// the tensor cores (or its own latency), the other by HBM, and a CTA of either fills an SM:
// side by side on shares of the SMs they end sooner than one after the other. Measured, in us
// (prefix kernel on 116 SMs and stream kernel on 36, against 152 and then 152): 256 rows on
// 32,768 + 1..1,024 keys 143 and 161. The stream's cost: 6 us, 8 tiles of 16 keys a us on an
// SM, 6.2 TB/s in all. The lengths are known on the device only, half of max_suffix is taken
// for their mean; with a quarter of the SMs at most the prefix loses a third at worst.
int split_sms(Args* a, int sms, int64_t key_bytes) {
  a->row_tiles = (a->T * a->group + kTcRows - 1) / kTcRows;
  a->tc_tiles = (a->prefix_len + kTcKeys - 1) / kTcKeys;
  const double keys = 0.5 * a->T * (double)a->max_suffix;
  auto stream = [&](int n) { return 6 + std::max(keys / kTile * a->head_items / (8.0 * n), keys * key_bytes / 6.2e6); };
  int prefix = 0, ctas = sms;
  double best = 0.92 * (prefix_tc_cost(*a, sms, &prefix) + stream(sms) - 3);
  for (int n = sms - sms / 4; n < sms && a->max_suffix > 0; ++n) {
    int used;
    const double t = std::max(prefix_tc_cost(*a, n, &used), stream(sms - n));
    if (t < best) best = t, prefix = used, ctas = sms - used;
  }
  plan_prefix_tc(a, prefix);
  return ctas;
}

// Checks shared by the call and its scratch size; fills the part plan. *sms: 0 for the current
// device's.
int plan(const pmoe_kv_desc* kv, int T, int q_heads, int prefix_len, int max_suffix, Args* a, int* sms) {
  const int r = check_kv(kv);
  if (r != PMOE_OK) return r;
  if (T < 0 || q_heads < 1 || q_heads % kv->kv_heads != 0 || prefix_len < 0 || max_suffix < 0) return PMOE_EINVAL;
  if ((int64_t)T * q_heads >= (1 << 24)) return PMOE_EINVAL;
  // no page list reaches further than the positions an int32 names
  if (prefix_len > INT32_MAX - 256 || max_suffix > INT32_MAX - 256) return PMOE_EINVAL;
  a->kv = *kv;
  a->T = T;
  a->q_heads = q_heads;
  a->group = q_heads / kv->kv_heads;
  a->group_magic = (uint32_t)((1ull << 32) / a->group + 1);
  a->prefix_len = prefix_len;
  a->max_suffix = max_suffix;
  if (a->group > kMaxGroup) return PMOE_EUNSUPPORTED;
  if (T == 0) return PMOE_OK;
  if (*sms == 0) *sms = sm_count();
  if (*sms == 0) return PMOE_ECUDA;

  const int rows = T * a->group, rts = (a->group + 15) / 16;
  a->head_items = kv->kv_heads * rts;
  int stream_ctas = *sms;
  a->prefix_parts = 0;
  const int64_t pre_rts = (rows + 15) / 16;
  const int64_t key_bytes = (int64_t)kv->kv_heads * kv->head_dim * (kv->dtype == PMOE_KV_E4M3 ? 2 : 4);  // a key's and value's
  // With few rows or keys the stream kernel takes the prefix along, 16 rows at a time, in one
  // launch less; from 340 keys x heads x row tiles an SM on the tensor cores are faster. In us,
  // prefix kernel / stream kernel, on 4 kv heads of 128 with 64 own keys a row: 64 rows of 32
  // heads 18.0 / 16.6 on 400 keys, 18.7 / 22.2 on 1,600; 8 rows 13.3 / 13.5 on 1,600, 15.9 /
  // 18.9 on 6,400; 3 rows 15.4 / 12.9 on 6,400, 23.3 / 22.9 on 25,600.
  const bool tc = prefix_len > 0 && pre_rts > 1 && pre_rts * kv->kv_heads * prefix_len > 340ll * *sms;
  // Short calls: a CTA or a cluster an item, without the launch that joins parts, as long as the
  // warps' chains of tiles are short. What is compared is a chain's tiles, 4 for start and end
  // and 1 for the exchange in a cluster. In us, in parts / with 1 / 2 / 4 / 8 CTAs an item (bf16
  // heads of 128, 4 kv heads): 1 row of 16 keys 9.3 / 3.8 / 4.7 / 4.7 / 4.6, of 564 9.4 / 7.6 / 7.6 /
  // 7.4 / 7.3, of 2,064 10.6 / 15.2 / 11.2 / 9.2 / 9.1, of 12,500 13.1 and 15.6 with 8; 16 rows of
  // 164 12.3 / 5.8 / 6.7, of 1,300 14.2 / 12.1 / 9.9; 76 rows (2 waves) of 300 13.4 / 12.4; 120 rows
  // (4 waves) of 164 14.0 / 18.9. Clusters of 8 fill half of the SMs at most (4 rows of 564 with
  // 16 of them: 13.4, with 16 clusters of 4 7.7). The prefix kernel starts late: against it (tensor
  // cores / whole) 32 rows of 1,300 keys take 15.6 / 12.3, of 1,664 15.6 / 13.6, 64 rows (2 waves)
  // of 514 15.9 / 15.2, 76 of 764 16.1 / 17.6.
  const int64_t tiles_whole = ((int64_t)prefix_len + kTile - 1) / kTile + ((int64_t)max_suffix + kTile - 1) / kTile;
  a->whole = 0;
  int64_t best = tc ? 20 : 14;
  for (int n = 1; n <= 8; n *= 2) {
    const int64_t ctas = (int64_t)T * a->head_items * n, waves = (ctas + *sms - 1) / *sms;
    if (n > 1 && ctas > (n == 8 ? 64 : 128)) break;
    const int64_t cost = waves * ((tiles_whole + n * kWarps - 1) / (n * kWarps) + 4) + (n > 1 ? 1 : 0);
    if (cost < best) best = cost, a->whole = n;
  }
  if (a->whole) {
    a->suffix_parts = 0;
    return PMOE_OK;
  }
  if (tc) stream_ctas = split_sms(a, *sms, key_bytes);
  a->warps = stream_ctas * kWarps;
  const int64_t tiles = ((int64_t)max_suffix + kTile - 1) / kTile;
  // A warp's run: 64 keys at least, and long enough that an item has few parts
  const int64_t items = (int64_t)T * a->head_items;
  const int64_t most = std::min<int64_t>(512, std::max<int64_t>(4, 4ll * a->warps / items));
  a->min_share = (int)std::max<int64_t>(4, (tiles + most - 1) / most);
  a->suffix_parts = tiles > 0 ? (int)((tiles - 1) / a->min_share + 2) : 0;
  if (prefix_len > 0 && !tc) {
    a->pre_tiles = (prefix_len + kTile - 1) / kTile;
    a->pre_items = (int)(pre_rts * kv->kv_heads);
    const int64_t units = (int64_t)(a->pre_tiles + kHead) * a->pre_items;
    const int64_t share = std::max<int64_t>(a->min_share, (units + a->warps - 1) / a->warps);
    a->prefix_parts = (int)((a->pre_tiles - 1) / share + 2);
  }
  return PMOE_OK;
}

}  // namespace
}  // namespace attn
}  // namespace pmoe

using namespace pmoe;

extern "C" int pmoe_attention_plan(const pmoe_kv_desc* kv, int T, int q_heads, int prefix_len, int max_suffix, int sms,
                                   pmoe_attention_plan_desc* out) {
  *out = pmoe_attention_plan_desc{};
  if (sms < 0) return PMOE_EINVAL;
  attn::Args a{};
  const int r = attn::plan(kv, T, q_heads, prefix_len, max_suffix, &a, &sms);
  if (r != PMOE_OK || T == 0) return r;
  out->scratch_bytes = attn::scratch_layout(a).bytes;
  out->scratch_bound = attn::scratch_bound(a, sms);
  out->cluster = a.whole;
  out->tc_ctas = a.tc_ctas;
  out->prefix_parts = a.prefix_parts;
  out->suffix_parts = a.suffix_parts;
  out->join_warps = a.whole ? 0 : attn::join_warps(a);
  return PMOE_OK;
}

extern "C" size_t moe_prefix_attention_scratch_bytes(const pmoe_kv_desc* kv, int T, int q_heads, int prefix_len,
                                                     int max_suffix) {
  pmoe_attention_plan_desc p;
  return pmoe_attention_plan(kv, T, q_heads, prefix_len, max_suffix, 0, &p) == PMOE_OK ? p.scratch_bound : 0;
}

extern "C" int moe_prefix_attention(const pmoe_kv_desc* kv, const void* q, int64_t q_stride, int T, int q_heads,
                                    float scale, const int32_t* prefix_pages, int prefix_len,
                                    const int32_t* page_table, int table_stride, int sequences, const int32_t* row_seq,
                                    const int32_t* suffix_len, int max_suffix, void* out, float* lse, void* scratch,
                                    size_t scratch_bytes, int32_t* err_out, void* stream) {
  attn::Args a{};
  // arguments first: the plan asks the device for its size
  if (check_kv(kv) == PMOE_OK && T > 0) {
    auto off = [](const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; };
    if (q == nullptr || out == nullptr || off(q, 16) || off(out, 16) || q_stride % 8 != 0 ||
        q_stride < (int64_t)q_heads * kv->head_dim || !(fabsf(scale) < INFINITY))
      return PMOE_EINVAL;
    if (prefix_len > 0 && (prefix_pages == nullptr || off(prefix_pages, 4))) return PMOE_EINVAL;
    if (max_suffix > 0 && (page_table == nullptr || suffix_len == nullptr || off(page_table, 4) || off(suffix_len, 4) ||
                           off(row_seq, 4) || sequences < 1 || (row_seq == nullptr && sequences < T) ||
                           table_stride < ((int64_t)max_suffix + kv->page_size - 1) / kv->page_size))
      return PMOE_EINVAL;
    if (off(lse, 4) || off(err_out, 4) || off(scratch, 16)) return PMOE_EINVAL;
  }
  int sms = 0;
  const int r = attn::plan(kv, T, q_heads, prefix_len, max_suffix, &a, &sms);
  if (r != PMOE_OK || T == 0) return r;
  const attn::Layout lay = attn::scratch_layout(a);
  if (scratch == nullptr || scratch_bytes < lay.bytes) return PMOE_EINVAL;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.scale = scale * attn::kLog2e;
  a.prefix_pages = prefix_pages;
  a.page_table = page_table;
  a.table_stride = table_stride;
  a.sequences = sequences;
  a.row_seq = row_seq;
  a.suffix_len = suffix_len;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = err_out;
  a.o_part = static_cast<float*>(scratch);
  a.ml_part = reinterpret_cast<float2*>(static_cast<uint8_t*>(scratch) + lay.ml);
  a.base = reinterpret_cast<int64_t*>(static_cast<uint8_t*>(scratch) + lay.base);
  cudaStream_t s = (cudaStream_t)stream;
  const bool f8 = kv->dtype == PMOE_KV_E4M3;
  if (kv->head_dim == 128) return f8 ? attn::launch_all<128, true>(a, s) : attn::launch_all<128, false>(a, s);
  return f8 ? attn::launch_all<64, true>(a, s) : attn::launch_all<64, false>(a, s);
}
