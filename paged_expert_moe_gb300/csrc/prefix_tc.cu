// The shared prefix of moe_prefix_attention on the tensor cores.
//
// All rows of a kv head (T tokens x its query heads) attend to the same keys, so the prefix
// is two matrix products a tile of 128 keys: S = Q K^T and O += P V, P the softmax weights.
// A CTA takes 256 rows (two 128-row query tiles, the M of an MMA) of one kv head and a range
// of key tiles; both query tiles share each K and V tile.
//
// Warps: 0-3 and 4-7 own one query tile each, a thread one row (a TMEM lane): scores from
// TMEM, weights back to TMEM in their place as the 16-bit A operand of the second product.
// Warp 8 issues the MMAs, in the order O0 += P0 V, S0 of the next tile, O1 += P1 V, S1 of
// the next tile, so that one query tile's softmax runs under the other's products. Warp 9
// loads K and V tiles by TMA, one box a page and 64 columns, into a ring of 128-key tiles (five
// of heads of 128, eight of 64); the bytes of an e4m3 cache land beside, and warps 12-15 convert
// them to fp16 (exact) into the same layout.
//
// The running maximum of a row moves only when a score exceeds it by 2^8 (any base gives the
// same quotient; weights up to 2^8 are far from overflow), so the accumulators in TMEM are
// rarely rescaled. Sums are fp32 of the unrounded weights.
//
// Work is split into equal runs of (group, key tile) units, one run per CTA and at most one CTA
// an SM: a group's parts are joined by the combine kernel.
//
// Bound: the tensor cores. Of the 3,050 cycles of a tile (256 rows x 128 keys, heads of 128) the
// issuing warp spends 2,270 handing over its 32 MMAs, which run no faster, 480 until it sees
// the next K and V, 370 until it sees P; the softmax of a query tile takes 1,370, under the other
// one's products. Measured with 256 rows of 32 heads on 32,768 keys (4 kv heads of 128): 103-106
// us, 1,300-1,335 TFLOP/s, 0.69-0.71 of a large matrix product; heads of 64 76 us (an MMA of 64
// columns takes as long as one of 128); e4m3 113 and 84 us (152 and 87 when the converting warps
// read the cache themselves, a tile ahead in registers: too little in flight). Few rows are bound by a run's start and end, 9 us.
#include "attn_tc.cuh"
#include "tc_gemm.h"

#include <algorithm>

namespace pmoe {
namespace attn {
namespace {

using namespace tc;

template <int D, bool F8>
struct TcCfg {
  static constexpr int kTileBytes = kTcKeys * D * 2;      // one K or V tile, 16-bit operands
  static constexpr int kQBytes = 128 * D * 2;             // one query tile
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
  static constexpr int kRawBytes = kTcKeys * D, kRawRing = F8 && D == 64 ? kSlots * kRawBytes : 0;
  static __device__ __forceinline__ uint8_t* raw(uint8_t* smem, uint32_t slot) {
    return D == 64 ? smem + kRing + slot * kRawBytes : smem + slot * kTileBytes + kRawBytes;
  }
  static constexpr int kSmem = kRing + kRawRing + 2 * kQBytes + 1024 /* alignment */ + 1024 /* row factors */ + 512;
  static constexpr int kTmemCols = 512;                   // S0 S1 at 0 and 128, O0 O1 at 256 and 384
};

struct Bars {
  uint64_t full[8], empty[8], raw[8];
  uint64_t sfull[2], pready[2], odone[2], qfull[2], staged[2], drain;
  uint32_t tmem;
  int abort;
};

// One segment of a CTA's run: key tiles [t0, t1) of one group.
struct Segment {
  int h, row0, rows, nq, t0, t1, part;
};
__device__ __forceinline__ bool segment(const Args& a, int64_t* u, int64_t end, Segment* s) {
  if (*u >= end) return false;
  const int g = (int)(*u / a.tc_tiles);
  s->t0 = (int)(*u - (int64_t)g * a.tc_tiles);
  s->t1 = (int)min((int64_t)a.tc_tiles, s->t0 + (end - *u));
  s->h = g % a.kv.kv_heads;
  s->row0 = g / a.kv.kv_heads * kTcRows;
  s->rows = min(kTcRows, a.T * a.group - s->row0);
  s->nq = s->rows > 128 ? 2 : 1;
  s->part = (int)blockIdx.x - tc_cta_of((int64_t)g * a.tc_tiles, tc_units(a), a.tc_ctas);
  *u += s->t1 - s->t0;
  return true;
}

template <int D, bool F8>
__global__ void __launch_bounds__(TcCfg<D, F8>::kThreads, 1)
    prefix_tc_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Args a) {
  using C = TcCfg<D, F8>;
  constexpr int kSlots = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qs = smem + C::kRing + C::kRawRing;
  float* qmul = reinterpret_cast<float*>(qs + 2 * C::kQBytes);  // [256]
  Bars& b = *reinterpret_cast<Bars*>(qmul + 256);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_flag = &b.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&b.full[i], F8 ? 4 : 1);
      mbar_init(&b.empty[i], 1);
      mbar_init(&b.raw[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&b.sfull[i], 1);
      mbar_init(&b.pready[i], 4);
      mbar_init(&b.odone[i], 1);
      mbar_init(&b.qfull[i], 4);
      mbar_init(&b.staged[i], 4);
    }
    mbar_init(&b.drain, 1);
    b.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  pdl_wait();     // the cache and q may come from the kernel ahead
  pdl_trigger();  // the stream kernel may take the SMs that this one is done with
  __syncthreads();
  // The issuing warp allocates all 512 columns: the base is column 0, lane 0. The other roles
  // touch TMEM only after its first products.
  constexpr uint32_t tmem = 0;
  const int64_t units = tc_units(a);
  int64_t u = (int64_t)blockIdx.x * units / a.tc_ctas;
  const int64_t end = (int64_t)(blockIdx.x + 1) * units / a.tc_ctas;
  const int psh = 31 - __clz(a.kv.page_size);
  Segment sg;

  if (warp < 8) {
    // ---------------- softmax: one thread a row
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kSoftmaxRegs));
    const int q = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = lanes + q * 128, to = lanes + 256 + q * 128;
    constexpr int LPR = D / 8;  // threads of a row while Q is loaded
    uint32_t n = 0, segs = 0;   // tiles and segments so far
    bool ok = true;
    while (ok && segment(a, &u, end, &sg)) {
      if (q >= sg.nq) continue;
      // the query tile, K-major with the 128-byte swizzle; rows beyond the last are zero.
      // What a score is multiplied by, scale x key scale x the row's power of two, has to be above
      // zero: then the largest score stays the largest, and a masked one -inf. So its sign goes
      // into Q, and a row whose factor is 0 (or vanishes in fp32) has Q = 0 and factor 1.
      const float ks = F8 ? a.kv.k_scale[sg.h] : 1.f;
      const uint32_t flip = (a.scale < 0.f) != (ks < 0.f) ? 0x80008000u : 0u;
      const int c = row % LPR;
      uint4 v[LPR];  // LPR rows a thread, all in flight
#pragma unroll
      for (int p = 0; p < LPR; ++p) {
        const int i = q * 128 + row / LPR + p * (128 / LPR);
        v[p] = make_uint4(0, 0, 0, 0);
        if (i < sg.rows) {
          const int rr = sg.row0 + i, t = row_token(a, rr);
          v[p] = __ldg(reinterpret_cast<const uint4*>(a.q + (int64_t)t * a.q_stride +
                                                      (sg.h * a.group + rr - t * a.group) * D + c * 8));
        }
      }
#pragma unroll
      for (int p = 0; p < LPR; ++p) {
        const int r = row / LPR + p * (128 / LPR);
        uint32_t w[4] = {v[p].x ^ flip, v[p].y ^ flip, v[p].z ^ flip, v[p].w ^ flip};
        if (F8) {
          float mx = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xffff0000u))));
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const int e = row_exponent(mx);
          const float factor = fabsf(a.scale) * fabsf(ks) * pow2(e), down = factor != 0.f ? pow2(-e) : 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = pack2<true>(__uint_as_float(w[k] << 16) * down, __uint_as_float(w[k] & 0xffff0000u) * down);
          if (c == 0) qmul[q * 128 + r] = factor != 0.f ? factor : 1.f;
        }
        *reinterpret_cast<uint4*>(qs + q * C::kQBytes + (c / 8) * (128 * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_async();
      warp_arrive(&b.qfull[q]);
      // the row factors of all threads
      if (!warp_wait(&b.qfull[q], segs++ & 1, abort_flag, a.err)) break;
      // (bf16, scale 0: times 2^-149 the largest score is below 2^-20)
      const float mul = F8 ? qmul[q * 128 + row] : a.scale != 0.f ? fabsf(a.scale) : __uint_as_float(1);

      float m = -INFINITY, l = 0.f;
      for (int t = sg.t0; t < sg.t1; ++t, ++n) {
        if (!warp_wait(&b.sfull[q], n & 1, abort_flag, a.err)) {
          ok = false;
          break;
        }
        fence_after();
        float s[128];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, reinterpret_cast<uint32_t*>(s) + 32 * i);
        tmem_wait_ld();
        const int valid = a.prefix_len - t * kTcKeys;
        if (valid < kTcKeys) {
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i >= valid) s[i] = -INFINITY;
        }
        float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 128; i += 2) x[(i >> 1) & 3] = max3(x[(i >> 1) & 3], s[i], s[i + 1]);
        const float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * mul;
        if (t == sg.t0) {
          m = mx;
        } else {
          const bool grow = mx > m + 8.f;
          if (__any_sync(0xffffffffu, grow)) {
            // the products so far are done: these scores were issued after them
            const float f = grow ? ex2(m - mx) : 1.f;
            if (grow) m = mx;
            l *= f;
#pragma unroll 1
            for (int i = 0; i < D; i += 16) {
              uint32_t o[16];
              tmem_ld16(to + i, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(to + i, o);
            }
          }
        }
        const float base = m == -INFINITY ? 0.f : m;
        const uint64_t mul2 = pair(mul, mul), base2 = pair(-base, -base);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t p[16];
          const float* sc = s + 32 * i;
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float y, z;
            unpair(fma2(pair(sc[2 * k], sc[2 * k + 1]), mul2, base2), y, z);
            y = ex2(y), z = ex2(z);
            sum[k & 1] = add2(sum[k & 1], pair(y, z));
            p[k] = pack2<F8>(y, z);
          }
          tmem_st16(ts + 16 * i, p);
        }
        tmem_wait_st();
        fence_before();
        warp_arrive(&b.pready[q]);
        float y, z;
        unpair(add2(sum[0], sum[1]), y, z);
        l += y + z;
      }
      if (!ok) break;
      if (!warp_wait(&b.odone[q], (segs - 1) & 1, abort_flag, a.err)) break;
      fence_after();
      // 32 columns at a time through shared memory (the query tile's, which is done with), so
      // that a store covers whole lines: 8 threads a row of 128 bytes, whose 16-byte chunks
      // are swizzled by the row
      const float vs = F8 ? a.kv.v_scale[sg.h] : 1.f;
      const int64_t part0 = (int64_t)sg.part * a.T * a.q_heads;
      uint8_t* stage = qs + q * C::kQBytes + (warp & 3) * (C::kQBytes / 4);
      float* dst[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = q * 128 + (warp & 3) * 32 + 4 * k + (lane >> 3), rr = sg.row0 + i, tok = row_token(a, rr);
        dst[k] = i < sg.rows ? a.o_part + (part0 + (int64_t)tok * a.q_heads + sg.h * a.group + rr - tok * a.group) * D + (lane & 7) * 4
                             : nullptr;
      }
#pragma unroll
      for (int d = 0; d < D; d += 32) {
        uint32_t o[32];
        tmem_ld32(to + d, o);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          *reinterpret_cast<float4*>(stage + lane * 128 + ((k ^ (lane & 7)) << 4)) =
              make_float4(__uint_as_float(o[4 * k]) * vs, __uint_as_float(o[4 * k + 1]) * vs,
                          __uint_as_float(o[4 * k + 2]) * vs, __uint_as_float(o[4 * k + 3]) * vs);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = 4 * k + (lane >> 3);
          const float4 v = *reinterpret_cast<const float4*>(stage + r * 128 + (((lane & 7) ^ (r & 7)) << 4));
          if (dst[k] != nullptr) *reinterpret_cast<float4*>(dst[k] + d) = v;
        }
        __syncwarp();
      }
      const int i = q * 128 + row;
      if (i < sg.rows) {
        const int rr = sg.row0 + i, tok = row_token(a, rr);
        a.ml_part[part0 + (int64_t)tok * a.q_heads + sg.h * a.group + rr - tok * a.group] = make_float2(m, l);
      }
      // every warp is done with its stage before Q is written again
      warp_arrive(&b.staged[q]);
      if (!warp_wait(&b.staged[q], (segs - 1) & 1, abort_flag, a.err)) break;
      fence_before();
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kMmaRegs));
    if (warp == 8) {
    // ---------------- MMA issuer
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&b.tmem)),
                 "r"(C::kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    const uint32_t is = idesc_bf16(128, kTcKeys) & (F8 ? ~((1u << 7) | (1u << 10)) : ~0u);
    const uint32_t io = (idesc_bf16(128, D) & (F8 ? ~((1u << 7) | (1u << 10)) : ~0u)) | (1u << 16);  // B: N contiguous
    const uint32_t ring = smem_u32(smem), qa = smem_u32(qs);
    uint32_t kv = 0;               // K and V tiles so far
    uint32_t seg[2] = {0, 0};      // segments of each query tile so far
    uint32_t pn[2] = {0, 0};       // products with V of each query tile so far
    bool ok = true;
    auto wait_kv = [&](uint32_t i) {
      return warp_wait(&b.full[i % kSlots], (i / kSlots) & 1, abort_flag, a.err);
    };
    auto scores = [&](int q, uint32_t slot, bool last) {  // last: of the query tiles on this slot
      if (converged_lane()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k / 4) * (128 * 128) + (k % 4) * 32;
          mma_bf16(tmem + q * 128, sw128_desc(qa + q * C::kQBytes + off), sw128_desc(ring + slot * C::kTileBytes + off), is,
                   k > 0);
        }
        mma_commit(&b.sfull[q]);
        if (last) mma_commit(&b.empty[slot]);
      }
      __syncwarp();
    };
    while (ok && segment(a, &u, end, &sg)) {
      for (int q = 0; q < sg.nq && ok; ++q) {
        ok = warp_wait(&b.qfull[q], seg[q] & 1, abort_flag, a.err);
        ++seg[q];
      }
      if (!ok || !wait_kv(kv)) break;
      fence_after();
      for (int q = 0; q < sg.nq; ++q) scores(q, kv % kSlots, q + 1 == sg.nq);
      for (int t = sg.t0; t < sg.t1; ++t, kv += 2) {
        const uint32_t vslot = (kv + 1) % kSlots;
        const bool more = t + 1 < sg.t1;
        if (!wait_kv(kv + 1) || (more && !wait_kv(kv + 2))) {
          ok = false;
          break;
        }
        const int valid = a.prefix_len - t * kTcKeys;
        if (!F8 && valid < kTcKeys) {
          // values beyond the prefix may be anything, and 0 x NaN is NaN
          for (int i = valid * 8 + lane; i < kTcKeys * 8; i += 32)
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
              *reinterpret_cast<uint4*>(smem + vslot * C::kTileBytes + hf * (kTcKeys * 128) + i * 16) = make_uint4(0, 0, 0, 0);
          fence_async();
          __syncwarp();
        }
        for (int q = 0; q < sg.nq; ++q) {
          if (!warp_wait(&b.pready[q], pn[q] & 1, abort_flag, a.err)) {
            ok = false;
            break;
          }
          ++pn[q];
          fence_after();
          if (converged_lane()) {
#pragma unroll
            for (int k = 0; k < kTcKeys / 16; ++k)
              mma_f16_ts(tmem + 256 + q * 128, tmem + q * 128 + k * 8, v_desc(ring + vslot * C::kTileBytes + k * 2048), io,
                         t > sg.t0 || k > 0);
            if (!more) mma_commit(&b.odone[q]);
            if (q + 1 == sg.nq) mma_commit(&b.empty[vslot]);
          }
          __syncwarp();
          if (more) scores(q, (kv + 2) % kSlots, q + 1 == sg.nq);
        }
        if (!ok) break;
      }
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
    const int box = min(a.kv.page_size, kTcKeys), boxes = kTcKeys / box;
    uint32_t kv = 0;
    bool ok = true;
    while (ok && segment(a, &u, end, &sg)) {
      for (int t = sg.t0; t < sg.t1 && ok; ++t) {
        const int used = min(boxes, (a.prefix_len - t * kTcKeys + box - 1) / box);
        const int pb = lane / kHalves, hf = lane % kHalves;
        const int key = t * kTcKeys + pb * box;
        int id = 0;
        if (pb < used) {
          id = __ldg(a.prefix_pages + (key >> psh));
          if ((unsigned)id >= (unsigned)a.kv.num_pages) {
            if (a.err != nullptr) atomicOr(a.err, kErrBadPage);
            id = a.kv.num_pages;  // out of the map's range: reads as zeros
          }
        }
        for (int v = 0; v < 2; ++v, ++kv) {
          const uint32_t slot = kv % kSlots;
          if (!warp_wait(&b.empty[slot], ((kv / kSlots) & 1) ^ 1, abort_flag, a.err)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&arrive[slot], used * box * D * kBytes);
          __syncwarp();
          uint8_t* dst = F8 ? C::raw(smem, slot) + pb * box * D : smem + slot * C::kTileBytes + hf * (kTcKeys * 128) + pb * box * 128;
          if (pb < used)
            tma_load_4d(dst, v ? &map_v : &map_k, &arrive[slot], hf * 64, key & (a.kv.page_size - 1), sg.h, id);
        }
      }
    }
    // copies in flight land before the CTA leaves, even where another role gave up
    for (uint32_t i = kv > kSlots ? kv - kSlots : 0; i < kv; ++i) {
      const long long t0 = clock64();
      while (!mbar_try_wait(&arrive[i % kSlots], (i / kSlots) & 1) && clock64() - t0 < kWaitLimit) {
      }
    }
    }
  } else if constexpr (F8) {
    // ---------------- e4m3 conversion: 16 codes a thread and step, to fp16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLoaderRegs));
    constexpr int CH = D / 16;  // 16-code chunks of a row
    constexpr int N = kTcKeys * CH / 128;
    const int tid = threadIdx.x - 12 * 32, ch = tid % CH, r0 = tid / CH;
    uint32_t kv = 0;
    bool ok = true;
    while (ok && segment(a, &u, end, &sg)) {
      for (int i2 = 2 * sg.t0; i2 < 2 * sg.t1; ++i2, ++kv) {  // K and V of each tile
        const uint32_t slot = kv % kSlots;
        if (!warp_wait(&b.raw[slot], (kv / kSlots) & 1, abort_flag, a.err)) {
          ok = false;
          break;
        }
        const uint8_t* src = C::raw(smem, slot);
        const int valid = a.prefix_len - i2 / 2 * kTcKeys;
        uint4 raw[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = r0 + i * (128 / CH);
          const int at = D == 128 ? r * 128 + ((ch ^ (r & 7)) << 4) : r * 64 + ((ch ^ ((r >> 1) & 3)) << 4);
          // values beyond the prefix may be anything, and 0 x NaN is NaN
          raw[i] = r < valid ? *reinterpret_cast<const uint4*>(src + at) : make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int r = r0 + i * (128 / CH);
          uint8_t* dst = smem + slot * C::kTileBytes + (ch / 4) * (kTcKeys * 128) + r * 128;
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

int make_map(const Args& a, void* base, CUtensorMap* m) {
  const bool f8 = a.kv.dtype == PMOE_KV_E4M3;
  const uint64_t D = a.kv.head_dim, page = a.kv.page_size, eb = f8 ? 1 : 2;
  const uint64_t dims[4] = {D, page, (uint64_t)a.kv.kv_heads, (uint64_t)a.kv.num_pages};
  const uint64_t strides[3] = {D * eb, page * D * eb, (uint64_t)a.kv.page_stride * eb};
  const uint32_t box[4] = {f8 ? (uint32_t)D : 64u, (uint32_t)std::min<uint64_t>(page, kTcKeys), 1, 1};
  return tc_encode_map(m, base, 4, dims, strides, box, !f8 ? kTcMapBf16Sw128 : D == 128 ? kTcMapBytesSw128 : kTcMapBytesSw64);
}

template <int D, bool F8>
int launch(const Args& a, cudaStream_t s) {
  using C = TcCfg<D, F8>;
  CUtensorMap mk, mv;
  static SmemLimit limit;
  int r = make_map(a, a.kv.k, &mk);
  if (r == PMOE_OK) r = make_map(a, a.kv.v, &mv);
  if (r != PMOE_OK) return r;
  r = limit.set(reinterpret_cast<const void*>(prefix_tc_kernel<D, F8>), C::kSmem, "moe_prefix_attention");
  if (r != PMOE_OK) return r;
  return pmoe::launch("moe_prefix_attention", prefix_tc_kernel<D, F8>, a.tc_ctas, C::kThreads, C::kSmem, s, true, 1, mk, mv, a);
}

}  // namespace

// What the prefix takes on at most `ctas` CTAs, in us, and how many it then uses: 9 for a run,
// 1.9 a tile of heads of 128 (1.4 of 64; 2.1 and 1.5 with e4m3) and 5.5 where a run crosses
// from one group into the next (query rows to load, a part to write). Runs that divide the
// groups evenly do not, and more runs than the tiles need only leave more parts: 64 rows on
// 8,192 keys take 20.9 us with 128 CTAs of 4 tiles each, 22.3 with 152 of 3 or 4.
double prefix_tc_cost(const Args& a, int ctas, int* used) {
  const bool f8 = a.kv.dtype == PMOE_KV_E4M3;
  const double tile = a.kv.head_dim == 128 ? (f8 ? 2.1 : 1.9) : (f8 ? 1.5 : 1.4);
  const int64_t units = tc_units(a), groups = units / a.tc_tiles;
  const int64_t run = (units + ctas - 1) / ctas;
  int64_t n = (units + run - 1) / run;
  double cost = 9 + tile * run + (n % groups != 0 ? 5.5 : 0);
  if (ctas >= groups) {
    const int64_t run1 = (a.tc_tiles + ctas / groups - 1) / (ctas / groups);
    const double cost1 = 9 + tile * run1;
    if (cost1 <= cost) cost = cost1, n = groups * ((a.tc_tiles + run1 - 1) / run1);
  }
  *used = (int)n;
  return cost;
}

void plan_prefix_tc(Args* a, int ctas) {
  a->tc_ctas = ctas;
  a->prefix_parts = 0;
  const int64_t units = tc_units(*a);
  for (int64_t u = 0; u < units; u += a->tc_tiles)
    a->prefix_parts = std::max(a->prefix_parts, tc_cta_of(u + a->tc_tiles - 1, units, ctas) - tc_cta_of(u, units, ctas) + 1);
}

int launch_prefix_tc(const Args& a, cudaStream_t s) {
  const bool f8 = a.kv.dtype == PMOE_KV_E4M3;
  if (a.kv.head_dim == 128) return f8 ? launch<128, true>(a, s) : launch<128, false>(a, s);
  return f8 ? launch<64, true>(a, s) : launch<64, false>(a, s);
}

}  // namespace attn
}  // namespace pmoe
