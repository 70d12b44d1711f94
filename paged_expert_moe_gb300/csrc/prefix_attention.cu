// moe_prefix_attention: attention over a paged cache for a batch that shares a prefix.
#include "attn.cuh"

#include <algorithm>
#include <cuda_fp16.h>
#include <math.h>

namespace pmoe {
namespace attn {
namespace {

constexpr int kTile = 64;       // keys of a tile
constexpr int kStages = 3;
constexpr int kThreads = 128;
constexpr int kMaxChunk = 4096; // keys of a part: its page ids lie in shared memory

__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// 16 bytes to shared memory; nothing is read and zeros are written where !live
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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

// Where 16-byte chunk c of key row r lies in a tile, so that the 8 rows (or the 2 rows x 4
// chunks) of one shared-memory access phase fall on distinct banks.
template <int ROWB, bool F8>
__device__ __forceinline__ uint32_t place(int r, int c) {
  int x;
  if (ROWB == 64) x = (r >> 1) & 3;
  else if (F8) x = ((r & 1) << 2) | ((r >> 1) & 3);
  else x = r & 7;
  return (uint32_t)(r * ROWB + ((c ^ x) << 4));
}

template <int D, bool F8>
struct StreamCfg {
  static constexpr int kRow = D * (F8 ? 1 : 2);         // bytes of a key row
  static constexpr int kTileBytes = kTile * kRow;       // of K, and of V
  static constexpr int kRing = kStages * 2 * kTileBytes;
  static constexpr int kMerge = 4 * 16 * (D + 4) * 4;   // the warps' sums at the end
  static constexpr int kSmem = (kRing > kMerge ? kRing : kMerge) + (kMaxChunk / 16) * 4;
};

// One CTA: up to 16 * WM query rows of one kv head against the keys [k0, k1) of one page
// list. The 4 warps are WM row tiles x 4 / WM key groups; each keeps its own running
// maximum and sum, joined at the end.
// rows: row i is head `h * group + i % group` of token t0 + i / group.
template <int D, bool F8, int WM>
__device__ void stream_part(const Args& a, uint8_t* smem, const int32_t* pages, int h, int row0, int rows, int k0,
                            int k1, int part) {
  using C = StreamCfg<D, F8>;
  constexpr int WK = 4 / WM, KW = kTile / WK, NT = KW / 8;  // keys of a warp, its 8-key tiles
  constexpr int CH = C::kRow / 16;                          // 16-byte chunks of a row
  int32_t* ids = reinterpret_cast<int32_t*>(smem + (C::kRing > C::kMerge ? C::kRing : C::kMerge));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wm = warp % WM, wk = warp / WM, g = lane >> 2, c = lane & 3;
  const int psh = 31 - __clz(a.kv.page_size);

  const int p0 = k0 >> psh, np = ((k1 - 1) >> psh) - p0 + 1;
  for (int i = tid; i < np; i += kThreads) {
    int id = pages[p0 + i];
    if ((unsigned)id >= (unsigned)a.kv.num_pages) {
      if (a.err != nullptr) atomicOr(a.err, kErrBadPage);
      id = -1;
    }
    ids[i] = id;
  }

  // query fragments; rows beyond the last are zero
  uint32_t qf[D / 16][4];
  float qmul[2];  // what a score of rows g and g + 8 is multiplied by
  {
    const __nv_bfloat16* qp[2];
    bool live[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = wm * 16 + g + 8 * e;
      live[e] = i < rows;
      const int r = row0 + (live[e] ? i : 0);
      qp[e] = a.q + (int64_t)(r / a.group) * a.q_stride + (h * a.group + r % a.group) * D;
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
      uint2 raw[2][D / 16];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = 0.f;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          raw[e][k] = live[e] ? __ldg(reinterpret_cast<const uint2*>(qp[e] + (k >> 2) * 64 + 16 * c + (k & 3) * 4))
                              : make_uint2(0, 0);
          const uint32_t w[2] = {raw[e][k].x, raw[e][k].y};
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const int ex = row_exponent(mx);
        const float down = pow2(-ex);
        qmul[e] = a.scale * a.kv.k_scale[h] * pow2(ex);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t w[2] = {raw[e][k].x, raw[e][k].y};
#pragma unroll
          for (int i = 0; i < 2; ++i)
            qf[k][2 * i + e] = pack2<true>(__uint_as_float(w[i] << 16) * down, __uint_as_float(w[i] & 0xffff0000u) * down);
        }
      }
    }
  }
  __syncthreads();  // ids

  const uint8_t* kb = static_cast<const uint8_t*>(a.kv.k);
  const uint8_t* vb = static_cast<const uint8_t*>(a.kv.v);
  const int64_t page_bytes = a.kv.page_stride * (F8 ? 1 : 2);
  const int64_t head_off = (int64_t)h * a.kv.page_size * C::kRow;
  const int tiles = (k1 - k0 + kTile - 1) / kTile;
  const uint32_t ring = smem_u32(smem);
  auto load = [&](int tile) {
    if (tile < tiles) {
      const uint32_t ks = ring + (tile % kStages) * 2 * C::kTileBytes, vs = ks + C::kTileBytes;
      const int ch = tid % CH;
#pragma unroll
      for (int r = tid / CH; r < kTile; r += kThreads / CH) {
        const int key = k0 + tile * kTile + r;
        int id = -1;
        if (key < k1) id = ids[(key >> psh) - p0];
        const int64_t off = id < 0 ? 0 : (int64_t)id * page_bytes + head_off + (int64_t)(key & (a.kv.page_size - 1)) * C::kRow + ch * 16;
        const uint32_t at = place<C::kRow, F8>(r, ch);
        cp16(ks + at, kb + off, id >= 0);
        cp16(vs + at, vb + off, id >= 0);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) load(i);

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  for (int tile = 0; tile < tiles; ++tile) {
    cp_wait<kStages - 2>();
    __syncthreads();  // the tile has landed, and every warp is done with the one before it
    load(tile + kStages - 1);
    const uint32_t ks = ring + (tile % kStages) * 2 * C::kTileBytes, vs = ks + C::kTileBytes;

    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      if constexpr (!F8) {
        const int r = wk * KW + n * 8 + (lane & 7);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          uint32_t b[4];
          ldsm4(b, ks + place<C::kRow, F8>(r, k * 4 + (lane >> 3)));
          mma<false>(s[n], qf[2 * k], b[0], b[1]);
          mma<false>(s[n], qf[2 * k + 1], b[2], b[3]);
        }
      } else {
        const int r = wk * KW + n * 8 + g;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          uint32_t b[4];
          lds128(b, ks + place<C::kRow, F8>(r, i * 4 + c));
#pragma unroll
          for (int k = 0; k < 4; ++k) mma<true>(s[n], qf[4 * i + k], e4m3x2(b[k] & 0xffffu), e4m3x2(b[k] >> 16));
        }
      }
    }
    // keys beyond the part; then the running maximum and the weights
    const int kw = k0 + tile * kTile + wk * KW;
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[n][i] = kw + n * 8 + 2 * c + (i & 1) < k1 ? s[n][i] * qmul[i >> 1] : -INFINITY;
        mx[i >> 1] = fmaxf(mx[i >> 1], s[n][i]);
      }
    float base[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      base[e] = mx[e] == -INFINITY ? 0.f : mx[e];
      const float f = ex2(m[e] - base[e]);
      m[e] = mx[e];
      l[e] *= f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) o[i][2 * e] *= f, o[i][2 * e + 1] *= f;
    }
    uint32_t pf[NT / 2][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float p[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] = ex2(s[n][i] - base[i >> 1]);
        l[i >> 1] += p[i];
      }
      pf[n / 2][(n & 1) * 2] = pack2<F8>(p[0], p[1]);
      pf[n / 2][(n & 1) * 2 + 1] = pack2<F8>(p[2], p[3]);
    }
#pragma unroll
    for (int n = 0; n < NT / 2; ++n) {
      const int r = wk * KW + n * 16 + (lane & 15);
      if constexpr (!F8) {
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t b[4];
          ldsm4t(b, vs + place<C::kRow, F8>(r, i * 2 + (lane >> 4)));
          mma<false>(o[2 * i], pf[n], b[0], b[1]);
          mma<false>(o[2 * i + 1], pf[n], b[2], b[3]);
        }
      } else {
        // a 16-bit element of the transposed load is 2 values of one key: the even and the
        // odd elements of 16 form an 8-column tile each
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          uint32_t b[4];
          ldsm4t(b, vs + place<C::kRow, F8>(r, i * 2 + (lane >> 4)));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            mma<true>(o[4 * i + 2 * j], pf[n], e4m3x2(__byte_perm(b[2 * j], 0, 0x4420)),
                      e4m3x2(__byte_perm(b[2 * j + 1], 0, 0x4420)));
            mma<true>(o[4 * i + 2 * j + 1], pf[n], e4m3x2(__byte_perm(b[2 * j], 0, 0x4431)),
                      e4m3x2(__byte_perm(b[2 * j + 1], 0, 0x4431)));
          }
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
  }
  cp_wait<0>();
  __syncthreads();  // the ring becomes the merge buffer

  // join the key groups of each row tile: buf[warp][16][D + 4], (m, l) after each row
  float* buf = reinterpret_cast<float*>(smem) + warp * 16 * (D + 4);
  const float vscale = F8 ? a.kv.v_scale[h] : 1.f;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    float* row = buf + (g + 8 * e) * (D + 4);
    if constexpr (!F8) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) *reinterpret_cast<float2*>(row + i * 8 + 2 * c) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        *reinterpret_cast<float4*>(row + i * 16 + 4 * c) =
            make_float4(o[2 * i][2 * e], o[2 * i + 1][2 * e], o[2 * i][2 * e + 1], o[2 * i + 1][2 * e + 1]);
    }
    if (c == 0) row[D] = m[e], row[D + 1] = l[e];
  }
  __syncthreads();
  const int64_t rh = (int64_t)a.T * a.q_heads;
  for (int i = warp; i < rows; i += 4) {
    const float* src = reinterpret_cast<float*>(smem) + ((i / 16) * 16 + (i % 16)) * (D + 4);  // key group 0
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < WK; ++w) mm = fmaxf(mm, src[w * WM * 16 * (D + 4) + D]);
    const float bb = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f, acc[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d) acc[d] = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const float* s2 = src + w * WM * 16 * (D + 4);
      const float f = ex2(s2[D] - bb);
      ll = fmaf(s2[D + 1], f, ll);
#pragma unroll
      for (int d = 0; d < D / 32; ++d) acc[d] = fmaf(s2[d * 32 + lane], f, acc[d]);
    }
    const int r = row0 + i;
    const int64_t at = (int64_t)part * rh + (int64_t)(r / a.group) * a.q_heads + h * a.group + r % a.group;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) a.o_part[at * D + d * 32 + lane] = acc[d] * vscale;
    if (lane == 0) a.ml_part[at] = make_float2(mm, ll);
  }
}

template <int D, bool F8, int WM>
__global__ void __launch_bounds__(kThreads) stream_kernel(const Args a, int prefix_blocks) {
  extern __shared__ __align__(128) uint8_t smem[];
  int b = blockIdx.x;
  if (b < prefix_blocks) {
    const int part = b % a.prefix_parts;
    b /= a.prefix_parts;
    const int h = b % a.kv.kv_heads, tile = b / a.kv.kv_heads;
    const int row0 = tile * 16 * WM, rows = min(16 * WM, a.T * a.group - row0);
    const int k0 = part * a.prefix_chunk, k1 = min(a.prefix_len, k0 + a.prefix_chunk);
    stream_part<D, F8, WM>(a, smem, a.prefix_pages, h, row0, rows, k0, k1, part);
    return;
  }
  b -= prefix_blocks;
  const int part = b % a.suffix_parts;
  b /= a.suffix_parts;
  const int h = b % a.kv.kv_heads, t = b / a.kv.kv_heads;
  const int n = suffix_keys(a, t), k0 = part * a.suffix_chunk;
  if (k0 >= n) return;
  const int seq = a.row_seq != nullptr ? a.row_seq[t] : t;
  const bool ok = (unsigned)seq < (unsigned)a.sequences;
  if (!ok && a.err != nullptr) atomicOr(a.err, kErrBadPage);
  // an invalid row reads row 0 of the table: in bounds, and its output is undefined
  stream_part<D, F8, WM>(a, smem, a.page_table + (int64_t)(ok ? seq : 0) * a.table_stride, h, t * a.group, a.group, k0,
                         min(n, k0 + a.suffix_chunk), a.prefix_parts + part);
}

// Joins the parts of one row-head; one warp each.
template <int D>
__global__ void __launch_bounds__(128) combine_kernel(const Args a) {
  const int64_t rh = (int64_t)a.T * a.q_heads;
  const int64_t i = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (i >= rh) return;
  const int lane = threadIdx.x & 31;
  const int t = (int)(i / a.q_heads), hq = (int)(i % a.q_heads);
  const int n = suffix_keys(a, t);
  // the row's prefix parts, then (from part prefix_parts on) its suffix parts
  const int pre = a.tc_ctas > 0 ? tc_parts(a, t * a.group + hq % a.group, hq / a.group) : a.prefix_parts;
  const int parts = pre + (n + a.suffix_chunk - 1) / a.suffix_chunk;
  const int skip = a.prefix_parts - pre;
  auto slot = [&](int p) { return (int64_t)(p < pre ? p : p + skip) * rh + i; };
  float m = -INFINITY;
  for (int p = lane; p < parts; p += 32) m = fmaxf(m, a.ml_part[slot(p)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d) acc[d] = 0.f;
  for (int p = 0; p < parts; ++p) {
    const int64_t at = slot(p);
    const float2 ml = a.ml_part[at];
    const float f = ex2(ml.x - base);
    l = fmaf(ml.y, f, l);
#pragma unroll
    for (int d = 0; d < D / 32; ++d) acc[d] = fmaf(a.o_part[at * D + d * 32 + lane], f, acc[d]);
  }
  const float inv = parts == 0 ? 0.f : 1.f / l;
#pragma unroll
  for (int d = 0; d < D / 32; ++d) a.out[i * D + d * 32 + lane] = __float2bfloat16(acc[d] * inv);
  if (a.lse != nullptr && lane == 0) a.lse[i] = parts == 0 ? -INFINITY : m * kLn2 + logf(l);
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

// Parts of the prefix and the suffix: enough CTAs for every SM to hold a few, no part
// shorter than 128 keys.
void plan_parts(Args* a, int wm, int sms) {
  const int want = sms * 3;
  auto split = [&](int keys, int64_t others, int* parts, int* chunk) {
    *parts = 0;
    *chunk = kTile;
    if (keys == 0) return;
    int64_t n = (want + others - 1) / others;
    n = std::max<int64_t>(1, std::min<int64_t>(n, (keys + 127) / 128));
    int64_t c = (keys + n - 1) / n;
    c = std::min<int64_t>(kMaxChunk, (c + kTile - 1) / kTile * kTile);
    *chunk = (int)c;
    *parts = (int)((keys + c - 1) / c);
  };
  a->tc_ctas = 0;
  if (a->prefix_len > 0 && a->T * a->group > 16 * wm) {
    plan_prefix_tc(a, sms);
  } else {
    a->row_tiles = (a->T * a->group + 16 * wm - 1) / (16 * wm);
    split(a->prefix_len, (int64_t)a->row_tiles * a->kv.kv_heads, &a->prefix_parts, &a->prefix_chunk);
  }
  split(a->max_suffix, (int64_t)a->T * a->kv.kv_heads, &a->suffix_parts, &a->suffix_chunk);
}

size_t scratch_layout(const Args& a, size_t* ml_at) {
  const size_t n = (size_t)(a.prefix_parts + a.suffix_parts) * a.T * a.q_heads;
  *ml_at = n * a.kv.head_dim * 4;
  return *ml_at + n * 8;
}

int wm_of(int group) { return group <= 16 ? 1 : group <= 32 ? 2 : 4; }

template <int D, bool F8, int WM>
int launch_stream(const Args& a, cudaStream_t s) {
  const int smem = StreamCfg<D, F8>::kSmem;
  static SmemLimit limit;
  const int r = limit.set(reinterpret_cast<const void*>(stream_kernel<D, F8, WM>), smem, "moe_prefix_attention");
  if (r != PMOE_OK) return r;
  const int64_t pb = a.tc_ctas > 0 ? 0 : (int64_t)a.prefix_parts * a.kv.kv_heads * a.row_tiles;
  const int64_t sb = (int64_t)a.suffix_parts * a.kv.kv_heads * a.T;
  if (pb + sb > INT32_MAX) return PMOE_EUNSUPPORTED;
  if (pb + sb > 0) stream_kernel<D, F8, WM><<<(unsigned)(pb + sb), kThreads, smem, s>>>(a, (int)pb);
  return launch_status("moe_prefix_attention");
}

template <int D, bool F8>
int launch_all(const Args& a, cudaStream_t s) {
  const int wm = wm_of(a.group);
  int r = a.tc_ctas > 0 ? launch_prefix_tc(a, s) : PMOE_OK;
  if (r != PMOE_OK) return r;
  r = wm == 1 ? launch_stream<D, F8, 1>(a, s) : wm == 2 ? launch_stream<D, F8, 2>(a, s) : launch_stream<D, F8, 4>(a, s);
  if (r != PMOE_OK) return r;
  const int64_t rh = (int64_t)a.T * a.q_heads;
  combine_kernel<D><<<(unsigned)((rh + 3) / 4), 128, 0, s>>>(a);
  return launch_status("moe_prefix_attention");
}

// Checks shared by the call and its scratch size; fills the part plan.
int plan(const pmoe_kv_desc* kv, int T, int q_heads, int prefix_len, int max_suffix, Args* a) {
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
  a->group_magic = (uint32_t)((1ull << 32) / a->group + 1);  // of no use for 1
  a->prefix_len = prefix_len;
  a->max_suffix = max_suffix;
  if (a->group > kMaxGroup) return PMOE_EUNSUPPORTED;
  if (T == 0) return PMOE_OK;
  const int sms = sm_count();
  if (sms == 0) return PMOE_ECUDA;
  plan_parts(a, wm_of(a->group), sms);
  return PMOE_OK;
}

}  // namespace
}  // namespace attn
}  // namespace pmoe

using namespace pmoe;

extern "C" size_t moe_prefix_attention_scratch_bytes(const pmoe_kv_desc* kv, int T, int q_heads, int prefix_len,
                                                     int max_suffix) {
  attn::Args a{};
  size_t ml = 0;
  if (attn::plan(kv, T, q_heads, prefix_len, max_suffix, &a) != PMOE_OK || T == 0) return 0;
  return attn::scratch_layout(a, &ml);
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
  int r = attn::plan(kv, T, q_heads, prefix_len, max_suffix, &a);
  if (r != PMOE_OK || T == 0) return r;
  size_t ml = 0;
  const size_t need = attn::scratch_layout(a, &ml);
  if (need > 0 && (scratch == nullptr || scratch_bytes < need)) return PMOE_EINVAL;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.scale = scale != 0.f ? scale * attn::kLog2e : 1e-30f;  // not 0: masked scores are -inf times it
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
  a.ml_part = reinterpret_cast<float2*>(static_cast<uint8_t*>(scratch) + ml);
  cudaStream_t s = (cudaStream_t)stream;
  const bool f8 = kv->dtype == PMOE_KV_E4M3;
  if (kv->head_dim == 128) return f8 ? attn::launch_all<128, true>(a, s) : attn::launch_all<128, false>(a, s);
  return f8 ? attn::launch_all<64, true>(a, s) : attn::launch_all<64, false>(a, s);
}
