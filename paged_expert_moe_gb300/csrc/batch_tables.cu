// moe_batch_tables: the pages, slots and positions of a step's tokens from the requests' lengths.
//
// Three running sums over the requests say everything: of their new tokens (where a request's rows
// lie), of the pages that ended requests give back (where those go on the stack of free pages), of
// the pages that the others need (which ones they get). From there each token works its own
// numbers out.
//
// Bound: latency, one launch. Every CTA of one cluster adds the sums up for itself (a request is 8
// bytes) and keeps what tokens look up in shared memory; the cluster's barrier stands between the
// ended requests' pages arriving on the stack and the new pages leaving it, and between the last
// read of the lengths and their update in place. Tokens are then spread over the cluster's threads.
// 256 requests of a token each take 6.5 us, 1,000 with 32,768 rows 11 us: three block-wide sums, two
// cluster barriers and two rounds of loads. Four tokens of a thread at a time, so that their searches
// overlap, cost the small call 0.6 us and gave the large one 0.3: not kept.
#include "pmoe_internal.h"

#include <cooperative_groups.h>

namespace pmoe {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaxRequests = 8192;

struct TableArgs {
  int32_t* page_table;
  int table_stride, page_size, num_pages;
  int32_t* free_pages;
  int free_capacity;
  const int32_t* free_count;
  int32_t* free_count_out;
  const int32_t *lens, *new_len;
  int R, T;
  int32_t *lens_out, *q_start, *positions, *slots, *row_seq, *row_len;
  int32_t* err;
};

// The sum over the threads before this one; *total: over all.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warps, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warps[warp] = x;
  __syncthreads();
  // every warp adds up the warps' sums for itself
  int64_t w = warps[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return (warp > 0 ? before : 0) + x - v;
}

__global__ void __launch_bounds__(kThreads) batch_tables_kernel(const TableArgs a) {
  extern __shared__ int32_t smem[];
  int32_t* start = smem;                 // [R + 1] first row
  int32_t* len = start + a.R + 1;        // [R] keys before the step
  int32_t* got = len + a.R;              // [R] new pages before its own; -1: the request gets none
  __shared__ int64_t warps[3][32];  // of three sums in turn, so that none waits for the one before to be read
  __shared__ int s_taken;
  const int tid = threadIdx.x, ctas = gridDim.x, cta = blockIdx.x, all = kThreads * ctas, me = cta * kThreads + tid;
  const int psh = 31 - __clz(a.page_size), round = a.page_size - 1;
  pdl_wait();
  pdl_trigger();
  if (tid == 0) s_taken = 0;
  const int64_t room = min((int64_t)a.table_stride << psh, (int64_t)INT32_MAX - 256);
  auto complain = [&](int32_t what) {
    if (a.err != nullptr && cta == 0) atomicOr(a.err, what);
  };
  int count = *a.free_count;
  if (count < 0 || count > a.free_capacity) {
    if (tid == 0) complain(kErrBadLength);
    count = count < 0 ? 0 : a.free_capacity;
  }

  // ---- where each request's rows lie; pages given back
  int64_t sum = 0, back = 0;
  for (int r0 = 0; r0 < a.R; r0 += kThreads) {
    const int r = r0 + tid;
    int have = 0, n = 0, old = 0;
    if (r < a.R) {
      old = a.lens[r], n = a.new_len[r];
      if (old < 0 || old > room || n < -1) {
        complain(kErrBadLength);
        old = old < 0 ? 0 : (int)min((int64_t)old, room);
      }
      have = (int)(((int64_t)old + round) >> psh);
    }
    const int ended = __syncthreads_or(n == -1);
    int64_t total;
    const int64_t at = sum + block_scan(max(n, 0), warps[0], &total);
    if (r < a.R) {
      start[r] = (int)min(at, (int64_t)a.T);
      // the row's end and the table's width decide first: what does not fit there takes no pages
      const bool fits = at + max(n, 0) <= a.T && (int64_t)old + max(n, 0) <= room;
      len[r] = old;
      got[r] = n > 0 && !fits ? -1 : 0;
      if (cta == 0) a.q_start[r] = start[r];
    }
    sum += total;
    if (ended) {
      const int64_t first = count + back + block_scan(n == -1 ? have : 0, warps[1], &total);
      back += total;
      // a warp hands back the pages of its lanes' requests, one request after another, each over
      // the whole cluster; eight loads of a lane are under way at a time
      const int lane = tid & 31, step = 32 * ctas;
      for (unsigned m = __ballot_sync(0xffffffffu, n == -1 && have > 0); m != 0; m &= m - 1) {
        const int k = __ffs(m) - 1, pages = __shfl_sync(0xffffffffu, have, k);
        const int64_t to = __shfl_sync(0xffffffffu, first, k);
        const int32_t* from = a.page_table + (int64_t)(r - lane + k) * a.table_stride;
        for (int i0 = cta * 32 + lane; i0 < pages; i0 += 8 * step) {
          int32_t page[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) page[u] = i0 + u * step < pages ? __ldcg(from + i0 + u * step) : 0;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * step;
            if (i >= pages) break;
            if (to + i < a.free_capacity)
              a.free_pages[to + i] = page[u];
            else if (a.err != nullptr)
              atomicOr(a.err, kErrBadLength);
          }
        }
      }
      __syncthreads();
    }
  }
  const int rows = (int)min(sum, (int64_t)a.T);
  if (tid == 0) {
    start[a.R] = rows;
    if (cta == 0) a.q_start[a.R] = rows;
  }
  const int64_t stack = min(count + back, (int64_t)a.free_capacity);
  cooperative_groups::this_cluster().sync();

  // ---- new pages, in order, off the top of the stack
  int64_t need_before = 0;
  for (int r0 = 0; r0 < a.R; r0 += kThreads) {
    const int r = r0 + tid;
    int old = 0, n = 0, have = 0;
    int64_t mine = 0;
    bool denied = false;
    if (r < a.R) {
      old = len[r], n = a.new_len[r];
      have = (int)(((int64_t)old + round) >> psh);
      denied = got[r] < 0;
      if (n > 0 && !denied) mine = (((int64_t)old + n + round) >> psh) - have;
    }
    int64_t total;
    const int64_t first = need_before + block_scan(mine, warps[2], &total);
    if (r < a.R) {
      if (mine > 0 && first + mine > stack) denied = true;
      if (denied) complain(kErrNoPages);
      got[r] = denied ? -1 : (int)min(first, stack);
      if (mine > 0 && !denied) atomicMax(&s_taken, (int)(first + mine));
    }
    need_before += total;
    if (r0 + kThreads < a.R) __syncthreads();
  }
  __syncthreads();
  if (me == 0) *a.free_count_out = (int)stack - s_taken;
  // (lens and lens_out may be the same, and new_len is read below no more than here: every CTA
  // has its own copies, and the cluster waits before the first write)
  cooperative_groups::this_cluster().sync();
  for (int r = me; r < a.R; r += all) {
    const int n = a.new_len[r];
    a.lens_out[r] = n == -1 ? 0 : got[r] >= 0 ? len[r] + max(n, 0) : len[r];
  }

  // ---- tokens; the first one of a page puts it into the table
  for (int t = me; t < a.T; t += all) {
    int pos = 0, slot = -1, seq = -1, seen = 0;
    if (t < rows) {
      int lo = 0, hi = a.R;  // start[lo] <= t < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t)
          lo = mid;
        else
          hi = mid;
      }
      seq = lo;
      const int old = len[seq];
      pos = old + (t - start[seq]);
      if (got[seq] >= 0) {
        const int page_of = pos >> psh, have = (int)(((int64_t)old + round) >> psh);
        int32_t* entry = a.page_table + (int64_t)seq * a.table_stride + page_of;
        int page;
        if (page_of < have) {
          page = *entry;
        } else {
          page = a.free_pages[stack - 1 - got[seq] - (page_of - have)];
          if ((pos & round) == 0) *entry = page;
        }
        seen = pos + 1;
        if ((unsigned)page < (unsigned)a.num_pages)
          slot = (page << psh) + (pos & round);
        else if (a.err != nullptr)
          atomicOr(a.err, kErrBadPage);
      }
    }
    a.positions[t] = pos;
    a.slots[t] = slot;
    a.row_seq[t] = seq;
    if (a.row_len != nullptr) a.row_len[t] = seen;
  }
}

}  // namespace
}  // namespace pmoe

using namespace pmoe;

extern "C" int moe_batch_tables(int32_t* page_table, int table_stride, int page_size, int num_pages, int32_t* free_pages,
                                int free_capacity, const int32_t* free_count, const int32_t* lens, const int32_t* new_len,
                                int R, int T, int32_t* lens_out, int32_t* free_count_out, int32_t* q_start,
                                int32_t* positions, int32_t* slots, int32_t* row_seq, int32_t* row_len, int32_t* err_out,
                                void* stream) {
  if (R < 0 || R > kMaxRequests || T < 0 || T > (1 << 24) || table_stride < 1 || num_pages < 1 || free_capacity < 0)
    return PMOE_EINVAL;
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0) return PMOE_EUNSUPPORTED;
  if ((int64_t)num_pages * page_size > INT32_MAX) return PMOE_EINVAL;
  if (free_count == nullptr || free_count_out == nullptr || q_start == nullptr || (free_pages == nullptr && free_capacity > 0) ||
      (R > 0 && (page_table == nullptr || lens == nullptr || new_len == nullptr || lens_out == nullptr)) ||
      (T > 0 && (positions == nullptr || slots == nullptr || row_seq == nullptr)))
    return PMOE_EINVAL;
  const void* all[] = {page_table, free_pages, free_count, lens, new_len, lens_out, free_count_out,
                       q_start,    positions,  slots,      row_seq, row_len, err_out};
  for (const void* p : all)
    if (reinterpret_cast<uintptr_t>(p) % 4 != 0) return PMOE_EINVAL;
  if (R > 0 && (new_len == lens_out || new_len == lens)) return PMOE_EINVAL;
  const TableArgs a{page_table, table_stride, page_size, num_pages, free_pages, free_capacity, free_count, free_count_out,
                    lens,       new_len,      R,         T,         lens_out,   q_start,       positions,  slots,
                    row_seq,    row_len,      err_out};
  const size_t smem = ((size_t)3 * R + 1) * 4;
  // a cluster of 8 for what a CTA's threads do not cover; fewer CTAs meet sooner
  const unsigned ctas = T <= 1024 ? 1 : T <= 2048 ? 2 : T <= 4096 ? 4 : 8;
  static SmemLimit limit;
  const int r = limit.set(reinterpret_cast<const void*>(batch_tables_kernel), (3 * kMaxRequests + 1) * 4, "moe_batch_tables");
  if (r != PMOE_OK) return r;
  return launch("moe_batch_tables", batch_tables_kernel, ctas, kThreads, smem, (cudaStream_t)stream, true, ctas, a);
}
