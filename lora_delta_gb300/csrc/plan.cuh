// Batch plan of a serving step, built on the GPU from the requests' lengths:
// row starts, each row's request, position, cache slot and adapter slot, and
// the pages that the step's new tokens need.
#pragma once

#include "common.cuh"

namespace lora {

constexpr int kPlanMaxReqs = 4096;
constexpr int kPlanThreads = 512;
constexpr int kPlanRowsPerThread = 4;
constexpr int kPlanMaxCluster = 8;

struct PlanArgs {
  const int32_t* ctx_len;
  const int32_t* new_len;
  const int32_t* req_slot;  // NULL: every row's adapter slot is -1
  int B, n, page_size, max_pages;
  int32_t* table;
  int64_t ld_table;
  const int32_t* free_pages;  // NULL: the tables hold every page already
  int free_cap;               // entries of free_pages
  const int32_t* free_count;
  int32_t* free_left;
  int32_t* row_start;
  int32_t* seq_len;
  int32_t* row_req;
  int32_t* position;
  int64_t* slot_map;
  int32_t* seq_slot;
  uint32_t* err;
};

inline size_t plan_smem_bytes(int B) { return (size_t)(3 * B + 1) * sizeof(int32_t); }

// Exclusive sums over a block of kPlanThreads threads of a 64-bit and a 32-bit
// value; the block's totals are returned in tot_a / tot_b.  `buf` holds one
// slot a warp.
__device__ __forceinline__ void block_scan2(int64_t a, int b, int64_t& ex_a, int& ex_b,
                                            int64_t& tot_a, int& tot_b, int64_t* buf_a,
                                            int* buf_b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t sa = a;
  int sb = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t ua = __shfl_up_sync(0xffffffffu, sa, d);
    const int ub = __shfl_up_sync(0xffffffffu, sb, d);
    if (lane >= d) {
      sa += ua;
      sb += ub;
    }
  }
  __syncthreads();  // (the buffers may still be read from an earlier call)
  if (lane == 31) {
    buf_a[warp] = sa;
    buf_b[warp] = sb;
  }
  __syncthreads();
  int64_t base_a = 0;
  int base_b = 0;
  tot_a = 0;
  tot_b = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    const int64_t va = buf_a[w];
    const int vb = buf_b[w];
    if (w < warp) {
      base_a += va;
      base_b += vb;
    }
    tot_a += va;
    tot_b += vb;
  }
  ex_a = base_a + sa - a;
  ex_b = base_b + sb - b;
}

// Every CTA scans all requests (12 bytes each, in L2 after the first), so no CTA
// waits for another's sums; the rows are then shared out in contiguous chunks
// and each row finds its request by binary search in shared memory.  Table
// entries below ceil(ctx / P) are only read and the others only written.  What is
// replaced in place (free_left that is free_count, seq_len that is ctx_len) is
// stored behind a barrier of one thread-block cluster (`cluster`), after every CTA
// has read it; else there are CTAs for all rows.
// Bound: latency (20 bytes a row; three dependent round trips to L2/HBM): 64
// single tokens 4.7 us, 512 requests with 75 thousand rows 5.9 us.
__global__ void __launch_bounds__(kPlanThreads) batch_plan_kernel(const PlanArgs a, int cluster) {
  extern __shared__ int32_t plan_smem[];
  int32_t* start_s = plan_smem;           // [B + 1] first row, clipped to n
  int32_t* ctx_s = plan_smem + a.B + 1;   // [B]
  int32_t* first_s = ctx_s + a.B;         // [B] number of the request's first new page
  __shared__ int64_t buf_a[kPlanThreads / 32];
  __shared__ int buf_b[kPlanThreads / 32];
  __shared__ int used_s;
  const int rank = blockIdx.x, n_ctas = gridDim.x, P = a.page_size;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (what the kernel before wrote is read from here on)
  const int64_t cap = (int64_t)a.max_pages * P;
  const int told = a.free_pages ? *a.free_count : 0;
  const int count = told < 0 ? 0 : (told < a.free_cap ? told : a.free_cap);
  if (threadIdx.x == 0) used_s = 0;
  uint32_t bad = a.free_pages && told != count ? LORA_DEV_ERR_PAGE : 0u;
  int64_t carry_rows = 0;
  int carry_pages = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    int64_t ctx = 0, add = 0;
    if (b < a.B) {
      ctx = a.ctx_len[b];
      add = a.new_len[b];
      if (ctx < 0 || add < 0 || ctx + add > cap) bad |= LORA_DEV_ERR_LENGTH;
      ctx = ctx < 0 ? 0 : (ctx > cap ? cap : ctx);
      add = add < 0 ? 0 : (ctx + add > cap ? cap - ctx : add);
    }
    const int held = (int)((ctx + P - 1) / P);
    const int need = (int)((ctx + add + P - 1) / P) - held;
    int64_t start, rows;
    int first, pages;
    block_scan2(add, need, start, first, rows, pages, buf_a, buf_b);
    start += carry_rows;
    first += carry_pages;
    if (b < a.B) {
      // rows past n are cut off; at most one request is cut in the middle,
      // and the requests after it have no rows
      const int64_t lo = start < a.n ? start : a.n;
      const int64_t hi = start + add < a.n ? start + add : a.n;
      if (hi - lo < add) bad |= LORA_DEV_ERR_LENGTH;
      const int64_t seq = ctx + (hi - lo);
      start_s[b] = (int32_t)lo;
      ctx_s[b] = (int32_t)ctx;
      first_s[b] = first;
      const int got = (int)((seq + P - 1) / P) - held;
      if (got > 0) atomicMax(&used_s, first + got);
      if (rank == 0) {
        a.row_start[b] = (int32_t)lo;
        if (!cluster) a.seq_len[b] = (int32_t)seq;  // (one CTA: by the thread that has read ctx_len[b])
      }
    }
    carry_rows += rows;
    carry_pages += pages;
  }
  const int total = (int)(carry_rows < a.n ? carry_rows : a.n);
  if (threadIdx.x == 0) {
    start_s[a.B] = total;
    if (rank == 0) a.row_start[a.B] = total;
  }
  __syncthreads();

  for (int64_t i0 = ((int64_t)rank * kPlanThreads + threadIdx.x) * kPlanRowsPerThread; i0 < a.n;
       i0 += (int64_t)n_ctas * kPlanThreads * kPlanRowsPerThread) {
    int b = 0;
    if (i0 < total) {  // the last request whose start is not past i0
      int lo = 0, hi = a.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start_s[mid] <= i0) lo = mid; else hi = mid;
      }
      b = lo;
    }
    int32_t req[kPlanRowsPerThread], pos[kPlanRowsPerThread], slot[kPlanRowsPerThread];
    int64_t map[kPlanRowsPerThread];
#pragma unroll
    for (int u = 0; u < kPlanRowsPerThread; ++u) {
      const int64_t i = i0 + u;
      req[u] = -1;
      pos[u] = 0;
      slot[u] = -1;
      map[u] = -1;
      if (i >= total) continue;
      while (start_s[b + 1] <= i) ++b;
      const int p = ctx_s[b] + (int)(i - start_s[b]);
      const int pg = p / P, held = (ctx_s[b] + P - 1) / P;
      int32_t* entry = a.table + (int64_t)b * a.ld_table + pg;
      int page;
      if (pg < held || !a.free_pages) {
        page = *entry;
      } else {
        const int at = count - 1 - (first_s[b] + pg - held);
        page = at >= 0 ? a.free_pages[at] : -1;
        if (p - pg * P == 0) *entry = page;  // the page's first token is a new row
      }
      if (page < 0) bad |= LORA_DEV_ERR_PAGE;
      req[u] = b;
      pos[u] = p;
      slot[u] = a.req_slot ? a.req_slot[b] : -1;
      map[u] = page < 0 ? -1 : (int64_t)page * P + (p - pg * P);
    }
    if (i0 + kPlanRowsPerThread <= a.n) {
      *reinterpret_cast<int4*>(a.row_req + i0) = make_int4(req[0], req[1], req[2], req[3]);
      *reinterpret_cast<int4*>(a.position + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      *reinterpret_cast<int4*>(a.seq_slot + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      longlong2* m = reinterpret_cast<longlong2*>(a.slot_map + i0);
      m[0] = make_longlong2(map[0], map[1]);
      m[1] = make_longlong2(map[2], map[3]);
    } else {
      for (int u = 0; i0 + u < a.n; ++u) {
        a.row_req[i0 + u] = req[u];
        a.position[i0 + u] = pos[u];
        a.seq_slot[i0 + u] = slot[u];
        a.slot_map[i0 + u] = map[u];
      }
    }
  }
  if (bad) set_error(a.err, bad);
  if (cluster) {
    cluster_arrive();
    cluster_wait();
  }
  if (cluster && rank == 0)
    for (int b = threadIdx.x; b < a.B; b += kPlanThreads) a.seq_len[b] = ctx_s[b] + start_s[b + 1] - start_s[b];
  if (a.free_pages && rank == 0 && threadIdx.x == 0) {
    const int left = count - used_s;
    *a.free_left = left > 0 ? left : 0;
  }
}

// Pages of finished requests back onto the free stack: the entries >= 0 of
// the first ceil(seq / P) pages of every request with done[b] != 0, in
// (request, page) order, from free_pages[*free_count] up; their entries (and
// the holes among them) become -1.  One CTA: a warp a request counts, the
// block sums, and a warp a request writes.
__global__ void __launch_bounds__(kPlanThreads)
    pages_release_kernel(const int32_t* __restrict__ done, const int32_t* __restrict__ seq_len,
                         int B, int page_size, int32_t* table, int64_t ld_table, int max_pages,
                         int32_t* free_pages, int free_cap, int32_t* free_count, uint32_t* err) {
  __shared__ int base_s[kPlanMaxReqs];
  __shared__ int64_t buf_a[kPlanThreads / 32];
  __shared__ int buf_b[kPlanThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int count = *free_count;
  uint32_t bad = count < 0 ? LORA_DEV_ERR_PAGE : 0u;
  auto pages_of = [&](int b) -> int {
    if (done[b] == 0) return 0;
    const int64_t seq = seq_len[b], p = seq < 0 ? 0 : (seq + page_size - 1) / page_size;
    if (seq < 0 || p > max_pages) bad |= LORA_DEV_ERR_LENGTH;
    return (int)(p > max_pages ? max_pages : p);
  };
  for (int b = warp; b < B; b += kPlanThreads / 32) {
    const int np = pages_of(b);
    int c = 0;
    for (int p = lane; p < np; p += 32) c += table[(int64_t)b * ld_table + p] >= 0;
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) base_s[b] = c;
  }
  __syncthreads();
  int carry = count < 0 ? 0 : count;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + threadIdx.x;
    const int c = b < B ? base_s[b] : 0;
    int64_t ea, ta;
    int eb, tb;
    block_scan2(0, c, ea, eb, ta, tb, buf_a, buf_b);
    if (b < B) base_s[b] = carry + eb;
    carry += tb;
  }
  __syncthreads();
  for (int b = warp; b < B; b += kPlanThreads / 32) {
    const int np = pages_of(b);
    int at = base_s[b];
    for (int p0 = 0; p0 < np; p0 += 32) {
      int32_t* entry = table + (int64_t)b * ld_table + p0 + lane;
      const int page = p0 + lane < np ? *entry : -1;
      const uint32_t held = __ballot_sync(0xffffffffu, page >= 0);
      const int to = at + __popc(held & ((1u << lane) - 1u));
      if (page >= 0) {
        if (to < free_cap) {
          free_pages[to] = page;
          *entry = -1;
        } else {
          bad |= LORA_DEV_ERR_PAGE;  // no room: the entry stays
        }
      }
      at += __popc(held);
    }
  }
  if (bad) set_error(err, bad);
  __syncthreads();
  if (threadIdx.x == 0) *free_count = carry < free_cap ? carry : free_cap;
}

}  // namespace lora
