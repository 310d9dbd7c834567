// Tokens sorted by expert and back: the plan of a routing, the rows' gather
// and scatter, their weighted sum and its gradient.
//
// A pair p = t * top_k + j sends token t to one expert.  Pairs are sorted by
// expert, stable in p; row r of the sorted batch is pair row_pair[r], and
// pair_row is the inverse.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "kv4.cuh"
#include "route.cuh"

namespace lora {

// The wait for the call before, and leave for the next one's CTAs to come: in this
// order, so that what those do ahead of their own wait finds the calls before this
// one done.
__device__ __forceinline__ void after_previous_call() {
  cudaGridDependencySynchronize();
  cudaTriggerProgrammaticLaunchCompletion();
}

constexpr int kMoeMaxExperts = 1024;
constexpr int kMoeSortCluster = 16;
constexpr int kMoeThreads = 256;

// The expert of a pair on this rank, or E: none.
struct ExpertKey {
  const int32_t* topk_ids;
  const int32_t* expert_map;
  int n_global, E;
  __device__ int operator()(int p, uint32_t& err) const {
    int e = topk_ids[p];
    if (e == -1) return E;
    if (expert_map) {
      if (e < 0 || e >= n_global) {
        err |= LORA_DEV_ERR_EXPERT;
        return E;
      }
      e = expert_map[e];
      if (e < 0) return E;  // the expert lives on another rank
    }
    if (e < 0 || e >= E) {
      err |= LORA_DEV_ERR_EXPERT;
      return E;
    }
    return e;
  }
};

struct MoePlanArgs {
  ExpertKey key;
  const int32_t* lora_ids;
  int P, top_k;
  int32_t *seg_start, *row_pair, *pair_row, *row_expert, *row_lora;
  uint32_t* err;
};

// Pair p of an expert (E: none) at row `at`.
__device__ __forceinline__ void place_pair(const MoePlanArgs& a, int p, int key, int lora, int at) {
  const bool there = key < a.key.E;
  a.pair_row[p] = there ? at : -1;
  a.row_pair[at] = there ? p : -1;
  a.row_expert[at] = there ? key : -1;
  a.row_lora[at] = there ? lora : -1;
}

inline size_t moe_sort_smem(int E) { return sizeof(uint32_t) * ((size_t)kRouteWarps + 3) * (size_t)(E + 1); }

// One cluster; a contiguous block of pairs a CTA and within it a warp, counted
// per (warp, expert), the counts made positions over the cluster, then placed.
// Bound: a chain of some ten trips (loads, barriers, distributed shared memory); 32768
// pairs 13.6 us, 4104 pairs 10.
__global__ void __launch_bounds__(kRouteThreads) moe_sort_kernel(const MoePlanArgs a) {
  extern __shared__ uint32_t cnt[];  // [kRouteWarps][E + 1], then mine, before, total
  __shared__ uint32_t warp_sums[kRouteWarps];
  after_previous_call();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = a.key.E, nkb = E + 1, nblk = (int)gridDim.x, blk = (int)blockIdx.x;
  uint32_t *mine = cnt + kRouteWarps * nkb, *before = mine + nkb, *total = before + nkb;
  for (int i = tid; i < kRouteWarps * nkb; i += kRouteThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t parts = (int64_t)nblk * kRouteWarps, part = (int64_t)blk * kRouteWarps + warp;
  const int b0 = (int)(a.P * part / parts), b1 = (int)(a.P * (part + 1) / parts);
  uint32_t errbits = 0;
  uint32_t* my = cnt + warp * nkb;
  // The first 256 pairs' keys and adapters of a warp stay in registers for the
  // placing below (65536 pairs: all of them).
  int key[8], lora[8];
  auto load = [&](int base, uint32_t& err) {
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int p = base + u * 32 + lane;
      key[u] = p < b1 ? a.key(p, err) : -1;
      lora[u] = p < b1 && a.lora_ids ? a.lora_ids[p / a.top_k] : -1;
    }
  };
  load(b0, errbits);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const unsigned peers = __match_any_sync(0xffffffffu, key[u]);
    if (key[u] >= 0 && lane == __ffs(peers) - 1) my[key[u]] += __popc(peers);
    __syncwarp();
  }
  warp_count<4>(a.key, b0 + 256, b1, nkb, my, errbits);
  errbits = __reduce_or_sync(0xffffffffu, errbits);
  if (lane == 0 && errbits) set_error(a.err, errbits);
  __syncthreads();
  for (int k = tid; k < nkb; k += kRouteThreads) {
    uint32_t t = 0;
    for (int w = 0; w < kRouteWarps; ++w) t += cnt[w * nkb + k];
    mine[k] = t;
  }
  cluster_arrive_release_smem();
  cluster_wait();
  for (int k = tid; k < nkb; k += kRouteThreads) {
    uint32_t b = 0, t = 0;
#pragma unroll 8
    for (int c = 0; c < nblk; ++c) {
      const uint32_t v = __float_as_uint(dsmem_ld_f32(dsmem_map(smem_addr(mine) + 4u * (uint32_t)k, (uint32_t)c)));
      t += v;
      b += c < blk ? v : 0u;
    }
    before[k] = b;
    total[k] = t;
  }
  cluster_arrive_relaxed();  // done reading the peers (waited on before exit)
  __syncthreads();
  int k0, k1;
  uint32_t run = block_scan_keys(nkb, [&](int k) { return total[k]; }, k0, k1, warp_sums);
  for (int k = k0; k < k1; ++k) {
    if (blk == 0) a.seg_start[k] = (int32_t)run;
    uint32_t at = run + before[k];
    for (int w = 0; w < kRouteWarps; ++w) {
      const uint32_t c = cnt[w * nkb + k];
      cnt[w * nkb + k] = at;
      at += c;
    }
    run += total[k];
  }
  __syncthreads();
  for (int base = b0; base < b1; base += 256) {
    uint32_t dummy = 0;
    if (base > b0) load(base, dummy);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (base + u * 32 >= b1) break;
      const unsigned peers = __match_any_sync(0xffffffffu, key[u]);
      if (key[u] >= 0) place_pair(a, base + u * 32 + lane, key[u], lora[u], (int)my[key[u]] + __popc(peers & ((1u << lane) - 1u)));
      __syncwarp();
      if (key[u] >= 0 && lane == __ffs(peers) - 1) my[key[u]] += __popc(peers);
      __syncwarp();
    }
  }
  cluster_wait();  // the peers have read this CTA's totals
}

struct MoveArgs {
  void* out;  // dispatch: rows; combine: out; combine_grad: grad_rows
  int64_t ld_out;
  const void* x;  // dispatch: x; combine_grad: grad_out
  int64_t ld_x;
  const void* rows;
  int64_t ld_rows;
  const void* residual;
  int64_t ld_residual;
  const int32_t* pair_row;
  const float* weights;
  float* grad_weights;
  int T, top_k, H, P;
};

// The row of a pair, or -1.
__device__ __forceinline__ int row_of(const MoveArgs& a, int64_t p) {
  const int r = a.pair_row[p];
  return (unsigned)r < (unsigned)a.P ? r : -1;
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpack2<BF16>(w[i]);
    f[2 * i] = x.x;
    f[2 * i + 1] = x.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]), pack2<BF16>(f[6], f[7]));
}
__device__ __forceinline__ uint4 load8(const void* base, int64_t ld, int64_t row, int col) {
  return *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + row * ld + col);
}
__device__ __forceinline__ void store8(void* base, int64_t ld, int64_t row, int col, const uint4& v) {
  *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + row * ld + col) = v;
}

// A token's row into its pairs' rows.
__device__ __forceinline__ void scatter_row(const MoveArgs& a, int t, const int* row) {
  for (int c = threadIdx.x * 8; c < a.H; c += kMoeThreads * 8) {
    const uint4 v = load8(a.x, a.ld_x, t, c);
#pragma unroll 4
    for (int j = 0; j < a.top_k; ++j)
      if (row[j] >= 0) store8(a.out, a.ld_out, row[j], c, v);
  }
}

// rows[pair_row[t, j]] = x[t].  A CTA a token: x is read once, each row written once.
// Bound: the rows' bytes (8192 tokens of 4096 into 65536 rows 95 us, 6.4 TB/s, behind
// the sort; stores marked as streaming, two vectors a thread or x brought to L2 while the
// sort runs change nothing).
__global__ void __launch_bounds__(kMoeThreads) moe_scatter_kernel(const MoveArgs a) {
  __shared__ int row[LORA_MOE_MAX_TOP_K];
  const int t = blockIdx.x;
  after_previous_call();
  if ((int)threadIdx.x < a.top_k) row[threadIdx.x] = row_of(a, (int64_t)t * a.top_k + threadIdx.x);
  __syncthreads();
  scatter_row(a, t, row);
}

// Sort and scatter of few pairs in one launch: every token's CTA counts, among all
// pairs' keys, those that come before each of its own.  Bound: latency; 64 tokens of 8
// experts, rows of 2048, 3.0 us where two launches take 6.2, 512 tokens 12.6 and 14.5.
constexpr int kMoeFewPairs = 4096;
__global__ void __launch_bounds__(kMoeThreads) moe_dispatch_few_kernel(const MoePlanArgs a, const MoveArgs m) {
  extern __shared__ uint32_t few_s[];  // hist[E + 1] (of CTA 0), then the pairs' keys
  __shared__ int row[LORA_MOE_MAX_TOP_K];
  __shared__ uint32_t warp_sums[kMoeThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, t = blockIdx.x;
  const int E = a.key.E, nkb = E + 1;
  uint32_t* hist = few_s;
  uint16_t* key = reinterpret_cast<uint16_t*>(few_s + nkb);
  after_previous_call();
  uint32_t bad = 0;
  if (t == 0)
    for (int k = tid; k < nkb; k += kMoeThreads) hist[k] = 0;
#pragma unroll 4
  for (int p = tid; p < a.P; p += kMoeThreads) key[p] = (uint16_t)a.key(p, bad);
  if (bad && t == 0) set_error(a.err, bad);
  __syncthreads();
  for (int j = warp; j < a.top_k; j += kMoeThreads / 32) {
    const int p = t * a.top_k + j, e = key[p];
    int before = 0;
    for (int q = lane; q < a.P; q += 32) {
      const int k = key[q];
      before += k < e || (k == e && q < p);
    }
    before = __reduce_add_sync(0xffffffffu, before);
    if (lane == 0) {
      place_pair(a, p, e, a.lora_ids ? a.lora_ids[t] : -1, before);
      row[j] = e < E ? before : -1;
    }
  }
  __syncthreads();
  scatter_row(m, t, row);
  if (t == 0) {  // the experts' first rows
    for (int p = tid; p < a.P; p += kMoeThreads) atomicAdd(&hist[key[p]], 1u);
    __syncthreads();
    uint32_t carry = 0;
    for (int k0 = 0; k0 < nkb; k0 += kMoeThreads) {
      const uint32_t v = k0 + tid < nkb ? hist[k0 + tid] : 0u;
      uint32_t inc = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += u;
      }
      if (lane == 31) warp_sums[warp] = inc;
      __syncthreads();
      uint32_t base = carry;
      for (int w = 0; w < kMoeThreads / 32; ++w) {
        base += w < warp ? warp_sums[w] : 0u;
        carry += warp_sums[w];
      }
      if (k0 + tid < nkb) a.seg_start[k0 + tid] = (int32_t)(base + inc - v);
      __syncthreads();
    }
  }
}

// out[t] = residual[t] + sum_j w[t, j] rows[pair_row[t, j]], in the order of j, 8 rows
// on their way at once.  A CTA a token.  Bound: the rows' bytes (65536 rows of 4096
// into 8192: 86.5 us, 7.0 TB/s, some of it from L2; one row after another 97), for few
// tokens latency (64: 2.4 us).
template <bool BF16>
__global__ void __launch_bounds__(kMoeThreads) moe_combine_kernel(const MoveArgs a) {
  __shared__ int row[LORA_MOE_MAX_TOP_K];
  __shared__ float weight[LORA_MOE_MAX_TOP_K];
  after_previous_call();
  const int t = blockIdx.x;
  if ((int)threadIdx.x < a.top_k) {
    const int64_t p = (int64_t)t * a.top_k + threadIdx.x;
    row[threadIdx.x] = row_of(a, p);
    weight[threadIdx.x] = a.weights ? a.weights[p] : 1.0f;
  }
  __syncthreads();
  for (int c = threadIdx.x * 8; c < a.H; c += kMoeThreads * 8) {
    float sum[8] = {};
    uint4 res = make_uint4(0, 0, 0, 0);
    if (a.residual) res = load8(a.residual, a.ld_residual, t, c);
    for (int j0 = 0; j0 < a.top_k; j0 += 8) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u < a.top_k && row[j0 + u] >= 0) v[u] = load8(a.rows, a.ld_rows, row[j0 + u], c);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (j0 + u < a.top_k && row[j0 + u] >= 0) {
          float y[8];
          unpack8<BF16>(v[u], y);
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[i] = fmaf(weight[j0 + u], y[i], sum[i]);
        }
    }
    if (a.residual) {
      float y[8];
      unpack8<BF16>(res, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += y[i];
    }
    store8(a.out, a.ld_out, t, c, pack8<BF16>(sum));
  }
}

// grad_rows[pair_row[t, j]] = w[t, j] grad_out[t]; grad_weights[t, j] = grad_out[t] .
// rows[pair_row[t, j]].  A CTA a token; 4 pairs at a time, so that grad_out is read
// from L1 after the first and their rows are on their way together; dots are summed
// in a fixed order (a thread's columns, a warp's lanes, the warps).  Bound: the rows'
// bytes, once in and once out (65536 rows of 2048: 84.7 us, 6.7 TB/s; one pair after
// another 96).
constexpr int kGradPairs = 4;
template <bool BF16>
__global__ void __launch_bounds__(kMoeThreads) moe_combine_grad_kernel(const MoveArgs a) {
  __shared__ float part[kMoeThreads / 32][kGradPairs];
  __shared__ int row[LORA_MOE_MAX_TOP_K];
  __shared__ float weight[LORA_MOE_MAX_TOP_K];
  after_previous_call();
  const int t = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if ((int)threadIdx.x < a.top_k) {
    const int64_t p = (int64_t)t * a.top_k + threadIdx.x;
    row[threadIdx.x] = row_of(a, p);
    weight[threadIdx.x] = a.weights ? a.weights[p] : 1.0f;
  }
  __syncthreads();
  for (int j0 = 0; j0 < a.top_k; j0 += kGradPairs) {
    float dot[kGradPairs] = {};
    for (int c = threadIdx.x * 8; c < a.H; c += kMoeThreads * 8) {
      uint4 v[kGradPairs];
#pragma unroll
      for (int u = 0; u < kGradPairs; ++u)
        if (j0 + u < a.top_k && row[j0 + u] >= 0 && a.grad_weights) v[u] = load8(a.rows, a.ld_rows, row[j0 + u], c);
      float g[8];
      unpack8<BF16>(load8(a.x, a.ld_x, t, c), g);
#pragma unroll
      for (int u = 0; u < kGradPairs; ++u)
        if (j0 + u < a.top_k && row[j0 + u] >= 0) {
          float y[8];
          if (a.grad_weights) {
            unpack8<BF16>(v[u], y);
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[u] = fmaf(g[i], y[i], dot[u]);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = g[i] * weight[j0 + u];
          store8(a.out, a.ld_out, row[j0 + u], c, pack8<BF16>(y));
        }
    }
    if (!a.grad_weights) continue;
#pragma unroll
    for (int u = 0; u < kGradPairs; ++u) {
#pragma unroll
      for (int d = 16; d; d >>= 1) dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], d);
      if (lane == 0) part[warp][u] = dot[u];
    }
    __syncthreads();
    if ((int)threadIdx.x < kGradPairs && j0 + (int)threadIdx.x < a.top_k) {
      const int j = j0 + threadIdx.x;
      float sum = 0.0f;
      for (int w = 0; w < kMoeThreads / 32; ++w) sum += part[w][threadIdx.x];
      a.grad_weights[(int64_t)t * a.top_k + j] = row[j] >= 0 ? sum : 0.0f;
    }
    __syncthreads();
  }
}

}  // namespace lora
