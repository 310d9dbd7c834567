// Tokens sorted by expert and back: the plan of a routing, the rows' gather
// and scatter, their weighted sum and its gradient.
//
// A pair p = t * top_k + j sends token t to one expert.  Pairs are sorted by
// expert, stable in p; row r of the sorted batch is pair row_pair[r], and
// pair_row is the inverse.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "route.cuh"

namespace lora {

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

inline size_t moe_sort_smem(int E) { return sizeof(uint32_t) * ((size_t)kRouteWarps + 3) * (size_t)(E + 1); }

// One cluster; a contiguous block of pairs a CTA and within it a warp, counted
// per (warp, expert), the counts made positions over the cluster, then placed.
__global__ void __launch_bounds__(kRouteThreads) moe_sort_kernel(const MoePlanArgs a) {
  extern __shared__ uint32_t cnt[];  // [kRouteWarps][E + 1], then mine, before, total
  __shared__ uint32_t warp_sums[kRouteWarps];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int E = a.key.E, nkb = E + 1, nblk = (int)gridDim.x, blk = (int)blockIdx.x;
  uint32_t *mine = cnt + kRouteWarps * nkb, *before = mine + nkb, *total = before + nkb;
  for (int i = tid; i < kRouteWarps * nkb; i += kRouteThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t parts = (int64_t)nblk * kRouteWarps, part = (int64_t)blk * kRouteWarps + warp;
  const int b0 = (int)(a.P * part / parts), b1 = (int)(a.P * (part + 1) / parts);
  uint32_t errbits = 0;
  uint32_t* my = cnt + warp * nkb;
  warp_count<4>(a.key, b0, b1, nkb, my, errbits);
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
  for (int base = b0; base < b1; base += 32) {
    const int p = base + lane;
    uint32_t dummy = 0;
    const int key = p < b1 ? a.key(p, dummy) : -1;
    const unsigned peers = __match_any_sync(0xffffffffu, key);
    if (key >= 0) {
      const uint32_t at = my[key] + __popc(peers & ((1u << lane) - 1u));
      const bool there = key < E;
      a.pair_row[p] = there ? (int32_t)at : -1;
      a.row_pair[at] = there ? p : -1;
      a.row_expert[at] = there ? key : -1;
      a.row_lora[at] = there && a.lora_ids ? a.lora_ids[p / a.top_k] : -1;
    }
    __syncwarp();
    if (key >= 0 && lane == __ffs(peers) - 1) my[key] += __popc(peers);
    __syncwarp();
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
    if (BF16) {
      f[2 * i] = bf16lo(w[i]);
      f[2 * i + 1] = bf16hi(w[i]);
    } else {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (BF16) {
      w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
    } else {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 load8(const void* base, int64_t ld, int64_t row, int col) {
  return *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(base) + row * ld + col);
}
__device__ __forceinline__ void store8(void* base, int64_t ld, int64_t row, int col, const uint4& v) {
  *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + row * ld + col) = v;
}

// rows[pair_row[t, j]] = x[t]
__global__ void __launch_bounds__(kMoeThreads) moe_scatter_kernel(const MoveArgs a) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int t = blockIdx.x;
  for (int c = threadIdx.x * 8; c < a.H; c += kMoeThreads * 8) {
    const uint4 v = load8(a.x, a.ld_x, t, c);
    for (int j = 0; j < a.top_k; ++j) {
      const int r = row_of(a, (int64_t)t * a.top_k + j);
      if (r >= 0) store8(a.out, a.ld_out, r, c, v);
    }
  }
}

// out[t] = residual[t] + sum_j w[t, j] rows[pair_row[t, j]], in the order of j
template <bool BF16>
__global__ void __launch_bounds__(kMoeThreads) moe_combine_kernel(const MoveArgs a) {
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int t = blockIdx.x;
  for (int c = threadIdx.x * 8; c < a.H; c += kMoeThreads * 8) {
    float sum[8] = {};
    for (int j = 0; j < a.top_k; ++j) {
      const int64_t p = (int64_t)t * a.top_k + j;
      const int r = row_of(a, p);
      if (r < 0) continue;
      const float w = a.weights ? a.weights[p] : 1.0f;
      float y[8];
      unpack8<BF16>(load8(a.rows, a.ld_rows, r, c), y);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = fmaf(w, y[i], sum[i]);
    }
    if (a.residual) {
      float y[8];
      unpack8<BF16>(load8(a.residual, a.ld_residual, t, c), y);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += y[i];
    }
    store8(a.out, a.ld_out, t, c, pack8<BF16>(sum));
  }
}

// grad_rows[pair_row[t, j]] = w[t, j] grad_out[t]; grad_weights[t, j] = grad_out[t] . rows[pair_row[t, j]]
template <bool BF16>
__global__ void __launch_bounds__(kMoeThreads) moe_combine_grad_kernel(const MoveArgs a) {
  __shared__ float part[kMoeThreads / 32];
  cudaTriggerProgrammaticLaunchCompletion();
  cudaGridDependencySynchronize();
  const int t = blockIdx.x;
  for (int j = 0; j < a.top_k; ++j) {
    const int64_t p = (int64_t)t * a.top_k + j;
    const int r = row_of(a, p);
    const float w = a.weights ? a.weights[p] : 1.0f;
    float dot = 0.0f;
    if (r >= 0)
      for (int c = threadIdx.x * 8; c < a.H; c += kMoeThreads * 8) {
        float g[8], y[8];
        unpack8<BF16>(load8(a.x, a.ld_x, t, c), g);
        unpack8<BF16>(load8(a.rows, a.ld_rows, r, c), y);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(g[i], y[i], dot);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= w;
        store8(a.out, a.ld_out, r, c, pack8<BF16>(g));
      }
#pragma unroll
    for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0 && a.grad_weights) {
      float sum = 0.0f;
      for (int i = 0; i < kMoeThreads / 32; ++i) sum += part[i];
      a.grad_weights[p] = r >= 0 ? sum : 0.0f;
    }
    __syncthreads();
  }
}

}  // namespace lora
