// Matrix product with bias, delta, activation and residual: for the rows r of
// a group (one, or the experts' segments of sorted rows)
//   z = x[r] W^T + bias + delta[r]
//   out[r] = act(z) + residual[r], or act(z[0:I]) * z[I:2I] + residual[r]
// summed in float32 and rounded once.
#pragma once

#include "common.cuh"
#include "moe.cuh"

namespace lora {

struct LinearArgs {
  void* out;
  int64_t ld_out;
  const void* x;
  int64_t ld_x;
  const void* w;
  int64_t ld_w, stride_w;  // of a row, of a group
  const void* bias;        // [groups, N]
  const void* delta;
  int64_t ld_delta;
  const void* residual;
  int64_t ld_residual;
  const int32_t* seg_start;  // [groups + 1], or null: one group of all rows
  int groups, n, K, N, n_out;  // N rows of a group's W; n_out columns of out
  int act, gated;
  uint32_t* err;
  uint64_t wait_ns;
};

// Rows [start, end) of a group.
__device__ __forceinline__ int2 group_rows(const LinearArgs& a, int g, uint32_t& bad) {
  if (!a.seg_start) return make_int2(0, a.n);
  const int s = a.seg_start[g], e = a.seg_start[g + 1];
  if (s < 0 || e < s || e > a.n) bad |= LORA_DEV_ERR_SEGMENT;
  const int s1 = min(max(s, 0), a.n);
  return make_int2(s1, min(max(e, s1), a.n));
}

__device__ __forceinline__ float activate(float z, int act) {
  switch (act) {
    case LORA_ACT_RELU: return z > 0.0f ? z : (z != z ? z : 0.0f);
    case LORA_ACT_SILU: return z / (1.0f + expf(-z));
    case LORA_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    case LORA_ACT_GELU_TANH: return 0.5f * z * (1.0f + tanhf(0.79788456f * (z + 0.044715f * z * z * z)));
    default: return z;
  }
}

template <bool BF16>
__device__ __forceinline__ float elem(const void* base, int64_t i) {
  return BF16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[i])
              : __half2float(reinterpret_cast<const __half*>(base)[i]);
}

// A tile of 64 rows x 64 columns a CTA, 4 x 4 a thread.
template <bool BF16>
__global__ void __launch_bounds__(256) linear_simple_kernel(const LinearArgs a) {
  __shared__ float xs[16][65], ws[2][16][65];
  cudaGridDependencySynchronize();
  const int tid = threadIdx.x, tr = tid / 16, tc = tid % 16, c0 = blockIdx.x * 64, g = blockIdx.y;
  uint32_t bad = 0;
  const int2 seg = group_rows(a, g, bad);
  if (bad && tid == 0) set_error(a.err, bad);
  const int halves = a.gated ? 2 : 1;
  for (int r0 = seg.x + blockIdx.z * 64; r0 < seg.y; r0 += gridDim.z * 64) {
    float acc[2][4][4] = {};
    for (int k0 = 0; k0 < a.K; k0 += 16) {
      for (int i = tid; i < 16 * 64; i += 256) {
        const int r = i / 16, k = k0 + i % 16;
        xs[i % 16][r] = r0 + r < seg.y && k < a.K ? elem<BF16>(a.x, (int64_t)(r0 + r) * a.ld_x + k) : 0.0f;
        for (int h = 0; h < halves; ++h)
          ws[h][i % 16][r] = c0 + r < a.n_out && k < a.K
                                 ? elem<BF16>(a.w, (int64_t)g * a.stride_w + (int64_t)(h * a.n_out + c0 + r) * a.ld_w + k)
                                 : 0.0f;
      }
      __syncthreads();
      for (int k = 0; k < 16; ++k)
        for (int h = 0; h < halves; ++h)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[h][i][j] = fmaf(xs[k][tr * 4 + i], ws[h][k][tc + 16 * j], acc[h][i][j]);
      __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
      for (int j = 0; j < 4; ++j) {
        const int64_t r = r0 + tr * 4 + i;
        const int c = c0 + tc + 16 * j;
        if (r >= seg.y || c >= a.n_out) continue;
        float z[2];
        for (int h = 0; h < halves; ++h) {
          z[h] = acc[h][i][j];
          if (a.bias) z[h] += elem<BF16>(a.bias, (int64_t)g * a.N + h * a.n_out + c);
          if (a.delta) z[h] += elem<BF16>(a.delta, r * a.ld_delta + h * a.n_out + c);
        }
        float y = activate(z[0], a.act);
        if (a.gated) y *= z[1];
        if (a.residual) y += elem<BF16>(a.residual, r * a.ld_residual + c);
        if (BF16)
          reinterpret_cast<__nv_bfloat16*>(a.out)[r * a.ld_out + c] = __float2bfloat16_rn(y);
        else
          reinterpret_cast<__half*>(a.out)[r * a.ld_out + c] = __float2half_rn(y);
      }
  }
}

}  // namespace lora
