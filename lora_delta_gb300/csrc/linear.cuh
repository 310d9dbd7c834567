// Matrix product with bias, delta, activation and residual: for the rows r of
// a group (one, or the experts' segments of sorted rows)
//   z = x[r] W^T + bias + delta[r]
//   out[r] = act(z) + residual[r], or act(z[0:I]) * z[I:2I] + residual[r]
// summed in float32 and rounded once.
//
// W's rows are the M side of the tensor cores' products (128 a CTA) and x's rows
// the N side, whose size a product takes as it comes: a segment of 40 rows costs
// 48 columns, not a tile of 128.  Gated, a CTA's 128 rows are 64 of each half.
// The sums go through shared memory to the threads that finish 4 or 8 columns of
// a row of out, where delta and residual are read and out is written whole sectors
// at a time.  Two kernels: few rows a group stream W and are bound by its bytes, many
// rows by the tensor cores (64 FLOP and more a byte of W).
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "kv4_attn.cuh"
#include "moe.cuh"
#include "tc.cuh"

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
  uint32_t* counters;  // of shared tiles, zero between calls; or null: no tile is shared
  float* parts;
};

// Rows [start, end) of a group.
__device__ __forceinline__ int2 group_rows(const LinearArgs& a, int g, uint32_t& bad) {
  if (!a.seg_start) return make_int2(0, a.n);
  const int s = a.seg_start[g], e = a.seg_start[g + 1];
  if (s < 0 || e < s || e > a.n) bad |= LORA_DEV_ERR_SEGMENT;
  const int s1 = min(max(s, 0), a.n);
  return make_int2(s1, min(max(e, s1), a.n));
}

// 1 / x for x in [1, 8]: within 2^-23 of it.
__device__ __forceinline__ float rcp_near(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// gelu of a value: z / 2 erfc(-z / sqrt 2) = max(z, 0) - a G e^(-a^2 / 2) with a = |z| and
// G = erfcx(a / sqrt 2) / 2, so that nothing cancels in the lower tail, where z / 2 (1 + erf)
// keeps no digit from -5.5 on.  G is a polynomial in t = 1 / (1 + 0.3 a), fitted by weighted
// least squares to within 1.5e-7 of it from 0 to 14, where the result leaves float32.  The
// power is the square of that of half its exponent, so that its underflow is the result's.
// With CUDA's erfcf in its place 8192 rows of 4096 by 28672 took 1255 us for 1139 to 1181,
// gated 1155 for 1114.
__device__ __forceinline__ float gelu_erf(float z) {
  const float a = fminf(fabsf(z), 20.0f), t = rcp_near(fmaf(a, 0.3f, 1.0f));
  float g = 0.03567515f;
  g = fmaf(g, t, -0.15720464f);
  g = fmaf(g, t, 0.20635618f);
  g = fmaf(g, t, -0.053686097f);
  g = fmaf(g, t, 0.12856292f);
  g = fmaf(g, t, 0.099913100f);
  g = fmaf(g, t, 0.12075402f);
  g = fmaf(g, t, 0.11962929f);
  const float h = exp2_fast(a * a * -0.36067376f);  // e^(-a^2 / 4)
  return fmaf(-(a * (g * t) * h), h, z < 0.0f ? 0.0f * z : z);
}

// z / (1 + e^-t), where t has z's sign: silu (t = z) and gelu by tanh (t = 2 u).  With
// e = e^-|t| it is z / (1 + e) or z e / (1 + e), so that the divisor is 1 to 2 and, for far
// negative t, the value leaves float32 no earlier than it has to (z / (1 + e^-t) is 0 from
// -87.4 on, where bf16 holds it to -97).
__device__ __forceinline__ float times_sigmoid(float z, float t) {
  const float h = exp2_fast(fabsf(t) * -0.72134752f);  // e^(-|t| / 2)
  return (t < 0.0f ? z * h * h : z) * rcp_near(fmaf(h, h, 1.0f));
}

// Of N values.  (Few instructions matter more than the time they take: the roles of a
// CTA run at once and fetch theirs side by side.)
template <int N>
__device__ __forceinline__ void activate(float* z, int act) {
  if (act == LORA_ACT_NONE) return;
  if (act == LORA_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = z[i] < 0.0f ? 0.0f : z[i];
  } else if (act == LORA_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = gelu_erf(z[i]);
  } else {
    const float cubic = act == LORA_ACT_SILU ? 0.0f : 2.0f * 0.79788456f * 0.044715f;
    const float linear = act == LORA_ACT_SILU ? 1.0f : 2.0f * 0.79788456f;
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] = times_sigmoid(z[i], z[i] * (cubic == 0.0f ? linear : fmaf(cubic * z[i], z[i], linear)));
  }
}

// Tensor maps of x for boxes of 16, 32, 64 and 128 rows: one copy a step, of the
// least box that holds the rows.  (Copies of 32 rows took the place of one of 128 in
// 1440 us where this takes 1205, 8192 x 4096 by 28672: what bounds them is their number.)
struct RowMaps {
  CUtensorMap box[4];
};
__host__ __device__ __forceinline__ int row_box(int rows) { return rows <= 16 ? 0 : (rows <= 32 ? 1 : (rows <= 64 ? 2 : 3)); }

// -------------------------------------------------------------- epilogue --
// 8 (V: uint4) or 4 (uint2) columns of a row of out: what is read for them, ahead of
// the sums, and what becomes of the sums z (and up, the second half's).
template <class V>
struct LinearTail {
  V delta[2], residual;
};
template <class V>
struct LinearBias {
  V half[2];
};

template <class V>
__device__ __forceinline__ V load_v(const void* base, int64_t at) {
  return *reinterpret_cast<const V*>(reinterpret_cast<const uint16_t*>(base) + at);
}

template <bool GATED, class V>
__device__ __forceinline__ LinearBias<V> linear_bias(const LinearArgs& a, int g, int col) {
  LinearBias<V> b = {};
  if (a.bias && col < a.n_out) {
    b.half[0] = load_v<V>(a.bias, (int64_t)g * a.N + col);
    if (GATED) b.half[1] = load_v<V>(a.bias, (int64_t)g * a.N + a.n_out + col);
  }
  return b;
}

template <bool GATED, class V>
__device__ __forceinline__ LinearTail<V> linear_tail(const LinearArgs& a, int64_t row, int col, bool use) {
  LinearTail<V> t = {};
  if (use && a.delta) {
    t.delta[0] = load_v<V>(a.delta, row * a.ld_delta + col);
    if (GATED) t.delta[1] = load_v<V>(a.delta, row * a.ld_delta + a.n_out + col);
  }
  if (use && a.residual) t.residual = load_v<V>(a.residual, row * a.ld_residual + col);
  return t;
}

template <bool BF16, class V>
__device__ __forceinline__ void add_v(float* z, const V& v) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < (int)(sizeof(V) / 4); ++i) {
    const float2 f = unpack2<BF16>(w[i]);
    z[2 * i] += f.x;
    z[2 * i + 1] += f.y;
  }
}

// EXTRA: with a delta (1), a residual (2).
template <bool BF16, bool GATED, int EXTRA, class V>
__device__ __forceinline__ V linear_finish(const LinearArgs& a, const LinearBias<V>& b, const LinearTail<V>& t, float* z, float* up) {
  constexpr int N = sizeof(V) / 2;
  if (a.bias) add_v<BF16>(z, b.half[0]);
  if ((EXTRA & 1) && a.delta) add_v<BF16>(z, t.delta[0]);
  activate<N>(z, a.act);
  if (GATED) {
    if (a.bias) add_v<BF16>(up, b.half[1]);
    if ((EXTRA & 1) && a.delta) add_v<BF16>(up, t.delta[1]);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] *= up[i];
  }
  if ((EXTRA & 2) && a.residual) add_v<BF16>(z, t.residual);
  V y;
  uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = pack2<BF16>(z[2 * i], z[2 * i + 1]);
  return y;
}

// ------------------------------------------------------------- few rows --
// A tile is 128 rows of W and up to NT of x.  The CTAs of a cluster share a
// tile's K out, so that few tiles still read W at the card's full rate; their
// parts are added in the order of K through distributed shared memory, each CTA
// finishing its share of the tile.  Grid: (feature tile, part of K), group, and
// row tiles in turn.  Two CTAs fit an SM.
// Bound: W's bytes, and launch, first copies and the parts' way where they are few.  1 row
// of 4096 by 6144 12 us (4.2 TB/s), 64 rows 14.5, 128 rows 17.4; 64 tokens of 8 experts,
// 2048 by 1536 gated, 67 to 74 us (5.5 to 6.1 TB/s).  Parts read 32 bytes a thread instead of 16, so
// that a warp's lie apart: 64 rows 16.3, 128 rows 21.0 (from the CTA's own memory 13.0).
// Tiles of 256 rows of x in this form lost to the pairs below, as the parts' way grows
// with the rows (192 rows of 2048 by 2048 26 us, 17 there).
template <int NT_>
struct Few {
  static constexpr int NT = NT_;
  static constexpr int W = 128 * 128, X = NT * 128, STAGE = W + X;
  static constexpr int STAGES = 106 * 1024 / STAGE;
  static constexpr int PAD = 132;  // floats between rows of a part
  static constexpr int THREADS = 256;  // load, MMA, 4 warps that read the sums; all finish
  static constexpr uint32_t COLS = NT < 32 ? 32 : NT;  // of tensor memory
  static constexpr size_t smem() { return 1024 + (size_t)STAGES * STAGE; }
  static_assert(NT * PAD * 4 <= STAGES * STAGE, "a part lies where the operands were");
};

// A CTA's share of a tile, from all parts: 4 columns of out a thread, so that a warp
// reads a part's 512 bytes in a row.  What is read from global memory for the first of
// them is on its way while the parts are awaited.
template <bool BF16, bool GATED, class C>
__device__ __forceinline__ void linear_few_finish(const LinearArgs& a, const float* own, int g, int ft, int r0, int rows, int part,
                                                  int split, bool use) {
  constexpr int width = GATED ? 16 : 32;
  LinearBias<uint2> bias;
  LinearTail<uint2> t;
  auto fetch = [&](int i) {
    const int col = (ft * width + i % width) * 4;
    bias = linear_bias<GATED, uint2>(a, g, use ? col : a.n_out);
    t = linear_tail<GATED, uint2>(a, r0 + i / width, col, use && i < rows * width && col < a.n_out);
  };
  int i = part * C::THREADS + (int)threadIdx.x;
  fetch(i);
  cluster_wait();
  for (; use && i < rows * width; i += split * C::THREADS) {
    const int r = i / width, b = i % width, col = (ft * width + b) * 4;
    float z[8] = {};
    const uint32_t at = smem_addr(own + r * C::PAD + b * 4);
    constexpr int AT_ONCE = GATED ? 4 : 8;
#pragma unroll 1
    for (int p = 0; p < split; p += AT_ONCE) {
      float4 f[AT_ONCE][GATED ? 2 : 1];
#pragma unroll
      for (int x = 0; x < AT_ONCE; ++x)
        if (p + x < split) {
          const uint32_t from = dsmem_map(at, p + x);
          f[x][0] = dsmem_ld_f32x4(from);
          if (GATED) f[x][GATED ? 1 : 0] = dsmem_ld_f32x4(from + 256);
        }
#pragma unroll
      for (int x = 0; x < AT_ONCE; ++x)
        if (p + x < split) {
#pragma unroll
          for (int j = 0; j < (GATED ? 2 : 1); ++j) {
            z[4 * j] += f[x][j].x;
            z[4 * j + 1] += f[x][j].y;
            z[4 * j + 2] += f[x][j].z;
            z[4 * j + 3] += f[x][j].w;
          }
        }
    }
    const uint2 y = linear_finish<BF16, GATED, 3>(a, bias, t, z, z + 4);
    if (col < a.n_out) *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(a.out) + (int64_t)(r0 + r) * a.ld_out + col) = y;
    if (i + split * C::THREADS < rows * width) fetch(i + split * C::THREADS);
  }
}

template <bool BF16, class C>
__global__ void __launch_bounds__(C::THREADS, 2) linear_few_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap map_w,
                                                               const __grid_constant__ RowMaps maps_x, int split) {
  extern __shared__ uint8_t few_smem_raw[];
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES], done;
  __shared__ uint32_t taddr_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint8_t* smem = few_smem_raw + ((1024 - (smem_addr(few_smem_raw) & 1023)) & 1023);
  const int part = blockIdx.x % split, ft = blockIdx.x / split, g = blockIdx.y;
  const int blocks = (a.K + 63) / 64;
  const int kb0 = (int)((int64_t)blocks * part / split), nkb = (int)((int64_t)blocks * (part + 1) / split) - kb0;
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&done, 1);
    fence_barrier_init();
  }
  // What the call before writes is not read ahead of the wait, but W may come to L2
  // (a product of one group knows its part; up to 48 MB of all CTAs' parts).
  if (warp == 0 && !a.seg_start && blockIdx.z == 0) {
    const int most = max(1, (int)((48ll << 20) / ((int64_t)gridDim.x * C::W)));
    for (int i = lane; i < min(nkb, most); i += 32) {
      tma_prefetch_3d(&map_w, (kb0 + i) * 64, ft * (a.gated ? 64 : 128), 0);
      if (a.gated) tma_prefetch_3d(&map_w, (kb0 + i) * 64, a.n_out + ft * 64, 0);
    }
  }
  // (tensor memory after the wait: the call before may still need all of it)
  after_previous_call();
  if (warp == 1) tc::tmem_alloc(&taddr_s, C::COLS);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = taddr_s;
  uint32_t bad = 0;
  const int2 seg = group_rows(a, g, bad);
  if (bad && tid == 0) set_error(a.err, bad);
  bool ok = true, dead = false;  // (dead: known to all threads of the CTA)
  uint32_t it = 0;               // steps of K so far
  uint32_t tiles = 0;
  for (int r0 = seg.x + (int)blockIdx.z * C::NT; r0 < seg.y; r0 += (int)gridDim.z * C::NT, ++tiles) {
    const int rows = min(C::NT, seg.y - r0), cols = (rows + 15) / 16 * 16, box = row_box(rows);
    if (!dead) {
      if (warp == 0) {
        if (lane == 0) {
          for (int i = 0; i < nkb; ++i, ++it) {
            const int s = it % C::STAGES;
            if (it >= C::STAGES && !mbar_wait_soon(&empty[s], (it / C::STAGES - 1) & 1, a.wait_ns)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&full[s], C::W + (2048 << box));
            uint8_t* st = smem + s * C::STAGE;
            if (a.gated) {
              tma_load_3d(st, &map_w, (kb0 + i) * 64, ft * 64, g, &full[s]);
              tma_load_3d(st + 64 * 128, &map_w, (kb0 + i) * 64, a.n_out + ft * 64, g, &full[s]);
            } else {
              tma_load_3d(st, &map_w, (kb0 + i) * 64, ft * 128, g, &full[s]);
            }
            tma_load_2d(st + C::W, &maps_x.box[box], (kb0 + i) * 64, r0, &full[s]);
          }
        }
      } else if (warp == 1) {
        if (lane == 0) {
          const uint32_t id = BF16 ? tc::idesc_bf16_f32(128, cols) : tc::idesc_f16_f32(128, cols);
          for (int i = 0; i < nkb; ++i, ++it) {
            const int s = it % C::STAGES;
            if (!mbar_wait_soon(&full[s], (it / C::STAGES) & 1, a.wait_ns)) {
              ok = false;
              break;
            }
            tc::fence_after_sync();
            const uint32_t at = smem_addr(smem + s * C::STAGE);
            const uint64_t wd = tc::sw128_desc(at), xd = tc::sw128_desc(at + C::W);
#pragma unroll
            for (int q = 0; q < 4; ++q) tc::mma_bf16(tmem, wd + q * 2, xd + q * 2, id, i > 0 || q > 0);
            tc::mma_commit(&empty[s]);
          }
          // (every product issued is awaited, after a wait that gave up too: they write
          // to the tensor memory that is freed below)
          tc::mma_commit(&done);
          if (!ok || !mbar_wait_soon(&done, tiles & 1, a.wait_ns)) {
            ok = false;
            mbar_wait_bounded(&done, tiles & 1, kWaitLimitNs);
          }
        }
      }
      dead = !__syncthreads_and(ok);
      if (dead && tid == 0) {
        set_error(a.err, LORA_DEV_ERR_TIMEOUT);
        // (this thread's copies in flight write to the CTA's memory)
        for (uint32_t j = it > C::STAGES ? it - C::STAGES : 0; j < it; ++j)
          mbar_wait_bounded(&full[j % C::STAGES], (j / C::STAGES) & 1, kWaitLimitNs);
      }
    }
    float* own = reinterpret_cast<float*>(smem);  // [rows][PAD]: this CTA's part of the sums
    if (!dead && warp >= 2 && warp < 6) {
      tc::fence_after_sync();
      const int q = warp & 3;
#pragma unroll 2
      for (int c = 0; c < rows; c += 16) {
        float v[16];
        tc::tmem_ld16(tmem + ((uint32_t)(q * 32) << 16) + c, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) own[(c + i) * C::PAD + q * 32 + lane] = v[i];
      }
      tc::fence_before_sync();
    }
    __syncwarp();
    cluster_arrive_release_smem();
    if (a.gated)
      linear_few_finish<BF16, true, C>(a, own, g, ft, r0, rows, part, split, !dead);
    else
      linear_few_finish<BF16, false, C>(a, own, g, ft, r0, rows, part, split, !dead);
    fence_proxy_async_smem();  // (the memory is next written by copies)
    __syncwarp();
    cluster_arrive();
    cluster_wait();
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 1) tc::tmem_dealloc(tmem, C::COLS);
}

// ------------------------------------------------------------ many rows --
// A pair of CTAs works on a tile of 256 rows of W and up to 256 of x: each holds
// half of both (cta_group::2), so that a step of 64 of K costs an SM 32 KB of
// copies for 512 cycles of products.  Persistent: a warp that lays out the pair's
// items ahead, a load warp, an MMA warp (of the even CTA) and 8 epilogue warps, the
// sums of one tile in one half of tensor memory while the epilogue reads the other's.
// Bound: the tensor cores while K is long (8192 x 4096 by 28672 1045 to 1075 us, 1790
// to 1840 TFLOP/s; gated with silu and delta 1060 to 1120; products without copies or an
// epilogue 1000, copies alone 875), W's bytes for the experts of few tokens (16384 rows
// of 64 experts, 2048 by 1536 gated with delta: 106 to 122 us, by the run; without an
// epilogue 88), and the epilogue where K is short (768 by 2048: 63 to 74 us, without one
// 48).  Tried:
// descriptors from one lane 1086 us where the whole warp takes 1000 (products alone); six
// stages and 16 columns of the epilogue at once, with flags instead of forms of the
// kernel, 154 us for the experts' 106; erf and tanh inlined for every value 376 us where
// 65536 rows of the experts now take 270, by what the roles then fetch of instructions.
struct Pair {
  static constexpr int W = 128 * 128, X = 128 * 128, STAGE = W + X, STAGES = 5;
  static constexpr int EPI = 8, EPI_WARP = 4, THREADS = (EPI_WARP + EPI) * 32;
  static constexpr int PAD = 36, BUF = 32 * PAD;  // floats: 32 rows of 32 sums
  static constexpr int UNIT = 64, UNITS = 4;      // a tile is 1 to 4 units of rows
  static constexpr int BAND = 16;                 // row tiles that a feature tile is used for in turn
  static constexpr int BAND_COST = BAND * 16;
  static constexpr int MAX = 80;                  // pairs that share tiles
  static constexpr int PART = 128 * 256;          // floats of a CTA's part of a tile
  static constexpr int ITEMS = 4;                 // items laid out ahead
  static constexpr int SHARE = 512;               // what sharing tiles costs a pair, as 32 steps of a full tile
  static constexpr size_t smem(int groups) { return 1024 + (size_t)STAGES * STAGE + EPI * BUF * 4 + (size_t)(groups + 1) * 8; }
};
constexpr size_t kLinearCounterBytes = (size_t)Pair::MAX * 8 * 4;
constexpr size_t kLinearPartFloats = (size_t)Pair::MAX * 2 * 2 * Pair::PART;

// What a step of 64 of K costs by a tile's units of rows (measured: 0.22, 0.23, 0.26,
// 0.31 us).
__device__ __forceinline__ int unit_cost(int units) { return units == 4 ? 16 : 10 + units; }

// A pair's work: steps [kb0, kb1) of a tile's K.  A tile that several pairs share
// is finished by the last of them, which adds the others' parts in the order of K.
struct PairItem {
  int g, row0, rows, ft, kb0, kb1;
  int head, parts, part;  // the pair that has the tile's first steps, how many share it, which this one is
  int last;               // of the pair's items
};

// The pairs' items.  Tiles lie end to end: by group, band of 16 row tiles, feature
// tile, row tile.  Whole rounds of tiles are taken in turns, so that the pairs use
// the same rows and weights at the same time (contiguous shares of all: 16384 rows
// of 64 experts 197 us for 148, x read from memory again); the last rounds are cut
// into equal shares of cost, within tiles where need be.  A pair's place moves on by
// 13 a round: full and ragged row tiles alternate, and 76 pairs would meet the same
// of them each time (16384 rows of 64 experts, 768 by 2048: 158 us for 100).
struct PairWalk {
  const LinearArgs& a;
  const int2* pre;  // of the groups: tiles and cost (a step of K) so far
  int features, blocks, pairs, me;
  int round, t_end;                          // of the tiles in turn
  bool moved;
  int g, units, rts, band, width, ft, rt;    // the tile of the shares; row tiles of its band
  int2 seg;
  int at, base, total;                       // its position; of the shares: first position, cost (a step of K)
  int sharers, rest;                         // pairs that share, and what is left over of equal shares
  int64_t share;                             // a pair's cost

  __device__ __forceinline__ PairWalk(const LinearArgs& a, const int2* pre, int features, int pairs, int me)
      : a(a), pre(pre), features(features), blocks((a.K + 63) / 64), pairs(pairs), me(me) {}
  __device__ __forceinline__ void start() {
    const int tiles = pre[a.groups].x;
    round = 0;
    int turns = tiles / pairs;
    if (tiles % pairs && turns) --turns;
    t_end = a.counters ? turns * pairs : tiles;
    base = total = 0;
    if (t_end < tiles) {
      locate_tile(t_end);
      base = at;
      total = pre[a.groups].y - base;
      const int64_t whole = (int64_t)((unsigned)(tiles - t_end + pairs - 1) / (unsigned)pairs) * 16 * blocks;  // a pair's cost without
      // Shared, row tiles that use the same weights are no longer at the same place in
      // K, and weights that L2 does not hold meanwhile are read again (600 rows of 13824
      // by 5120: 71 us whole, 97 shared; 1023 rows, just above one tile a pair, 135 and 98).
      // Between 9/8 of a round and two, sharing is not measured (1280 rows, 1.32: whole 134).
      const int left = tiles - t_end;
      const bool again = a.groups == 1 && width > 1 && (int64_t)(left / width) * (256 * 2) * a.K > (64 << 20) &&
                         (left < pairs || left * 8 > pairs * 9);
      if (again || (int64_t)total * blocks + (int64_t)Pair::SHARE * pairs >= whole * pairs) {
        t_end = tiles;
        total = 0;
      }
    }
    // a share is at least 8 steps of a full tile
    const int64_t all = (int64_t)total * blocks, most = all >> 7;
    sharers = (int)(most < 1 ? 1 : (most < pairs ? most : pairs));
    share = all / sharers;
    rest = (int)(all - share * sharers);
    moved = true;  // (`next` begins the shares)
  }
  __device__ __forceinline__ int turn() const { return round * pairs + (int)((unsigned)(me + 13 * round) % (unsigned)pairs); }
  __device__ __forceinline__ void begin() {
    if (me < sharers && total > 0) locate((int)(edge(me) / blocks));
  }
  __device__ __forceinline__ int64_t edge(int i) const {
    return (int64_t)base * blocks + share * i + (unsigned)(rest * i) / (unsigned)sharers;
  }
  __device__ __forceinline__ int cost_of(int row_tile) const {
    return row_tile + 1 < rts ? 16 : unit_cost(units - row_tile * Pair::UNITS);
  }
  __device__ __forceinline__ void enter(int group) {
    g = group;
    uint32_t bad = 0;
    seg = group_rows(a, g, bad);
    units = (seg.y - seg.x + Pair::UNIT - 1) / Pair::UNIT;
    rts = (units + Pair::UNITS - 1) / Pair::UNITS;
  }
  __device__ __forceinline__ void enter_band(int b) {
    band = b;
    width = min(Pair::BAND, rts - b * Pair::BAND);
  }
  __device__ __forceinline__ int band_cost() const { return (width - 1) * 16 + cost_of(band * Pair::BAND + width - 1); }
  template <class F>
  __device__ __forceinline__ int group_of(F before) const {  // the last group before which it holds
    int lo = 0, hi = a.groups;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (before(pre[mid])) lo = mid; else hi = mid;
    }
    return lo;
  }
  __device__ __forceinline__ void locate_tile(int tile) {
    enter(group_of([&](int2 v) { return v.x <= tile; }));
    unsigned in = (unsigned)(tile - pre[g].x);
    enter_band((int)(in / (unsigned)(features * Pair::BAND)));
    in -= band * features * Pair::BAND;
    ft = (int)(in / (unsigned)width);
    rt = band * Pair::BAND + (int)in - ft * width;
    place();
  }
  __device__ __forceinline__ void place() {
    at = pre[g].y + band * features * Pair::BAND_COST + ft * band_cost() + (rt - band * Pair::BAND) * 16;
  }
  __device__ __forceinline__ void locate(int x) {  // the tile at a position
    enter(group_of([&](int2 v) { return v.y <= x; }));
    unsigned in = (unsigned)(x - pre[g].y);
    const unsigned whole = (unsigned)(features * Pair::BAND_COST);
    enter_band(min((int)(in / whole), (rts + Pair::BAND - 1) / Pair::BAND - 1));
    in -= band * whole;
    const unsigned row = (unsigned)band_cost();
    ft = (int)(in / row);
    in -= ft * row;
    rt = band * Pair::BAND + min((int)in / 16, width - 1);
    place();
  }
  // Where share i begins in the tile at `at`; near an end, there.
  __device__ __forceinline__ int bound(int i, int per_step) const {
    const int64_t d = edge(i) - (int64_t)at * blocks;
    if (d <= 0) return 0;
    if (d >= (int64_t)per_step * blocks) return blocks;
    const int kb = (int)((unsigned)d / (unsigned)per_step);
    return kb < 4 ? 0 : (blocks - kb < 4 ? blocks : kb);
  }
  __device__ __forceinline__ void fill(PairItem& p) const {
    p.g = g;
    p.ft = ft;
    p.row0 = seg.x + rt * Pair::UNITS * Pair::UNIT;
    p.rows = min(seg.y - p.row0, Pair::UNITS * Pair::UNIT);
    p.kb0 = 0;
    p.kb1 = blocks;
    p.parts = 1;
    p.head = p.part = p.last = 0;
  }
  __device__ __forceinline__ bool next(PairItem& p) {
    if (turn() < t_end) {
      locate_tile(turn());
      fill(p);
      ++round;
      moved = true;
      return true;
    }
    if (moved) begin();
    moved = false;
    if (me >= sharers || total <= 0) return false;
    const int64_t end = edge(me + 1);
    while (g < a.groups && (int64_t)at * blocks < end) {
      const int per_step = cost_of(rt), lo = bound(me, per_step), hi = bound(me + 1, per_step);
      if (lo < hi) {
        fill(p);
        p.kb0 = lo;
        p.kb1 = hi;
        int first = me, last = me;
        while (first > 0 && bound(first, per_step) > 0) --first;
        while (last + 1 < sharers && bound(last + 1, per_step) < blocks) ++last;
        p.head = first;
        p.parts = last - first + 1;
        p.part = me - first;
        p.last = hi < blocks || (int64_t)(at + per_step) * blocks >= end;
      }
      at += per_step;
      if (++rt == band * Pair::BAND + width) {
        if (++ft == features) {
          ft = 0;
          if ((band + 1) * Pair::BAND < rts) {
            enter_band(band + 1);
          } else {
            do {
              if (++g < a.groups) enter(g);
            } while (g < a.groups && rts == 0);
            if (g < a.groups) enter_band(0);
          }
        }
        rt = band * Pair::BAND;
      }
      if (lo < hi) return true;
    }
    return false;
  }
};

// AND of a predicate over the `threads` threads that meet at barrier `id`.
__device__ __forceinline__ bool barrier_and(int id, int threads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void barrier_sync(int id, int threads) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Where part x of a shared tile lies: [2 slots][2 CTAs][8 warps][128 columns][32
// rows of W] a pair; a pair has the first steps of one shared tile at most (slot 1)
// and later ones of one (slot 0).
__device__ __forceinline__ float* part_of(const LinearArgs& a, const PairItem& p, int x, uint32_t rank, int warp) {
  return a.parts + ((int64_t)((p.head + x) * 2 + (x == 0)) * 2 + rank) * Pair::PART + warp * 128 * 32;
}
// How many pairs have come to a shared tile, of the warps that meet at barrier `bar`.
__device__ __forceinline__ uint32_t* count_of(const LinearArgs& a, const PairItem& p, uint32_t rank, int bar) {
  return a.counters + (p.head * 2 + (int)rank) * 4 + bar - 1;
}

// Counts a pair's shared tiles from item `n` on, without finishing any: for warps that
// leave after a wait for an item gave up, so that the counters end at zero all the same.
// (Not inlined: it is reached after a failure only, and the epilogue has no registers left.)
__device__ __noinline__ void count_rest(const LinearArgs& a, const int2* pre, int features, uint32_t n, uint32_t rank, int bar) {
  PairWalk walk(a, pre, features, gridDim.x / 2, blockIdx.x / 2);
  walk.start();
  PairItem p;
  for (uint32_t i = 0; walk.next(p); ++i) {
    if (i < n || p.parts < 2) continue;
    uint32_t* count = count_of(a, p, rank, bar);
    if (atomicAdd(count, 1u) + 1 == (uint32_t)p.parts) *count = 0;
  }
}

template <bool BF16, bool GATED, int EXTRA>
__global__ void __launch_bounds__(Pair::THREADS, 1) linear_pair_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap map_w,
                                                                       const __grid_constant__ RowMaps maps_x) {
  using C = Pair;
  extern __shared__ uint8_t pair_smem_raw[];
  __shared__ uint64_t full[C::STAGES], empty[C::STAGES], acc_full[2], acc_empty[2], item_full[C::ITEMS], item_empty[C::ITEMS], drain;
  __shared__ uint64_t part_full[C::EPI];
  __shared__ PairItem items[C::ITEMS];
  __shared__ uint32_t taddr_s, failed_s, issued_s, tx_s[C::STAGES];  // (steps copied by this CTA, their bytes)
  __shared__ int2 scan_s[C::THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = cluster_rank();
  uint8_t* smem = pair_smem_raw + ((1024 - (smem_addr(pair_smem_raw) & 1023)) & 1023);
  float* epi_s = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE);
  int2* pre = reinterpret_cast<int2*>(epi_s + C::EPI * C::BUF);  // the groups' tiles and costs, summed
  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * C::EPI);
    }
    for (int i = 0; i < C::ITEMS; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], 1 + (rank == 0) + C::EPI);  // load, MMA and epilogue warps
    }
    for (int i = 0; i < C::EPI; ++i) mbar_init(&part_full[i], 1);
    mbar_init(&drain, 1);
    failed_s = 0;
    fence_barrier_init();
  }
  __syncwarp();
  cluster_arrive();  // (the barriers of both are ready at the wait)
  // (a product of one group lays out its work ahead of the wait for the call before)
  if (a.seg_start) after_previous_call();
  constexpr int per_pair = GATED ? 128 : 256;
  const int features = (a.n_out + per_pair - 1) / per_pair;
  {
    uint32_t bad = 0;
    const int per = (a.groups + C::THREADS - 1) / C::THREADS;
    int2 sum = make_int2(0, 0);
    for (int i = 0; i < per; ++i) {
      const int g = tid * per + i;
      if (g >= a.groups) break;
      const int2 seg = group_rows(a, g, bad);
      const int units = (seg.y - seg.x + C::UNIT - 1) / C::UNIT, whole = units / C::UNITS, rest = units % C::UNITS;
      const int2 v = make_int2(features * (whole + (rest != 0)), features * (whole * 16 + (rest ? unit_cost(rest) : 0)));
      pre[g] = v;
      sum.x += v.x;
      sum.y += v.y;
    }
    if (bad && blockIdx.x == 0) set_error(a.err, bad);
    // (segments that overlap could be more rows than there are: nothing is done then)
    const bool none = __syncthreads_or(bad != 0);
    if (none) sum = make_int2(0, 0);
    int2 inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc.x, d), y = __shfl_up_sync(0xffffffffu, inc.y, d);
      if (lane >= d) {
        inc.x += x;
        inc.y += y;
      }
    }
    if (lane == 31) scan_s[warp] = inc;
    __syncthreads();
    int2 run = make_int2(inc.x - sum.x, inc.y - sum.y);
    for (int w = 0; w < warp; ++w) {
      run.x += scan_s[w].x;
      run.y += scan_s[w].y;
    }
    for (int i = 0; i < per; ++i) {
      const int g = tid * per + i;
      if (g >= a.groups) break;
      const int2 v = none ? make_int2(0, 0) : pre[g];
      pre[g] = run;
      run.x += v.x;
      run.y += v.y;
    }
    if (tid == C::THREADS - 1) pre[a.groups] = run;
  }
  __syncthreads();
  PairWalk walk(a, pre, features, gridDim.x / 2, blockIdx.x / 2);
  PairItem p;
  if (warp == 3 && lane == 0) {
    walk.start();
    if (!walk.next(p)) p.parts = 0;
  }
  __syncwarp();
  if (!a.seg_start) after_previous_call();
  if (warp == 2) tc::tmem_alloc_pair(&taddr_s, 512);
  tc::fence_before_sync();
  __syncthreads();
  cluster_wait();
  tc::fence_after_sync();
  const uint32_t tmem = taddr_s;
  // An item from the warp that lays them out (false: there are no more) and, once
  // it is no longer needed, back.  After a wait that gave up a role passes on
  // without work, and leaves where it was one for an item.
  uint32_t n = 0;  // items so far
  bool ok = true;
  auto come = [&]() -> bool { return mbar_wait_soon(&item_full[n % C::ITEMS], (n / C::ITEMS) & 1, a.wait_ns); };
  auto take = [&]() -> bool {
    if (!come()) return ok = false;
    p = items[n % C::ITEMS];
    return p.parts > 0;
  };
  auto pass = [&]() {  // (by one thread)
    mbar_arrive(&item_empty[n % C::ITEMS]);
  };
  if (warp == 0) {
    // ------------------------------------------------------------------ load
    if (lane == 0) {
      uint32_t it = 0;
      const uint32_t leader_full = dsmem_map(smem_addr(full), 0);
      for (; take(); ++n) {
        pass();
        const int half = (p.rows + 63) / 64 * 32, box = row_box(half);
        const uint32_t bytes = C::W + (2048u << box);
        for (int kb = p.kb0; kb < p.kb1 && ok; ++kb, ++it) {
          const int s = it % C::STAGES;
          if (it >= C::STAGES && !mbar_wait_soon(&empty[s], (it / C::STAGES - 1) & 1, a.wait_ns)) {
            ok = false;
            break;
          }
          tx_s[s] = bytes;
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * bytes);
          const uint32_t bar = leader_full + s * 8;
          uint8_t* st = smem + s * C::STAGE;
          if (GATED) {
            tma_load_3d_pair(st, &map_w, kb * 64, p.ft * 128 + (int)rank * 64, p.g, bar);
            tma_load_3d_pair(st + 64 * 128, &map_w, kb * 64, a.n_out + p.ft * 128 + (int)rank * 64, p.g, bar);
          } else {
            tma_load_3d_pair(st, &map_w, kb * 64, p.ft * 256 + (int)rank * 128, p.g, bar);
          }
          tma_load_2d_pair(st + C::W, &maps_x.box[box], kb * 64, p.row0 + (int)rank * half, bar);
        }
      }
      issued_s = it;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------- MMA
    // The warp runs whole, so that descriptors stay in uniform registers; one
    // lane is elected at each product and commit.
    if (rank == 0) {
      uint32_t s = 0, ph = 0;  // place and parity of the next step
      const uint64_t base = tc::sw128_desc(smem_addr(smem));
      auto commit = [&](uint64_t* bar, uint16_t mask) {
        if (tc::elect_one()) tc::mma_commit_pair(bar, mask);
      };
      for (; __all_sync(0xffffffffu, take()); ++n) {
        __syncwarp();
        if (lane == 0) pass();
        if (!ok) continue;
        const int cols = (p.rows + 63) / 64 * 64;
        const uint32_t id = BF16 ? tc::idesc_bf16_f32(256, cols) : tc::idesc_f16_f32(256, cols);
        const uint32_t acc = tmem + (n & 1) * 256;
        if (n >= 2) ok = __all_sync(0xffffffffu, mbar_wait_soon(&acc_empty[n & 1], (n / 2 - 1) & 1, a.wait_ns));
        if (!ok) continue;
        tc::fence_after_sync();
        for (int kb = p.kb0; kb < p.kb1; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait_soon(&full[s], ph, a.wait_ns));
          if (!ok) break;
          tc::fence_after_sync();
          const uint64_t wd = base + (uint64_t)(s * (C::STAGE / 16)), xd = wd + C::W / 16;
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (tc::elect_one()) tc::mma_pair(acc, wd + q * 2, xd + q * 2, id, kb > p.kb0 || q > 0);
          commit(&empty[s], 3);
          s = s + 1 == C::STAGES ? 0 : s + 1;
          ph ^= s == 0;
        }
        if (ok) commit(&acc_full[n & 1], 3);
      }
      // (every product issued is awaited before tensor memory is freed, whatever the limit)
      commit(&drain, 1);
      if (!mbar_wait_bounded(&drain, 0, max(a.wait_ns, (uint64_t)kWaitLimitNs))) ok = false;
    }
  } else if (warp == 3) {
    // ----------------------------------------------------------------- items
    if (lane == 0) {
      for (bool more = true; more; ++n) {  // (the first is laid out already)
        if (n > 0 && !walk.next(p)) p.parts = 0;
        more = p.parts > 0;
        if (n >= C::ITEMS && !mbar_wait_bounded(&item_empty[n % C::ITEMS], (n / C::ITEMS - 1) & 1, a.wait_ns)) {
          ok = false;
          break;
        }
        items[n % C::ITEMS] = p;
        mbar_arrive(&item_full[n % C::ITEMS]);
      }
    }
  } else if (warp >= C::EPI_WARP) {
    // -------------------------------------------------------------- epilogue
    // A warp reads 32 rows of W of half of the tile's columns.  Gated, the warps
    // of a half's first and second 32 rows work with those of the other half's.
    const int ew = warp - C::EPI_WARP, q = warp & 3, side = ew / 4, bar = 1 + side * 2 + (q & 1);
    float* buf = epi_s + ew * C::BUF;
    const float *first_half = epi_s + (side * 4 + (GATED ? q & 1 : q)) * C::BUF, *second_half = epi_s + (side * 4 + 2 + (q & 1)) * C::BUF;
    constexpr int MINE = GATED ? 2 : 4;  // of 32 rows, a lane's, 8 apart
    const int block = lane % 4, my_row = (GATED ? (q >> 1) * 16 : 0) + lane / 4;
    const uint32_t leader_empty = dsmem_map(smem_addr(acc_empty), 0);
    const bool counts = q < 2 && lane == 0;  // (one thread of the warps that work together)
    // (after a wait that gave up, shared tiles are still counted, so that the
    // counters end at zero)
    for (;; ++n) {
      // (the warps that work together take an item, or leave, together: one alone
      // would wait for the other without end)
      if (!barrier_and(bar, 64, come())) {
        ok = false;
        if (counts && a.counters) count_rest(a, pre, features, n, rank, bar);
        break;
      }
      p = items[n % C::ITEMS];
      if (p.parts == 0) break;
      __syncwarp();
      if (lane == 0) pass();
      const int cols = (p.rows + 63) / 64 * 64, c0 = side * cols / 2, c1 = min(c0 + cols / 2, p.rows);
      const int col = p.ft * per_pair + (int)rank * (per_pair / 2) + (GATED ? q & 1 : q) * 32 + block * 8;
      // delta and residual on their way to L2 while the products run: 64 bytes a row,
      // half of the rows for the warps that work together (read from there as each part
      // begins; into registers a part ahead instead, 1023 rows down 111 us for 103)
      if (EXTRA) {
        const int first = col - block * 8;
        for (int r = c0 + lane + (GATED ? (q >> 1) * 32 : 0); r < c1 && first < a.n_out; r += GATED ? 64 : 32) {
          const int64_t row = p.row0 + r;
          if (EXTRA & 1) {
            prefetch_l2(reinterpret_cast<const uint16_t*>(a.delta) + row * a.ld_delta + first);
            if (GATED) prefetch_l2(reinterpret_cast<const uint16_t*>(a.delta) + row * a.ld_delta + a.n_out + first);
          }
          if (EXTRA & 2) prefetch_l2(reinterpret_cast<const uint16_t*>(a.residual) + row * a.ld_residual + first);
        }
      }
      if (ok) ok = mbar_wait_soon(&acc_full[n & 1], (n / 2) & 1, a.wait_ns);
      ok = barrier_and(bar, 64, ok);  // (the warps that work together go on together)
      tc::fence_after_sync();
      const uint32_t acc = tmem + (n & 1) * 256 + ((uint32_t)(q * 32) << 16);
      bool finish = ok;
      if (p.parts > 1) {
        // The last to come finishes the tile.  Who finds all others there need
        // not write a part; else it writes, and may be the last all the same.
        uint32_t* count = count_of(a, p, rank, bar);
        bool last = true;
        if (counts) {
          last = atomicAdd(count, 0u) + 1 == (uint32_t)p.parts;
          __threadfence();
        }
        if (!barrier_and(bar, 64, last)) {
          float* own = part_of(a, p, p.part, rank, ew) + lane;
          if (ok)
            for (int c = c0; c < c1; c += 32) {
              float v[32];
              tc::tmem_ld32(acc + c, v);
#pragma unroll
              for (int i = 0; i < 32; ++i) __stcg(own + (c - c0 + i) * 32, v[i]);
            }
          __threadfence();
          fence_proxy_async_global();  // (the part may be read by a bulk copy)
          barrier_sync(bar, 64);
          last = true;
          if (counts) {
            last = atomicAdd(count, 1u) + 1 == (uint32_t)p.parts;
            __threadfence();
          }
          last = barrier_and(bar, 64, last);
        } else {
          last = true;
        }
        if (last && counts) *count = 0;
        finish = last && ok;
        if (finish) {
          // The others' parts are added in the order of K, whoever adds, and the sums
          // go back to tensor memory.  Where this is the pair's last item, as it mostly
          // is, the operands' memory is free, and the parts come there by bulk copies,
          // `step` columns at once.
          const int others = p.parts - 1, step = C::STAGES * C::STAGE / (C::EPI * 128 * others) / 32 * 32;
          const bool copy = p.last && step > 0;
          float* room = reinterpret_cast<float*>(smem) + ew * (C::STAGES * C::STAGE / (C::EPI * 4));
          for (int c = c0, from_c = c0, ready = c0; c < c1; c += 32) {
            if (copy && c == ready) {
              const int count = min(step, c0 + cols / 2 - c);
              __syncwarp();
              if (lane == 0) {
                fence_proxy_async_global();
                mbar_arrive_expect_tx(&part_full[ew], others * count * 128);
                for (int x = 0, at = 0; x < p.parts; ++x)
                  if (x != p.part) bulk_g2s(room + at++ * step * 32, part_of(a, p, x, rank, ew) + (c - c0) * 32, count * 128, &part_full[ew]);
              }
              const uint32_t parity = ((c - c0) / step) & 1;
              ok = __all_sync(0xffffffffu, mbar_wait_soon(&part_full[ew], parity, a.wait_ns));
              if (!ok) {  // (what is on its way to the CTA's memory is awaited all the same)
                mbar_wait_bounded(&part_full[ew], parity, kWaitLimitNs);
                break;
              }
              from_c = c;
              ready += step;
            }
            float own[32], sum[32];
            tc::tmem_ld32(acc + c, own);
            for (int x = 0, at = 0; x < p.parts; ++x) {
              if (x == p.part) {
#pragma unroll
                for (int i = 0; i < 32; ++i) sum[i] = x ? sum[i] + own[i] : own[i];
                continue;
              }
              const float* from = copy ? room + (at * step + c - from_c) * 32 + lane : part_of(a, p, x, rank, ew) + (c - c0) * 32 + lane;
              ++at;
              float part[32];
              if (copy) {
#pragma unroll
                for (int i = 0; i < 32; ++i) part[i] = from[i * 32];
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) part[i] = __ldcg(from + i * 32);
              }
#pragma unroll
              for (int i = 0; i < 32; ++i) sum[i] = x ? sum[i] + part[i] : part[i];
            }
            tc::tmem_st16(acc + c, reinterpret_cast<const uint32_t*>(sum));
            tc::tmem_st16(acc + c + 16, reinterpret_cast<const uint32_t*>(sum + 16));
          }
          tc::tmem_wait_st();
          finish = barrier_and(bar, 64, ok);
        }
      }
      if (finish) {
        const LinearBias<uint4> bias = linear_bias<GATED, uint4>(a, p.g, col);
        LinearTail<uint4> tail[MINE];
        // (columns and rows past the tile's are read as the last, and not written)
        const int from_col = min(col, a.n_out - 8);
        auto fetch = [&](int c, int i) {
          const int64_t row = p.row0 + min(c + my_row + 8 * i, c1 - 1);
          if (EXTRA & 1) {
            tail[i].delta[0] = load8(a.delta, a.ld_delta, row, from_col);
            if (GATED) tail[i].delta[1] = load8(a.delta, a.ld_delta, row, a.n_out + from_col);
          }
          if (EXTRA & 2) tail[i].residual = load8(a.residual, a.ld_residual, row, from_col);
        };
        uint32_t sums[32];
        if (c0 < c1) tc::tmem_ld32_start(acc + c0, sums);
        for (int c = c0; c < c1; c += 32) {
#pragma unroll
          for (int i = 0; i < MINE; ++i) fetch(c, i);
          tc::tmem_ld32_wait(sums);
#pragma unroll
          for (int i = 0; i < 32; ++i) buf[i * C::PAD + lane] = __uint_as_float(sums[i]);
          if (GATED) barrier_sync(bar, 64); else __syncwarp();
          float z[MINE][GATED ? 16 : 8];
#pragma unroll
          for (int i = 0; i < MINE; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int at = (my_row + 8 * i) * C::PAD + block * 8 + 4 * j;
              *reinterpret_cast<float4*>(z[i] + 4 * j) = *reinterpret_cast<const float4*>(first_half + at);
              if (GATED) *reinterpret_cast<float4*>(z[i] + 8 + 4 * j) = *reinterpret_cast<const float4*>(second_half + at);
            }
          if (GATED) barrier_sync(bar, 64); else __syncwarp();
          if (c + 32 < c1) tc::tmem_ld32_start(acc + c + 32, sums);  // (ahead)
#pragma unroll
          for (int i = 0; i < MINE; ++i) {
            const uint4 y = linear_finish<BF16, GATED, EXTRA>(a, bias, tail[i], z[i], z[i] + 8);
            const int r = c + my_row + 8 * i;
            if (r < c1 && col < a.n_out) store8(a.out, a.ld_out, p.row0 + r, col, y);
          }
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(leader_empty + (n & 1) * 8);
    }
  }
  if (!ok) {
    set_error(a.err, LORA_DEV_ERR_TIMEOUT);
    for (int r = 0; r < 2; ++r) dsmem_st_f32(dsmem_map(smem_addr(&failed_s), r), 1.0f);
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  cluster_arrive();  // (neither CTA leaves while the other's products or copies use its memory)
  cluster_wait();
  if (*reinterpret_cast<volatile uint32_t*>(&failed_s)) {
    // After a wait that gave up, copies are still in flight: both CTAs' complete the
    // even one's barriers, which here come to expect what each has copied.
    if (tid == 0 && rank == 0) {
      const uint32_t mine = issued_s, other = dsmem_ld_u32(dsmem_map(smem_addr(&issued_s), 1)), most = max(mine, other);
      for (uint32_t j = mine; j < other; ++j)
        mbar_arrive_expect_tx(&full[j % C::STAGES], dsmem_ld_u32(dsmem_map(smem_addr(&tx_s[j % C::STAGES]), 1)));
      for (uint32_t j = other; j < mine; ++j) mbar_complete_tx(&full[j % C::STAGES], tx_s[j % C::STAGES]);
      for (uint32_t j = most > C::STAGES ? most - C::STAGES : 0; j < most; ++j)
        if (!mbar_wait_bounded(&full[j % C::STAGES], (j / C::STAGES) & 1, kWaitLimitNs)) set_error(a.err, LORA_DEV_ERR_INTERNAL);
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
  }
  if (warp == 2) tc::tmem_dealloc_pair(tmem, 512);
  cluster_arrive();
  cluster_wait();
}

}  // namespace lora
