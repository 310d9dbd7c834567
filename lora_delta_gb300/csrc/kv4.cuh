// The key/value cache held in 4 bits: its layout, the quantising store of new
// rows and the read of stored rows.
//
// A head's D dims (64, 128 or 256) form groups of 64.  A (token, head, group)
// keeps m = f16(min), s = f16((max - min) * (1 / 15)) and codes
// c = clamp(rint((x - m) * (1 / s)), 0, 15), each step rounded to float32, and
// stands for s * c + m.  Rounding s and m to f16 before the codes are taken
// makes the codes the nearest ones on the grid that is read back.  A group that
// f16 does not hold (an infinity, a NaN, a magnitude above 65504) keeps NaNs.
//
// Pages are [num_pages][kv_heads][page_size / 16] tiles of 16 tokens, so one
// (page, head) is contiguous and a bulk copy brings a tile whole:
//   key codes 8 D bytes | key (s, m) f16 pairs [16][D / 64] | value codes |
//   value pairs
// The codes lie so that the words a lane loads are operands of the
// 16 x 8 x 16 matrix instruction after one AND: a 4-bit code in bits 0-3 of a
// 16-bit half is the f16 subnormal code * 2^-24, in bits 4-7 code * 2^-20, and
// a shift by 8 brings the word's other two pairs there.  In a plane of
// W = min(D, 128) dims:
//   keys   [token 16][c 4][W / 32 words]: nibble i of word w is dim
//          64 (w / 2) + 16 c + 8 (w % 2) + i;
//   values [h 2][g 8][c 4][W / 32 words]: nibble j of a word's low / high half
//          is dim 64 (w / 2) + 8 g + 4 (w % 2) + j of token 8 h + 2 c / + 1.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace lora {

constexpr int kKvTile = 16;    // tokens of a tile
constexpr int kKvGroup = 64;   // dims that share a scale
constexpr int kKvThreads = 128;  // of a store or read CTA

__host__ __device__ constexpr int kv4_half_bytes(int D) { return 8 * D + 64 * (D / kKvGroup); }
__host__ __device__ constexpr int kv4_tile_bytes(int D) { return 2 * kv4_half_bytes(D); }

// Two packed 16-bit floats of the cache's type as float32, and back.
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if (BF16) return make_float2(bf16lo(v), bf16hi(v));
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF16) return pack_bf16x2(lo, hi);
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Least and largest of two pairs of the row type (a NaN stays one).
template <bool BF16>
__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <bool BF16>
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A group's least value and step from the lanes' least and largest pairs, over
// the lanes that differ in the bits from FROM to below TO of their number.
struct Kv4Scale {
  float m, r;     // least value and 1 / step as they are read back
  uint32_t pair;  // (s, m) as stored
};
template <bool BF16, int FROM, int TO>
__device__ __forceinline__ Kv4Scale kv4_scale(uint32_t lo2, uint32_t hi2) {
#pragma unroll
  for (int d = FROM; d < TO; d <<= 1) {
    lo2 = min2<BF16>(lo2, __shfl_xor_sync(0xffffffffu, lo2, d));
    hi2 = max2<BF16>(hi2, __shfl_xor_sync(0xffffffffu, hi2, d));
  }
  lo2 = min2<BF16>(lo2, lo2 >> 16 | lo2 << 16);
  hi2 = max2<BF16>(hi2, hi2 >> 16 | hi2 << 16);
  const float lo = unpack2<BF16>(lo2).x, hi = unpack2<BF16>(hi2).x;
  // (beyond f16, or not a number: neither is kept, and the group reads as NaN)
  const bool held = fabsf(lo) <= 65504.0f && fabsf(hi) <= 65504.0f;
  const __half m = held ? __float2half_rn(__fadd_rn(lo, 0.0f)) : __ushort_as_half(0x7fff);
  const __half s = held ? __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f)) : m;
  const float sf = __half2float(s);
  Kv4Scale q;
  q.m = __half2float(m);
  q.r = sf > 0.0f ? __frcp_rn(sf) : 0.0f;
  const __half2 sm = __halves2half2(s, m);
  q.pair = *reinterpret_cast<const uint32_t*>(&sm);
  return q;
}

// Codes of 8 values, the first in the lowest bits.  Each rounding is written
// out (no contraction), so that the codes are the format's, bit for bit; adding
// 1.5 2^23 rounds to whole numbers, ties to even, and a NaN becomes 0.  Four
// codes are put together as c0 + 16 c1 + 256 c2 + 4096 c3, exact in float32.
template <bool BF16>
__device__ __forceinline__ uint32_t kv4_codes(const uint4& raw, const Kv4Scale& q) {
  constexpr float kRound = 12582912.0f;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t half[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float c[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 v = unpack2<BF16>(w[2 * h + i]);
      c[2 * i] = fminf(fmaxf(__fmul_rn(__fsub_rn(v.x, q.m), q.r), 0.0f), 15.0f);
      c[2 * i + 1] = fminf(fmaxf(__fmul_rn(__fsub_rn(v.y, q.m), q.r), 0.0f), 15.0f);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __fsub_rn(__fadd_rn(c[i], kRound), kRound);
    const float all = fmaf(c[3], 4096.0f, fmaf(c[2], 256.0f, fmaf(c[1], 16.0f, c[0])));
    half[h] = __float_as_uint(__fadd_rn(all, kRound)) & 0xffffu;
  }
  return half[0] | half[1] << 16;
}

// The values of 8 codes, rounded once to the row type.
template <bool BF16>
__device__ __forceinline__ uint4 kv4_values(uint32_t codes, uint32_t pair) {
  const float2 sm = __half22float2(*reinterpret_cast<const __half2*>(&pair));
  auto v = [&](int i) { return fmaf(sm.x, (float)((codes >> (4 * i)) & 15u), sm.y); };
  return make_uint4(pack2<BF16>(v(0), v(1)), pack2<BF16>(v(2), v(3)), pack2<BF16>(v(4), v(5)),
                    pack2<BF16>(v(6), v(7)));
}

struct Kv4Rows {
  const void* k;  // read: destination
  const void* v;
  int64_t ld_k, ld_v;  // elements between rows
  uint8_t* pages;
  int64_t num_slots;  // num_pages * page_size
  int page_size, page_shift;  // log2 of the page size, or -1
  int heads, task_heads;      // heads, and heads of a task
  const int64_t* slot_map;
  int n;
  uint32_t* err;
};

// Store and read work in tasks of 8 adjacent rows' keys or values of some heads,
// a warp each: one head where there are few rows, else more, which share the
// look-up of the rows' places.
// Keys: a lane has a row and 16 bytes of its codes (16 dims of each group of a
// plane), so rows may lie anywhere.  Values: a lane has rows 2 c and 2 c + 1 and
// 8 dims of each group; where the two are one pair of a tile, as in a prompt
// begun at an even place, its words are whole, else they go by halves.
// Bound: the chain of a task (slots, rows, their shuffles, stores) and its
// instructions, 23 a value stored and 14 a value read: issue slots are two thirds
// full while an SM is active, half of the whole time, and most other cycles wait for
// rows.  HBM would allow 12.8 us of 8192 rows of 8 heads of 128 stored and read back:
// 27.7 us, 3.1 TB/s of the 86 MB that both move (12 CTAs an SM; at 8: 29.7).
template <int D, bool BF16, bool STORE>
__global__ void __launch_bounds__(kKvThreads, 12) kv4_rows_kernel(const Kv4Rows a) {
  constexpr int W = D < 128 ? D : 128, NP = D / W, WD = W / 32, GP = WD / 2;  // GP groups a plane
  constexpr int TILE = kv4_tile_bytes(D), HALF = kv4_half_bytes(D), G = D / kKvGroup;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int64_t head_step = (int64_t)(a.page_size / kKvTile) * TILE;
  const int blocks = (a.n + 7) / 8;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // (what the kernel before wrote is read from here on)
  constexpr int kWarps = kKvThreads / 32;
  const int parts = (a.heads + a.task_heads - 1) / a.task_heads;
  for (int task = blockIdx.x * kWarps + (threadIdx.x >> 5); task < 2 * blocks * parts; task += gridDim.x * kWarps) {
    const int block = (task >> 1) / parts, part = (task >> 1) - block * parts, row0 = block * 8;
    const int head0 = part * a.task_heads;
    const int head1 = head0 + a.task_heads < a.heads ? head0 + a.task_heads : a.heads;
    // the 8 rows' slots, one a lane, and where they are
    const int row = row0 + (lane & 7);
    const int64_t my_slot = row < a.n ? a.slot_map[row] : -1;
    if (my_slot >= a.num_slots && lane < 8) set_error(a.err, LORA_DEV_ERR_PAGE);
    int64_t my_place = -1;  // byte of its tile of the first head, + its place in the tile (tiles begin at 128s)
    if (my_slot >= 0 && my_slot < a.num_slots) {
      const int64_t page = a.page_shift >= 0 ? my_slot >> a.page_shift : my_slot / a.page_size;
      const int off = (int)(my_slot - page * a.page_size);
      my_place = ((page * a.heads + head0) * (a.page_size / kKvTile) + off / kKvTile) * TILE + off % kKvTile;
    }
    auto find = [&](int r, int& t) -> uint8_t* {  // the r-th row's tile and token
      const int64_t place = __shfl_sync(0xffffffffu, my_place, r);
      t = (int)(place & 15);
      return place >= 0 ? a.pages + (place - t) : nullptr;
    };
    if (task & 1) {  // keys: row g
      int t;
      uint8_t* tile = find(g, t);
      const uint16_t* row_k = reinterpret_cast<const uint16_t*>(a.k) + (int64_t)(row0 + g) * a.ld_k + head0 * D + c * 16;
#pragma unroll 1
      for (int head = head0; head < head1; ++head, tile += tile ? head_step : 0, row_k += D)
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        uint4* words = reinterpret_cast<uint4*>(tile + p * 8 * W + t * (W / 2) + c * (W / 8));
        uint32_t* pairs = reinterpret_cast<uint32_t*>(tile + 8 * D) + t * G + p * GP;
        uint32_t w[4] = {0, 0, 0, 0};
        if (STORE) {
          uint4 raw[WD];
#pragma unroll
          for (int x = 0; x < WD; ++x)
            raw[x] = row0 + g < a.n ? ldg_nc_v4(row_k + p * 128 + (x / 2) * 64 + (x % 2) * 8) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int q = 0; q < GP; ++q) {
            const uint4 &u = raw[2 * q], &v = raw[2 * q + 1];
            const Kv4Scale sc = kv4_scale<BF16, 1, 4>(
                min2<BF16>(min2<BF16>(min2<BF16>(u.x, u.y), min2<BF16>(u.z, u.w)),
                           min2<BF16>(min2<BF16>(v.x, v.y), min2<BF16>(v.z, v.w))),
                max2<BF16>(max2<BF16>(max2<BF16>(u.x, u.y), max2<BF16>(u.z, u.w)),
                           max2<BF16>(max2<BF16>(v.x, v.y), max2<BF16>(v.z, v.w))));
            w[2 * q] = kv4_codes<BF16>(u, sc);
            w[2 * q + 1] = kv4_codes<BF16>(v, sc);
            if (tile && c == 0) pairs[q] = sc.pair;
          }
          if (tile) {
            if (WD == 4)
              *words = make_uint4(w[0], w[1], w[2], w[3]);
            else
              *reinterpret_cast<uint2*>(words) = make_uint2(w[0], w[1]);
          }
        } else if (row0 + g < a.n) {
          uint32_t pair[2] = {0, 0};
          if (tile) {
            if (WD == 4) {
              *reinterpret_cast<uint4*>(w) = *words;
              *reinterpret_cast<uint2*>(pair) = *reinterpret_cast<const uint2*>(pairs);
            } else {
              *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(words);
              pair[0] = *pairs;
            }
          }
#pragma unroll
          for (int x = 0; x < WD; ++x)
            *reinterpret_cast<uint4*>(const_cast<uint16_t*>(row_k) + p * 128 + (x / 2) * 64 + (x % 2) * 8) =
                kv4_values<BF16>(w[x], pair[x / 2]);
        }
      }
    } else {  // values: rows 2 c and 2 c + 1, dims 8 g .. of each group
      uint8_t* tile[2];
      int t[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) tile[e] = find(2 * c + e, t[e]);
      const bool whole = tile[0] && tile[0] == tile[1] && t[0] % 2 == 0 && t[1] == t[0] + 1;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (tile[e]) tile[e] += HALF;
      const uint16_t* row_v = reinterpret_cast<const uint16_t*>(a.v) + (int64_t)(row0 + 2 * c) * a.ld_v + head0 * D + g * 8;
#pragma unroll 1
      for (int head = head0; head < head1; ++head, tile[0] += tile[0] ? head_step : 0, tile[1] += tile[1] ? head_step : 0, row_v += D)
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        // the place of the first word of the lane's dims, in a row's pair
        auto place = [&](int e) { return tile[e] + p * 8 * W + (t[e] / 8) * 4 * W + g * (W / 2) + (t[e] % 8 / 2) * (W / 8); };
        auto pairs = [&](int e) { return reinterpret_cast<uint32_t*>(tile[e] + 8 * D) + t[e] * G + p * GP; };
        uint32_t code[2][GP];  // 8 codes of a row and group
        if (STORE) {
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int q = 0; q < GP; ++q) {
              const uint4 u = row0 + 2 * c + e < a.n ? ldg_nc_v4(row_v + e * a.ld_v + p * 128 + q * 64) : make_uint4(0, 0, 0, 0);
              const Kv4Scale sc = kv4_scale<BF16, 4, 32>(min2<BF16>(min2<BF16>(u.x, u.y), min2<BF16>(u.z, u.w)),
                                                         max2<BF16>(max2<BF16>(u.x, u.y), max2<BF16>(u.z, u.w)));
              code[e][q] = kv4_codes<BF16>(u, sc);
              if (tile[e] && g == 0) pairs(e)[q] = sc.pair;
            }
          if (whole) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < GP; ++q) {
              w[2 * q] = __byte_perm(code[0][q], code[1][q], 0x5410);
              w[2 * q + 1] = __byte_perm(code[0][q], code[1][q], 0x7632);
            }
            if (WD == 4)
              *reinterpret_cast<uint4*>(place(0)) = make_uint4(w[0], w[1], w[2], w[3]);
            else
              *reinterpret_cast<uint2*>(place(0)) = make_uint2(w[0], w[1]);
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (tile[e]) {
                uint16_t* to = reinterpret_cast<uint16_t*>(place(e)) + t[e] % 2;
#pragma unroll
                for (int q = 0; q < GP; ++q) {
                  to[4 * q] = (uint16_t)code[e][q];
                  to[4 * q + 2] = (uint16_t)(code[e][q] >> 16);
                }
              }
          }
        } else {
          if (whole) {
            uint32_t w[4];
            if (WD == 4)
              *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(place(0));
            else
              *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(place(0));
#pragma unroll
            for (int q = 0; q < GP; ++q) {
              code[0][q] = __byte_perm(w[2 * q], w[2 * q + 1], 0x5410);
              code[1][q] = __byte_perm(w[2 * q], w[2 * q + 1], 0x7632);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int q = 0; q < GP; ++q) {
                code[e][q] = 0;
                if (tile[e]) {
                  const uint16_t* from = reinterpret_cast<const uint16_t*>(place(e)) + t[e] % 2;
                  code[e][q] = from[4 * q] | (uint32_t)from[4 * q + 2] << 16;
                }
              }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (row0 + 2 * c + e < a.n) {
#pragma unroll
              for (int q = 0; q < GP; ++q)
                *reinterpret_cast<uint4*>(const_cast<uint16_t*>(row_v) + e * a.ld_v + p * 128 + q * 64) =
                    kv4_values<BF16>(code[e][q], tile[e] ? pairs(e)[q] : 0u);
            }
        }
      }
    }
  }
}

}  // namespace lora
