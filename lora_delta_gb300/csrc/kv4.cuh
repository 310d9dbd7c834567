// The key/value cache held in 4 bits: its layout, the quantising store of new
// rows and the read of stored rows.
//
// A head's D dims (64, 128 or 256) form groups of 64.  A (token, head, group)
// keeps m = f16(min), s = f16((max - min) * (1 / 15)) and codes
// c = clamp(rint((x - m) * (1 / s)), 0, 15), each step rounded to float32, and
// stands for s * c + m.  Rounding s and m to f16 before the codes are taken
// makes the codes the nearest ones on the grid that is read back.
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

__host__ __device__ constexpr int kv4_half_bytes(int D) { return 8 * D + 64 * (D / kKvGroup); }
__host__ __device__ constexpr int kv4_tile_bytes(int D) { return 2 * kv4_half_bytes(D); }

// Byte of a tile's key codes that holds dims 8 * d8 .. + 7 of token t (a word).
template <int D>
__device__ __forceinline__ int kv4_key_word(int t, int d8) {
  constexpr int W = D < 128 ? D : 128;
  const int plane = d8 / (W / 8), e = d8 % (W / 8), group = e / 8, r = e % 8;
  return plane * 8 * W + t * (W / 2) + (r / 2) * (W / 8) + (2 * group + r % 2) * 4;
}
// Byte of a tile's value codes that holds dims 8 * d8 .. + 3 of token t (half
// a word); dims + 4 .. + 7 are 4 bytes on.
template <int D>
__device__ __forceinline__ int kv4_value_half(int t, int d8) {
  constexpr int W = D < 128 ? D : 128;
  const int plane = d8 / (W / 8), e = d8 % (W / 8), group = e / 8, g = e % 8;
  return plane * 8 * W + (t / 8) * 4 * W + g * (W / 2) + ((t % 8) / 2) * (W / 8) +
         2 * group * 4 + (t % 2) * 2;
}

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

struct Kv4Rows {
  const void* k;  // read: destination
  const void* v;
  int64_t ld_k, ld_v;  // elements between rows
  uint8_t* pages;
  int64_t num_slots;  // num_pages * page_size
  int page_size, heads;
  const int64_t* slot_map;
  int n;
  uint32_t* err;
};

// Tile of (slot, head) and the token within it.
__device__ __forceinline__ uint8_t* kv4_tile(uint8_t* pages, int64_t slot, int head, int page_size,
                                             int heads, int tile_bytes, int& token) {
  const int64_t page = slot / page_size;
  const int off = (int)(slot - page * page_size);
  token = off % kKvTile;
  const int64_t tile = (page * heads + head) * (page_size / kKvTile) + off / kKvTile;
  return pages + tile * tile_bytes;
}

// Store: 8 lanes quantise the 64 dims of one (row, head, group, key or value);
// a lane loads 16 bytes, and writes a word of key codes or two half words of
// value codes.  Each rounding is written out (no contraction), so that the
// codes are the format's, bit for bit.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) kv4_append_kernel(const Kv4Rows a) {
  constexpr int C8 = D / 8;
  const int64_t per_row = (int64_t)2 * a.heads * C8;
  const int64_t total = (int64_t)a.n * per_row;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < (total + 31) / 32 * 32;
       it += step) {
    const bool live = it < total;
    const int64_t row = live ? it / per_row : 0;
    int rest = live ? (int)(it - row * per_row) : 0;
    const int is_v = rest / (a.heads * C8);
    rest -= is_v * a.heads * C8;
    const int head = rest / C8, d8 = rest % C8;
    const int64_t slot = live ? a.slot_map[row] : -1;
    const bool good = slot >= 0 && slot < a.num_slots;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (good) {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(is_v ? a.v : a.k) +
                            row * (is_v ? a.ld_v : a.ld_k) + head * D + d8 * 8;
      raw = ldg_nc_v4(src);
    }
    float x[8];
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<BF16>(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
    float lo = x[0], hi = x[0];
    bool nan = x[0] != x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
      nan |= x[i] != x[i];
    }
    int any = nan;
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
      any |= __shfl_xor_sync(0xffffffffu, any, d);
    }
    if (slot >= a.num_slots) set_error(a.err, LORA_DEV_ERR_PAGE);
    if (!good) continue;
    const float kNan = __int_as_float(0x7fffffff);
    const __half m = __float2half_rn(any ? kNan : lo);
    const __half s = __float2half_rn(any ? kNan : __fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f));
    const float mf = __half2float(m), sf = __half2float(s);
    const float r = sf > 0.0f ? __frcp_rn(sf) : 0.0f;
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = rintf(__fmul_rn(__fsub_rn(x[i], mf), r));
      c[i] = (uint32_t)fminf(fmaxf(q, 0.0f), 15.0f);  // (a NaN becomes 0)
    }
    const uint32_t lo4 = c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12;
    const uint32_t hi4 = c[4] | c[5] << 4 | c[6] << 8 | c[7] << 12;
    int token;
    uint8_t* tile = kv4_tile(a.pages, slot, head, a.page_size, a.heads, kv4_tile_bytes(D), token) +
                    (is_v ? kv4_half_bytes(D) : 0);
    if (is_v) {
      uint16_t* p = reinterpret_cast<uint16_t*>(tile + kv4_value_half<D>(token, d8));
      p[0] = (uint16_t)lo4;
      p[2] = (uint16_t)hi4;
    } else {
      *reinterpret_cast<uint32_t*>(tile + kv4_key_word<D>(token, d8)) = lo4 | hi4 << 16;
    }
    if (d8 % 8 == 0)
      reinterpret_cast<__half2*>(tile + 8 * D)[token * (D / kKvGroup) + d8 / 8] =
          __halves2half2(s, m);
  }
}

// Read: the values that stored rows stand for, rounded once to the cache's
// type; a row whose slot is outside the cache reads zeros.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) kv4_read_kernel(const Kv4Rows a) {
  constexpr int C8 = D / 8;
  const int64_t per_row = (int64_t)2 * a.heads * C8;
  const int64_t total = (int64_t)a.n * per_row;
  const int64_t step = (int64_t)gridDim.x * 256;
  for (int64_t it = (int64_t)blockIdx.x * 256 + threadIdx.x; it < total; it += step) {
    const int64_t row = it / per_row;
    int rest = (int)(it - row * per_row);
    const int is_v = rest / (a.heads * C8);
    rest -= is_v * a.heads * C8;
    const int head = rest / C8, d8 = rest % C8;
    const int64_t slot = a.slot_map[row];
    uint4 o = make_uint4(0, 0, 0, 0);
    if (slot >= 0 && slot < a.num_slots) {
      int token;
      const uint8_t* tile =
          kv4_tile(a.pages, slot, head, a.page_size, a.heads, kv4_tile_bytes(D), token) +
          (is_v ? kv4_half_bytes(D) : 0);
      uint32_t lo4, hi4;
      if (is_v) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(tile + kv4_value_half<D>(token, d8));
        lo4 = p[0];
        hi4 = p[2];
      } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + kv4_key_word<D>(token, d8));
        lo4 = w & 0xffffu;
        hi4 = w >> 16;
      }
      const float2 sm = __half22float2(reinterpret_cast<const __half2*>(
          tile + 8 * D)[token * (D / kKvGroup) + d8 / 8]);
      auto val = [&](uint32_t h, int i) { return fmaf(sm.x, (float)((h >> (4 * i)) & 15u), sm.y); };
      o.x = pack2<BF16>(val(lo4, 0), val(lo4, 1));
      o.y = pack2<BF16>(val(lo4, 2), val(lo4, 3));
      o.z = pack2<BF16>(val(hi4, 0), val(hi4, 1));
      o.w = pack2<BF16>(val(hi4, 2), val(hi4, 3));
    } else if (slot >= a.num_slots) {
      set_error(a.err, LORA_DEV_ERR_PAGE);
    }
    uint16_t* dst = reinterpret_cast<uint16_t*>(const_cast<void*>(is_v ? a.v : a.k)) +
                    row * (is_v ? a.ld_v : a.ld_k) + head * D + d8 * 8;
    *reinterpret_cast<uint4*>(dst) = o;
  }
}

}  // namespace lora
