// Attention over the 4-bit key/value cache for many query rows per request.
#pragma once

#include "kv4_attn.cuh"

namespace lora {

// One CTA per (row, query head): tokens in chunks of 128, a thread's token's
// score, then the chunk's values with a thread per dim.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) kv4_attn_simple_kernel(const AttnArgs a) {
  const int row = blockIdx.x, qh = blockIdx.y, head = qh / a.group, tid = threadIdx.x;
  constexpr int G = D / kKvGroup;
  __shared__ float q_s[D];
  __shared__ float p_s[128];
  __shared__ float red_s[8];
  __shared__ int req_s;
  uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)row * a.ld_out + qh * D;
  if (tid == 0) {
    int b = -1;
    for (int i = 0; i < a.B; ++i)
      if (a.row_start[i] <= row && row < a.row_start[i + 1]) b = i;
    req_s = b;
  }
  __syncthreads();
  const int b = req_s;
  int64_t hi = 0, lo = 0;
  if (b >= 0) {
    const int64_t seq = a.seq_len[b], cap = (int64_t)a.max_pages * a.page_size;
    hi = seq - (a.row_start[b + 1] - row) + 1;
    if (seq < 0 || seq > cap) {
      if (tid == 0) set_error(a.err, LORA_DEV_ERR_LENGTH);
      hi = hi > cap ? cap : hi;
    }
    if (a.row_start[b + 1] - a.row_start[b] > a.max_q_len) {
      if (tid == 0) set_error(a.err, LORA_DEV_ERR_LENGTH);
      hi = 0;
    }
    lo = a.window > 0 && hi > a.window ? hi - a.window : 0;
  }
  for (int d = tid; d < D; d += 128) {
    const uint16_t raw = reinterpret_cast<const uint16_t*>(a.q)[(int64_t)row * a.ld_q + qh * D + d];
    q_s[d] = unpack2<BF16>(raw).x * a.scale_log2;
  }
  __syncthreads();
  float m = -INFINITY, l = 0.0f, acc[(D + 127) / 128] = {};
  uint8_t* pages = const_cast<uint8_t*>(a.pages);
  const int64_t slots = a.num_pages * a.page_size;
  auto slot_of = [&](int64_t t) -> int64_t {
    const int page = a.table[(int64_t)b * a.ld_table + t / a.page_size];
    const int64_t s = (int64_t)page * a.page_size + t % a.page_size;
    return page >= 0 && s < slots ? s : -1;
  };
  for (int64_t t0 = lo; t0 < hi; t0 += 128) {
    const int64_t t = t0 + tid;
    float s = -INFINITY;
    if (t < hi) {
      const int64_t slot = slot_of(t);
      if (slot < 0) {
        set_error(a.err, LORA_DEV_ERR_PAGE);
      } else {
        int tok;
        const uint8_t* tile = kv4_tile(pages, slot, head, a.page_size, a.heads, kv4_tile_bytes(D), tok);
        const __half2* sm = reinterpret_cast<const __half2*>(tile + 8 * D) + tok * G;
        s = 0.0f;
        for (int d8 = 0; d8 < D / 8; ++d8) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(tile + kv4_key_word<D>(tok, d8));
          const float2 f = __half22float2(sm[d8 / 8]);
          for (int i = 0; i < 8; ++i)
            s = fmaf(q_s[d8 * 8 + i], fmaf(f.x, (float)((w >> (4 * i)) & 15u), f.y), s);
        }
      }
    }
    float top = s;
    for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if ((tid & 31) == 0) red_s[tid >> 5] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red_s[0], red_s[1]), fmaxf(red_s[2], red_s[3]));
    const float m1 = fmaxf(m, top), base = m1 == -INFINITY ? 0.0f : m1;
    const float p = exp2f(s - base), keep = exp2f(m - base);
    float sum = p;
    for (int d = 16; d; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    p_s[tid] = p;
    if ((tid & 31) == 0) red_s[4 + (tid >> 5)] = sum;
    __syncthreads();
    l = l * keep + red_s[4] + red_s[5] + red_s[6] + red_s[7];
    for (int u = 0; u < (D + 127) / 128; ++u) {
      acc[u] *= keep;
      const int d = tid + u * 128;
      if (d >= D) continue;
      for (int j = 0; j < 128 && t0 + j < hi; ++j) {
        if (p_s[j] == 0.0f) continue;
        const int64_t slot = slot_of(t0 + j);
        if (slot < 0) continue;
        int tok;
        const uint8_t* tile = kv4_tile(pages, slot, head, a.page_size, a.heads, kv4_tile_bytes(D), tok) +
                              kv4_half_bytes(D);
        const uint8_t* hp = tile + kv4_value_half<D>(tok, d / 8) + ((d / 4) % 2) * 4;
        const float2 f = __half22float2(reinterpret_cast<const __half2*>(tile + 8 * D)[tok * G + d / 64]);
        const uint32_t code = (*reinterpret_cast<const uint16_t*>(hp) >> (4 * (d % 4))) & 15u;
        acc[u] = fmaf(p_s[j], fmaf(f.x, (float)code, f.y), acc[u]);
      }
    }
    m = m1;
    __syncthreads();
  }
  for (int u = 0; u < (D + 127) / 128; ++u) {
    const int d = tid + u * 128;
    if (d < D) out[d] = (uint16_t)pack2<BF16>(l != 0.0f ? acc[u] / l : 0.0f, 0.0f);
  }
  if (a.lse && tid == 0)
    a.lse[(int64_t)row * a.q_heads + qh] = l != 0.0f ? (m + log2f(l)) * 0.69314718055994531f : -INFINITY;
}


}  // namespace lora
