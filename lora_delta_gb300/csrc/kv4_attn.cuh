// Attention over the 4-bit key/value cache for few query rows per request and
// key/value head (single tokens, a few tokens): the cache is read once and
// codes go from shared memory into matrix-instruction operands with one AND.
//
// Per 16-token tile and (request, head), with 8 NT query rows as columns:
//   S^T = K Q^T    A = codes of 16 tokens x 16 dims, B = q of 16 dims x 8 rows
//   O^T = V^T P^T  A = codes of 16 dims x 16 tokens, B = weights of 16 tokens x 8 rows
// A code c in bits 0-3 of a 16-bit half is the f16 subnormal c 2^-24 and in
// bits 4-7 c 2^-20.  Keys: the operand's odd code pairs are the latter, so q is
// laid out with 2^-4 on the dims they meet.  Values: the odd pairs are rows
// 8-15 of the product, which take 2^-4 at the end.  Scales and least values:
//   s_t,g sum_d q_d c_d + m_t,g sum_d q_d    per group g of 64 dims (float32)
//   sum_t (p_t s_t,g) (c_t - 8) + sum_t p_t (m_t,g + 8 s_t,g)
// Values' codes less 8 (one exact subtraction a register) and least values with
// 8 s (rounded to f16 once) keep both sums near the result's size: with c and m
// as they are they grow over a long context and cancel, and what the matrix
// unit's float32 sums drop of them shows (f16, 60 thousand tokens a warp's part:
// 1.1e-2 of the result's norm for 5.6e-4; 300 tokens 4.5e-4 for 2.9e-4; the
// price is 1 to 5% of the time, a product with the constant 8 was dearer).
// The last sum and the denominator sum_t p_t are one more product, with
// the m of each group and ones as its rows.  q is brought to f16 by a power of
// two of its row (exact: 8 or 11 significant bits).  p is 2^6 exp2(s - max)
// with a running maximum that follows lazily (p <= 2^14), rounded to f16 once;
// p s is rounded to f16 with s taken relative to the largest so far of all groups of
// the head.  Both keep 11 bits down to 2^-20 of the largest weight (p s where the
// group's steps are as large as the largest; of one whose steps are 2^-k of
// that, down to 2^(k - 20)).  Sums are float32.
//
// A warp works on units of two tiles, so that waits, votes and page look-ups
// are paid once for 32 tokens.
//
// Bound: HBM for the cache's bytes, then what surrounds the stream.  bf16, 8
// heads of 128, 4 query heads each: one context of 131072 tokens 44 us (151 MB,
// 3.4 TB/s; by the clocks of an instrumented copy of the kernel its copies alone take
// 29 us, the arithmetic that they do not cover 8 us and the joins of the 152 CTAs'
// parts 7 us; issue slots are 55% full while an SM is active); 64 requests of 256 to
// 8192 tokens 52 us (170 MB, 3.2 TB/s); 256 of 17 to 2048 with 40 heads and as many
// query heads 159 us (624 MB, 3.9 TB/s, where the instructions of the units' loop
// count: a matrix product's 8 columns hold one row).
#pragma once

#include "kv4.cuh"

namespace lora {

constexpr int kAttnMaxReqs = 4096;

// mbar_wait_bounded for waits that are short and frequent: the global timer is
// first asked after 64 polls, and a poll sleeps no longer than the hardware's
// own limit (sleeps of a microsecond as there: 1% slower prompts).
__device__ __forceinline__ bool mbar_wait_soon(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  if (limit_ns == 0) return false;
  uint64_t t0 = 0;
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      const uint64_t t = globaltimer_ns();
      if (t0 == 0) t0 = t;
      else if (t - t0 > limit_ns) return false;
    }
  }
}

struct AttnArgs {
  void* out;
  const void* q;
  int64_t ld_out, ld_q;
  int n, q_heads, heads, group;  // group = q_heads / heads
  uint32_t group_inv;            // ceil(2^31 / group), for x / group where x group < 2^31
  const uint8_t* pages;
  int64_t num_pages;
  int page_size;
  const int32_t* table;
  int64_t ld_table;
  int cap;           // max_pages * page_size tokens, at most 2^29
  uint32_t tpp_inv;  // ceil(2^31 / (page_size / 16)), for tile numbers
  const int32_t* row_start;
  const int32_t* seq_len;
  int B, max_q_len, window;
  float scale_log2;  // softmax scale * log2(e)
  float* lse;
  uint32_t* err;
  uint64_t wait_ns;
  uint32_t* counters;  // [4 kAttnMaxCtas], zero between calls
  float* partials;     // [kAttnMaxCtas][2] slots, then [kAttnMaxCtas * warps] slots
};

// x / group.
__device__ __forceinline__ int div_group(const AttnArgs& a, int x) {
  return (int)(((uint64_t)(uint32_t)x * a.group_inv) >> 31);
}

// The page of a tile of 16 tokens.
__device__ __forceinline__ int page_of_tile(const AttnArgs& a, int tile) {
  return (int)(((uint64_t)(uint32_t)tile * a.tpp_inv) >> 31);
}

constexpr int kAttnMaxCtas = 256;
constexpr float kNoMax = -3e38f;    // running maximum before any token
constexpr float kNoOffset = 3e38f;  // and what weights' exponents take for it
// Maxima (log2) past this are far: of their scores' products with the scale
// float32 keeps too little, so a row subtracts its largest score before it scales,
// and that score's weight is the planned one at any size.
constexpr float kFarScore = 4096.0f;

// d += a(16 x 16, row) * b(16 x 8, col), f16 operands.
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
      "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of the 8 x 8 matrix of 16-bit values held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two f16 less two others.
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

template <int D_, bool BF16_, int NT_, int NW_>
struct Dec {
  static constexpr int D = D_, NT = NT_, NW = NW_;
  static constexpr bool BF16 = BF16_;
  static constexpr int G = D / 64, W = D < 128 ? D : 128, NP = D / W, WD = W / 32;
  static constexpr int MM = D / 16;  // matrix products of a tile's values
  static constexpr int TILE = kv4_tile_bytes(D), HALF = kv4_half_bytes(D);
  static constexpr int UNIT = 2 * kKvTile;  // tokens of a unit
  static constexpr int ROWS = 8 * NT;
  static constexpr int QREGS = D / 8;  // q operands of one column tile
  // operands of q stay in registers where there is room beside the sums
  static constexpr bool QSMEM = QREGS * NT > 32;
  static constexpr int F4 = 32 * MM * NT;           // float4s of O in a partial result
  static constexpr int SLOT = 4 * (F4 + 32 * NT);   // floats of a partial result
  static constexpr int QBYTES = QSMEM ? QREGS * NT * 32 * 4 : 0;
  static constexpr int QROW = QSMEM ? 0 : ROWS * D * 2;  // bytes of the next item's q
  static constexpr int THREADS = NW * 32;
  // a warp's ring of units; it also holds a partial result.  Two or three
  // units a warp are some 150 KB in flight on an SM, more than HBM's latency
  // asks for; deeper rings only make the loads that a warp waits for (q, page
  // numbers) queue behind them.
  static constexpr int MIN_STAGES = (SLOT * 4 + 2 * TILE - 1) / (2 * TILE) < 2 ? 2 : (SLOT * 4 + 2 * TILE - 1) / (2 * TILE);
  static constexpr int MAX_STAGES = MIN_STAGES > (D == 64 ? 4 : 3) ? MIN_STAGES : (D == 64 ? 4 : 3);
  // (with the requests' row starts and lengths beside the sums of their work,
  // or without)
  static constexpr size_t smem(int B, int stages, bool cached) {
    return (size_t)NW * (stages * 2 * TILE + QROW + QBYTES) + (size_t)(B + 1) * (cached ? 12 : 4) + 16;
  }
};

// Running state of one (request, head): O^T sums, the sums of p m (lanes of
// row group g < G) and of p (g == G), and what the weights' exponents take, of the
// lane's columns, 2 c and 2 c + 1 of each column tile: 6 less the maximum (log2), or
// 6 where the bit of `far` is set and scores are taken less the largest, `thr`.
template <class C>
struct DecState {
  float o[C::NT][C::MM][4];
  float z[C::NT][4];
  float l[C::NT][2], off[C::NT][2], m[C::NT][2];  // (l and m once finished)
  uint32_t far;
  int sexp;  // scales are taken as s 2^-sexp
};
constexpr int kMinSexp = -14, kMaxSexp = 15;

template <class C>
__device__ __forceinline__ void dec_reset(DecState<C>& st) {
#pragma unroll
  for (int n = 0; n < C::NT; ++n) {
#pragma unroll
    for (int i = 0; i < C::MM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[n][i][j] = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) st.z[n][j] = 0.0f;
    st.off[n][0] = st.off[n][1] = kNoOffset;
  }
  st.far = 0;
  st.sexp = kMinSexp;
}

// The sums of p m and p to every lane; o becomes the sum of p v in float32.
template <class C>
__device__ __forceinline__ void dec_finish(DecState<C>& st, const float (&qa)[C::NT][2], const float (&thr)[C::NT][2]) {
  const int c = threadIdx.x & 3;
  const float f0 = pow2i(18 + st.sexp), f1 = f0 * 0.0625f;  // 2^24 for the codes, 2^-6 for p
#pragma unroll
  for (int n = 0; n < C::NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      st.m[n][e] = (st.far >> (2 * n + e)) & 1u ? thr[n][e] * qa[n][e] : 6.0f - st.off[n][e];
      st.l[n][e] = __shfl_sync(0xffffffffu, st.z[n][e], C::G * 4 + c) * 0.015625f;
#pragma unroll
      for (int g = 0; g < C::G; ++g) {
        const float z = __shfl_sync(0xffffffffu, st.z[n][e], g * 4 + c) * 0.015625f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          st.o[n][4 * g + i][e] = fmaf(st.o[n][4 * g + i][e], f0, z);
          st.o[n][4 * g + i][2 + e] = fmaf(st.o[n][4 * g + i][2 + e], f1, z);
        }
      }
    }
}

// A finished state to a slot: the float4s of O, then (m, l) of the columns, a
// lane's next to one another's.
template <class C>
__device__ __forceinline__ void dec_save(const DecState<C>& st, float* slot, int lane) {
  float4* p = reinterpret_cast<float4*>(slot) + lane;
#pragma unroll
  for (int n = 0; n < C::NT; ++n) {
#pragma unroll
    for (int i = 0; i < C::MM; ++i)
      p[(n * C::MM + i) * 32] = make_float4(st.o[n][i][0], st.o[n][i][1], st.o[n][i][2], st.o[n][i][3]);
    p[C::F4 + n * 32] = make_float4(st.m[n][0], st.m[n][1], st.l[n][0], st.l[n][1]);
  }
}
// (o, ml) += (o2, ml2), the latter relative to its own maxima, ml.x and ml.y
// being the largest already.
__device__ __forceinline__ void dec_join(float4& o, float4& ml, const float4& o2, const float4& ml2) {
  const float b0 = exp2_fast(ml2.x - ml.x), b1 = exp2_fast(ml2.y - ml.y);
  ml.z = fmaf(ml2.z, b0, ml.z);
  ml.w = fmaf(ml2.w, b1, ml.w);
  o = make_float4(fmaf(o2.x, b0, o.x), fmaf(o2.y, b1, o.y), fmaf(o2.z, b0, o.z), fmaf(o2.w, b1, o.w));
}

// What a (request, head) is: its rows, and the tiles that they see.
struct DecReq {
  int row0, rows;     // first row of the batch; query rows (tokens * group)
  int pos0;           // position of the first row
  int seq;            // tokens that may be seen (clipped to the table)
  int tile0, units;   // first tile and number of units, 0 for a request without rows here
};

// (start, end: its first row and the next request's; seq: its length)
__device__ __forceinline__ DecReq dec_request(const AttnArgs& a, int start, int end, int seq, int max_rows,
                                              uint32_t& bad) {
  DecReq r;
  r.row0 = start;
  r.rows = 0;
  r.pos0 = 0;
  r.seq = 0;
  r.tile0 = 0;
  r.units = 0;
  if (end <= start) return r;
  if (start < 0 || end > a.n || end - start > a.max_q_len) {
    bad |= LORA_DEV_ERR_LENGTH;
    return r;
  }
  const int rows = (end - start) * a.group;
  if (rows > max_rows) return r;
  r.rows = rows;
  if (seq < 0 || seq > a.cap) bad |= LORA_DEV_ERR_LENGTH;
  r.pos0 = seq - (end - start);
  r.seq = seq < 0 ? 0 : (seq > a.cap ? a.cap : seq);
  const int first = a.window > 0 && r.pos0 + 1 - a.window > 0 ? r.pos0 + 1 - a.window : 0;
  r.tile0 = first / kKvTile;
  const int last = (r.seq + kKvTile - 1) / kKvTile;
  // (a request that sees nothing keeps one unit, all of it masked)
  r.units = last > r.tile0 ? (last - r.tile0 + 1) / 2 : 1;
  return r;
}

// The finished state's rows to out and lse.
template <class C>
__device__ __forceinline__ void dec_write(const AttnArgs& a, const DecReq& r, int h,
                                          const DecState<C>& st, int lane) {
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int n = 0; n < C::NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = n * 8 + 2 * c + e;
      if (rr >= r.rows) continue;
      const int j = div_group(a, rr), head = h * a.group + rr - j * a.group;
      const float l = st.l[n][e], inv = l != 0.0f ? __frcp_rn(l) : 0.0f;
      uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)(r.row0 + j) * a.ld_out + head * C::D;
#pragma unroll
      for (int q = 0; q < C::G; ++q) {
        uint4 v;
        uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = pack2<C::BF16>(st.o[n][4 * q + i][e] * inv, st.o[n][4 * q + i][2 + e] * inv);
        *reinterpret_cast<uint4*>(out + q * 64 + 8 * g) = v;
      }
      if (a.lse && g == 0)
        a.lse[(int64_t)(r.row0 + j) * a.q_heads + head] =
            l != 0.0f ? (st.m[n][e] + log2f(l)) * 0.69314718055994531f : -INFINITY;
    }
}

// The float4 number x of a joined result to out: two columns' two adjacent dims.
template <class C>
__device__ __forceinline__ void dec_write_part(const AttnArgs& a, const DecReq& r, int h, int x,
                                               const float4& o, const float4& ml) {
  const int lane = x & 31, g = lane >> 2, c = lane & 3, i = (x >> 5) % C::MM, n = (x >> 5) / C::MM;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int rr = n * 8 + 2 * c + e;
    if (rr >= r.rows) continue;
    const int j = div_group(a, rr), head = h * a.group + rr - j * a.group;
    const float l = e ? ml.w : ml.z, inv = l != 0.0f ? __frcp_rn(l) : 0.0f;
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)(r.row0 + j) * a.ld_out + head * C::D;
    *reinterpret_cast<uint32_t*>(out + (i / 4) * 64 + 8 * g + 2 * (i % 4)) =
        pack2<C::BF16>((e ? o.y : o.x) * inv, (e ? o.w : o.z) * inv);
    if (a.lse && i == 0 && g == 0)
      a.lse[(int64_t)(r.row0 + j) * a.q_heads + head] =
          l != 0.0f ? ((e ? ml.y : ml.x) + log2f(l)) * 0.69314718055994531f : -INFINITY;
  }
}

// Zeros to the rows [lo, hi), shared out over `parts` CTAs.
template <class C>
__device__ __noinline__ void zero_rows(uint16_t* out, int64_t ld_out, int q_heads, float* lse, int lo,
                                       int hi, int part, int parts) {
  const int width = q_heads * (C::D / 8);
  for (int row = lo + part; row < hi; row += parts) {
    for (int k = threadIdx.x; k < width; k += blockDim.x)
      *reinterpret_cast<uint4*>(out + row * ld_out + k * 8) = make_uint4(0, 0, 0, 0);
    if (lse)
      for (int k = threadIdx.x; k < q_heads; k += blockDim.x) lse[(int64_t)row * q_heads + k] = -INFINITY;
  }
}

// One unit: scores, weights and sums of the two tiles at `unit`.  With `edge`
// (of the whole warp) some row does not see some token, or a tile was not read
// (its bit of `got` is 0).
template <class C>
__device__ __forceinline__ void dec_unit(const AttnArgs& a, const DecReq& r, DecState<C>& st,
                                         uint8_t* unit, int tok0, uint32_t got, bool edge, int pos1,
                                         const uint32_t* q_s,
                                         const uint32_t (&qf)[C::QSMEM ? 1 : C::NT][C::QSMEM ? 1 : C::QREGS],
                                         const float (&qa)[C::NT][2], const float (&qb)[C::NT][C::G][2],
                                         float (&thr)[C::NT][2], int lane) {
  const int g = lane >> 2, c = lane & 3;
  auto seen_by_any = [&](int t, int tok) {
    return ((got >> t) & 1u) && tok < r.seq && tok <= pos1 && (a.window <= 0 || tok > r.pos0 - a.window);
  };
  auto seen_by = [&](int tok, int col) {
    const int pos = r.pos0 + div_group(a, col);
    return tok <= pos && (a.window <= 0 || tok > pos - a.window);
  };
  if (edge) {
    // values' scales of tokens that no row sees may hold anything; a group's that
    // is not finite is left out here and makes its dims NaN of rows that do see it
    uint32_t* sp = reinterpret_cast<uint32_t*>(unit + (lane >> 4) * C::TILE + C::HALF + 8 * C::D) + (lane & 15) * C::G;
    const bool any = seen_by_any(lane >> 4, tok0 + lane);
#pragma unroll 1
    for (int q = 0; q < C::G; ++q) {
      const bool odd = (sp[q] & 0x7c00u) == 0x7c00u || (sp[q] & 0x7c000000u) == 0x7c000000u;
      if (!any || odd) sp[q] = 0;
      for (uint32_t lost = __ballot_sync(0xffffffffu, any && odd); lost; lost &= lost - 1)
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (g == q && seen_by(tok0 + __ffs(lost) - 1, n * 8 + 2 * c + k)) st.z[n][k] = __int_as_float(0x7fffffff);
    }
    fence_proxy_async_smem();  // (the stage is next written by a bulk copy)
    __syncwarp();
  }
  float s[2][C::NT][4];
  bool up = false;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const uint8_t* tile = unit + t * C::TILE;
    float sc[C::NT][C::G][4];
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
      for (int q = 0; q < C::G; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][q][i] = 0.0f;
#pragma unroll
    for (int p = 0; p < C::NP; ++p) {
      uint32_t k0[C::WD], k1[C::WD];  // tokens g and g + 8
      const uint8_t* kp = tile + p * 8 * C::W + g * (C::W / 2) + c * (C::W / 8);
      if (C::WD == 4) {
        *reinterpret_cast<uint4*>(k0) = *reinterpret_cast<const uint4*>(kp);
        *reinterpret_cast<uint4*>(k1) = *reinterpret_cast<const uint4*>(kp + 4 * C::W);
      } else {
        *reinterpret_cast<uint2*>(k0) = *reinterpret_cast<const uint2*>(kp);
        *reinterpret_cast<uint2*>(k1) = *reinterpret_cast<const uint2*>(kp + 4 * C::W);
      }
#pragma unroll
      for (int w = 0; w < C::WD; ++w)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t x0 = u ? k0[w] >> 8 : k0[w], x1 = u ? k1[w] >> 8 : k1[w];
          const uint32_t a0 = x0 & 0x000f000fu, a2 = x0 & 0x00f000f0u;
          const uint32_t a1 = x1 & 0x000f000fu, a3 = x1 & 0x00f000f0u;
          const int at = (p * C::WD + w) * 4 + 2 * u;
#pragma unroll
          for (int n = 0; n < C::NT; ++n) {
            const uint32_t b0 = C::QSMEM ? q_s[(n * C::QREGS + at) * 32] : qf[C::QSMEM ? 0 : n][C::QSMEM ? 0 : at];
            const uint32_t b1 = C::QSMEM ? q_s[(n * C::QREGS + at + 1) * 32] : qf[C::QSMEM ? 0 : n][C::QSMEM ? 0 : at + 1];
            mma_f16(sc[n][(p * C::WD + w) / 2], a0, a1, a2, a3, b0, b1);
          }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float2 ks[C::G];  // scales and least values of token g + 8 u
#pragma unroll
      for (int q = 0; q < C::G; ++q)
        ks[q] = __half22float2(*reinterpret_cast<const __half2*>(tile + 8 * C::D + ((g + 8 * u) * C::G + q) * 4));
#pragma unroll
      for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float v = ks[0].x * sc[n][0][2 * u + k];
#pragma unroll
          for (int q = 1; q < C::G; ++q) v = fmaf(ks[q].x, sc[n][q][2 * u + k], v);
#pragma unroll
          for (int q = 0; q < C::G; ++q) v = fmaf(ks[q].y, qb[n][q][k], v);
          s[t][n][2 * u + k] = v;
        }
    }
  }
  if (edge) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tok = tok0 + t * kKvTile + g + 8 * u;
        const bool any = seen_by_any(t, tok);
#pragma unroll
        for (int n = 0; n < C::NT; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k)
            if (!any || !seen_by(tok, n * 8 + 2 * c + k)) s[t][n][2 * u + k] = -INFINITY;
      }
  }
#pragma unroll
  for (int n = 0; n < C::NT; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k)
      up |= fmaxf(fmaxf(s[0][n][k], s[0][n][2 + k]), fmaxf(s[1][n][k], s[1][n][2 + k])) > thr[n][k];

  // scales and least values of tokens 2 c, 2 c + 1 and 2 c + 8, 2 c + 9, paired
  __half2 vs[2][2][C::G], vm[2][2][C::G];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t x[2][C::G];
      const uint8_t* sp = unit + t * C::TILE + C::HALF + 8 * C::D + (2 * c + 8 * u) * C::G * 4;
      if (C::G == 1) {
        const uint2 v = *reinterpret_cast<const uint2*>(sp);
        x[0][0] = v.x;
        x[1][0] = v.y;
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int q = 0; q < C::G; q += 2)
            *reinterpret_cast<uint2*>(&x[e][q]) = *reinterpret_cast<const uint2*>(sp + (e * C::G + q) * 4);
      }
#pragma unroll
      for (int q = 0; q < C::G; ++q) {
        const uint32_t lo = __byte_perm(x[0][q], x[1][q], 0x5410), hi = __byte_perm(x[0][q], x[1][q], 0x7632);
        vs[t][u][q] = *reinterpret_cast<const __half2*>(&lo);
        vm[t][u][q] = __hfma2(vs[t][u][q], __float2half2_rn(8.0f), *reinterpret_cast<const __half2*>(&hi));
      }
    }
  __half2 top2 = vs[0][0][0];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int q = 0; q < C::G; ++q) top2 = __hmax2(top2, vs[t][u][q]);
  const float stop = __half2float(__hmax(__low2half(top2), __high2half(top2)));
  up |= stop >= pow2i(st.sexp + 1) || st.far;

  // new maxima only where a score is 2^8 above the old one, or a scale 2^1
  // above its unit; and what far maxima take
  if (__any_sync(0xffffffffu, up)) {
    float smax = 0.0f;  // (a scale that is not finite poisons its own rows only)
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int q = 0; q < C::G; ++q) {
          const float2 f = __half22float2(vs[t][u][q]);
          smax = fmaxf(smax, fmaxf(f.x <= 65504.0f ? f.x : 0.0f, f.y <= 65504.0f ? f.y : 0.0f));
        }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, d));
    int e = (int)((__float_as_uint(smax) >> 23) & 255u) - 127;
    e = e > kMaxSexp ? kMaxSexp : e;
    e = e < st.sexp ? st.sexp : e;
    const float fold = pow2i(st.sexp - e);
    st.sexp = e;
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float top = fmaxf(fmaxf(s[0][n][k], s[0][n][2 + k]), fmaxf(s[1][n][k], s[1][n][2 + k]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        // (the sums move from one base and offset to the other)
        const uint32_t bit = 1u << (2 * n + k);
        const bool far0 = st.far & bit;
        const float base0 = far0 ? thr[n][k] : 0.0f, off0 = st.off[n][k];
        if (far0) top = fmaxf(top, base0);
        const float m0 = far0 ? kNoMax : 6.0f - off0, m1 = fmaxf(m0, top * qa[n][k]);
        const bool far1 = fabsf(m1) > kFarScore && m1 > kNoMax;
        const float base1 = far1 ? top : 0.0f, off1 = far1 ? 6.0f : m1 > m0 ? 6.0f - m1 : off0;
        const float keep = exp2_fast(fmaf(base0 - base1, qa[n][k], off1 - off0));
        st.far = far1 ? st.far | bit : st.far & ~bit;
        st.off[n][k] = off1;
        thr[n][k] = far1 ? top : __fdividef(m1 + 8.0f, qa[n][k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i >> 1][n][2 * (i & 1) + k] -= base1;
        st.z[n][k] *= keep;
        const float ko = keep * fold;
#pragma unroll
        for (int i = 0; i < C::MM; ++i) {
          st.o[n][i][k] *= ko;
          st.o[n][i][2 + k] *= ko;
        }
      }
  }

  const __half2 unit_s = __float2half2_rn(pow2i(-st.sexp));
  const uint32_t ones = g == C::G ? 0x3c003c00u : 0u;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    uint32_t pt[C::NT][2];  // weights of tokens 2 c, + 1 and + 8, + 9 of row g
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          p[k] = exp2_fast(fmaf(s[t][n][2 * u + k], qa[n][k], st.off[n][k]));
          if (edge && s[t][n][2 * u + k] == -INFINITY) p[k] = 0.0f;
        }
        pt[n][u] = transpose8(half2_bits(p[0], p[1]));
      }
    uint32_t za[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      za[u] = ones;
#pragma unroll
      for (int q = 0; q < C::G; ++q)
        if (g == q) za[u] = *reinterpret_cast<const uint32_t*>(&vm[t][u][q]);
    }
    uint32_t pw[C::NT][C::G][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int q = 0; q < C::G; ++q) {
        const __half2 f = __hmul2(vs[t][u][q], unit_s);
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
          const __half2 w = __hmul2(*reinterpret_cast<const __half2*>(&pt[n][u]), f);
          pw[n][q][u] = *reinterpret_cast<const uint32_t*>(&w);
        }
      }
#pragma unroll
    for (int n = 0; n < C::NT; ++n) mma_f16(st.z[n], za[0], 0u, za[1], 0u, pt[n][0], pt[n][1]);
#pragma unroll
    for (int p = 0; p < C::NP; ++p) {
      uint32_t v0[C::WD], v1[C::WD];  // tokens 2 c, + 1 and 2 c + 8, + 9
      const uint8_t* vp = unit + t * C::TILE + C::HALF + p * 8 * C::W + g * (C::W / 2) + c * (C::W / 8);
      if (C::WD == 4) {
        *reinterpret_cast<uint4*>(v0) = *reinterpret_cast<const uint4*>(vp);
        *reinterpret_cast<uint4*>(v1) = *reinterpret_cast<const uint4*>(vp + 4 * C::W);
      } else {
        *reinterpret_cast<uint2*>(v0) = *reinterpret_cast<const uint2*>(vp);
        *reinterpret_cast<uint2*>(v1) = *reinterpret_cast<const uint2*>(vp + 4 * C::W);
      }
#pragma unroll
      for (int w = 0; w < C::WD; ++w)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t x0 = u ? v0[w] >> 8 : v0[w], x1 = u ? v1[w] >> 8 : v1[w];
          const uint32_t a0 = sub2(x0 & 0x000f000fu, 0x00080008u), a1 = sub2(x0 & 0x00f000f0u, 0x00800080u);
          const uint32_t a2 = sub2(x1 & 0x000f000fu, 0x00080008u), a3 = sub2(x1 & 0x00f000f0u, 0x00800080u);
          const int q = (p * C::WD + w) / 2;
#pragma unroll
          for (int n = 0; n < C::NT; ++n)
            mma_f16(st.o[n][(p * C::WD + w) * 2 + u], a0, a1, a2, a3, pw[n][q][0], pw[n][q][1]);
        }
    }
  }
}

// The work of all (request, head)s, laid end to end, is shared out evenly: a
// CTA takes a contiguous range and its warps contiguous parts of that.  An item
// counts its units and kItemCost more, for what its beginning and end take
// (with 1, 2, 3, 4: 64 requests 55.1, 51.7, 51, 50.1 us; 256 requests of 40 heads
// 167, 146, 151, 158).  A
// warp streams its units through a ring of bulk copies of its own; the next
// item's q comes by asynchronous copies meanwhile.  Where a (request, head)
// lies inside a warp's part it is written; what crosses parts is joined over
// the CTA's warps, and over CTAs by the last of them to arrive, in the order of
// the units (so results do not depend on the order of events).
constexpr int kItemCost = 3;

// A place in the work: request, head, unit (up to units + kItemCost).
struct DecPlace {
  int b, h, u;
};
__device__ __forceinline__ DecPlace dec_find(const AttnArgs& a, const int32_t* pre, int f) {
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] * a.heads <= f) lo = mid; else hi = mid;
  }
  const int cost = pre[lo + 1] - pre[lo], rest = f - pre[lo] * a.heads, h = rest / cost;
  return DecPlace{lo, h, rest - h * cost};
}

struct DecCross {  // an item that crosses CTAs: the first and last, its place in the first
  int c0, c1, into, h;
  DecReq r;
};
template <class C>
struct DecShared {
  // segments of items that cross the warps' parts: [0] the warp's first, [1]
  // its last (b -1: none), and the items' first and last + 1 unit
  int seg_b[C::NW][2], seg_h[C::NW][2], seg_lo[C::NW][2], seg_hi[C::NW][2];
  int chain_s[2 * C::NW], chains_s, last_s[2];
  DecCross cross_s[2];
};

// The end of a CTA: its warps' and the CTAs' parts of items put together.  Of
// its own, so that its registers do not weigh on the units' loop.
template <class C>
__device__ __noinline__ void dec_join_all(const AttnArgs& a, DecShared<C>& sh, uint8_t* dec_smem, int ring_bytes,
                                          const int32_t* starts, const int32_t* seqs, const int32_t* pre, int t0,
                                          int t1, int part, int chunk) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  uint32_t unused = 0;
  auto request = [&](int b) { return dec_request(a, starts[b], starts[b + 1], seqs[b], C::ROWS, unused); };
  // Joining in the CTA.  An item's segments are those of adjacent warps; its
  // first one here stands for it: warp w's, where the item began in w's part
  // or before the CTA's range.
  if (warp == 0) {
    const int w = lane >> 1, which = lane & 1;
    const bool head = w < C::NW && sh.seg_b[w][which] >= 0 && (sh.seg_lo[w][which] >= t0 + w * part || w == 0);
    const uint32_t heads = __ballot_sync(0xffffffffu, head);
    if (head) sh.chain_s[__popc(heads & ((1u << lane) - 1u))] = lane;
    if (lane == 0) sh.chains_s = __popc(heads);
  }
  __syncthreads();
  for (int y = tid; y < sh.chains_s * C::F4; y += C::THREADS) {
    const int x = y % C::F4, w = sh.chain_s[y / C::F4] >> 1, which = sh.chain_s[y / C::F4] & 1;
    const int lo = sh.seg_lo[w][which], hi = sh.seg_hi[w][which];
    const int to = ((hi < t1 ? hi : t1) - t0 + part - 1) / part;
    const int mlx = C::F4 + x / (32 * C::MM) * 32 + (x & 31);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f), ml = make_float4(kNoMax, kNoMax, 0.0f, 0.0f);
    // All but the last warp's segment are those warps' last ones, in the rings;
    // the last warp's, or a single one, may be a first one, in memory.  First
    // the largest maxima, then the sums.
    const bool far = to - 1 == w ? which == 0 : sh.seg_b[to - 1][0] >= 0 && sh.seg_lo[to - 1][0] == lo;
    const int near_to = far ? to - 1 : to;
    const float4* mem = reinterpret_cast<const float4*>(a.partials + (2 * kAttnMaxCtas + cta * C::NW + to - 1) * (int64_t)C::SLOT);
    const float4* slots = reinterpret_cast<const float4*>(dec_smem);
    const int stride = ring_bytes / 16;
    float4 far_o, far_ml;
    if (far) {
      far_o = mem[x];
      far_ml = mem[mlx];
      ml.x = far_ml.x;
      ml.y = far_ml.y;
    }
#pragma unroll 4
    for (int i = w; i < near_to; ++i) {
      const float2 m2 = *reinterpret_cast<const float2*>(slots + i * stride + mlx);
      ml.x = fmaxf(ml.x, m2.x);
      ml.y = fmaxf(ml.y, m2.y);
    }
#pragma unroll 4
    for (int i = w; i < near_to; ++i) dec_join(o, ml, slots[i * stride + x], slots[i * stride + mlx]);
    if (far) dec_join(o, ml, far_o, far_ml);
    if (lo >= t0 && hi <= t1) {
      const DecReq rq = request(sh.seg_b[w][which]);
      dec_write_part<C>(a, rq, sh.seg_h[w][which], x, o, ml);
    } else {
      float4* slot = reinterpret_cast<float4*>(a.partials + (2 * cta + (lo > t0 ? 1 : 0)) * (int64_t)C::SLOT);
      slot[x] = o;
      if (x / 32 % C::MM == 0) slot[mlx] = ml;
    }
  }
  if (chunk == 0) return;

  // Joining over CTAs: at most two items, the one that the CTA's first unit is
  // part of and the one that its last is part of.  Where the threads are more
  // than a result's float4s, each group of threads adds some of the CTAs.
  constexpr int PAR = C::THREADS > C::F4 ? C::THREADS / C::F4 : 1;
  // (One thread arrives for the CTA: the barrier orders the others' writes
  // before its fence.)
  auto crossing = [&](int side, DecPlace& p, DecReq& rq, int& lo) {
    const int ref = side == 0 ? t0 : t1 - 1;
    p = dec_find(a, pre, ref);
    rq = request(p.b);
    lo = ref - p.u;
    const int hi = lo + rq.units;
    // (not an item that lies in the CTA, or whose cost alone reaches into it,
    // or that side 0 has seen)
    return !((lo >= t0 && hi <= t1) || hi <= t0 || (side == 1 && lo <= t0));
  };
  __syncthreads();
  if (tid < 2) {
    DecPlace p;
    DecReq rq;
    int lo;
    bool last = false;
    if (crossing(tid, p, rq, lo)) {
      const int c0 = lo / chunk, c1 = (lo + rq.units - 1) / chunk;
      __threadfence();
      last = atomicAdd(&a.counters[c0], 1u) == (uint32_t)(c1 - c0);
      if (last) {
        a.counters[c0] = 0;
        __threadfence();
        sh.cross_s[tid] = DecCross{c0, c1, lo - c0 * chunk, p.h, rq};
      }
    }
    sh.last_s[tid] = last;
  }
  __syncthreads();
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    if (!sh.last_s[side]) continue;
    __syncthreads();  // (side 0's shares are read)
    const DecCross cr = sh.cross_s[side];
    const int c0 = cr.c0, c1 = cr.c1;
    const DecReq rq = cr.r;
    float4* share = reinterpret_cast<float4*>(dec_smem);  // [PAR][F4][2], PAR * F4 <= THREADS
#pragma unroll 1
    for (int x = tid % C::F4, k = tid / C::F4; x < C::F4 && k < PAR; x += C::THREADS) {
      const int mlx = C::F4 + x / (32 * C::MM) * 32 + (x & 31);
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f), ml = make_float4(kNoMax, kNoMax, 0.0f, 0.0f);
      // eight at once, as their latency is what this costs
#pragma unroll 1
      for (int i0 = c0 + k; i0 <= c1; i0 += 8 * PAR) {
        float4 o2[8], ml2[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const int i = i0 + y * PAR;
          ml2[y] = make_float4(kNoMax, kNoMax, 0.0f, 0.0f);
          o2[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (i <= c1) {
            // (the second of a CTA's two slots only where the item began within it)
            const float4* slot = reinterpret_cast<const float4*>(
                a.partials + (2 * i + (i == c0 && cr.into > 0 ? 1 : 0)) * (int64_t)C::SLOT);
            ml2[y] = __ldcg(slot + mlx);
            o2[y] = __ldcg(slot + x);
          }
        }
        const float4 old = ml;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          ml.x = fmaxf(ml.x, ml2[y].x);
          ml.y = fmaxf(ml.y, ml2[y].y);
        }
        const float4 o1 = o;
        o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        ml.z = ml.w = 0.0f;
        dec_join(o, ml, o1, old);
#pragma unroll
        for (int y = 0; y < 8; ++y) dec_join(o, ml, o2[y], ml2[y]);
      }
      if (PAR == 1) {
        dec_write_part<C>(a, rq, cr.h, x, o, ml);
      } else {
        share[(k * C::F4 + x) * 2] = o;
        share[(k * C::F4 + x) * 2 + 1] = ml;
      }
    }
    if (PAR > 1) {
      __syncthreads();
      if (tid < C::F4) {
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f), ml = make_float4(kNoMax, kNoMax, 0.0f, 0.0f);
#pragma unroll
        for (int k = 0; k < PAR; ++k) {
          const float4 m2 = share[(k * C::F4 + tid) * 2 + 1];
          ml.x = fmaxf(ml.x, m2.x);
          ml.y = fmaxf(ml.y, m2.y);
        }
#pragma unroll
        for (int k = 0; k < PAR; ++k)
          dec_join(o, ml, share[(k * C::F4 + tid) * 2], share[(k * C::F4 + tid) * 2 + 1]);
        dec_write_part<C>(a, rq, cr.h, tid, o, ml);
      }
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) kv4_decode_kernel(const __grid_constant__ AttnArgs a, int stages,
                                                                   int cached, int min_units) {
  extern __shared__ __align__(128) uint8_t dec_smem[];
  __shared__ uint64_t bars[C::NW][C::MAX_STAGES];
  __shared__ int scan_s[C::NW];
  __shared__ int max_s, over_s;
  __shared__ DecShared<C> sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int ring_bytes = stages * 2 * C::TILE;
  uint8_t* ring = dec_smem + warp * ring_bytes;
  uint8_t* q_next = dec_smem + C::NW * ring_bytes + warp * C::QROW;
  uint32_t* q_s = reinterpret_cast<uint32_t*>(dec_smem + C::NW * (ring_bytes + C::QROW) + warp * C::QBYTES) + lane;
  int32_t* pre = reinterpret_cast<int32_t*>(dec_smem + C::NW * (ring_bytes + C::QROW + C::QBYTES));
  const int cta = blockIdx.x, n_ctas = gridDim.x;
  // the requests' row starts and lengths, in shared memory where there is room
  int32_t* const copy = pre + a.B + 1;
  const int32_t* const starts = cached ? copy : a.row_start;
  const int32_t* const seqs = cached ? copy + a.B + 1 : a.seq_len;

  if (lane < stages) mbar_init(&bars[warp][lane], 1);
  if (lane < 2) sh.seg_b[warp][lane] = -1;
  if (tid == 0) max_s = over_s = 0;
  fence_barrier_init();
  // (what the kernel before wrote is read from here on)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  // work of one head, summed over the requests
  uint32_t bad = 0;
  {
    const int per = (a.B + C::THREADS - 1) / C::THREADS;
    int sum = 0, most = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= a.B) break;
      const int start = a.row_start[b], end = a.row_start[b + 1], seq = a.seq_len[b];
      if (cached) {
        copy[b] = start;
        if (b == a.B - 1) copy[a.B] = end;
        copy[a.B + 1 + b] = seq;
      }
      const int units = dec_request(a, start, end, seq, C::ROWS, bad).units;
      pre[b] = units ? units + kItemCost : 0;
      sum += pre[b];
      most = most > units ? most : units;
    }
    if (bad) over_s = 1;
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += u;
    }
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 31) scan_s[warp] = inc;
    if (lane == 0) atomicMax(&max_s, most);
    __syncthreads();
    int base = inc - sum;
    for (int w = 0; w < warp; ++w) base += scan_s[w];
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= a.B) break;
      const int t = pre[b];
      pre[b] = base;
      base += t;
    }
    if (tid == C::THREADS - 1) pre[a.B] = base;
  }
  __syncthreads();
  if (cta == 0 && bad) set_error(a.err, bad);
  // rows that no request covers, and requests that are refused
  uint16_t* const out = reinterpret_cast<uint16_t*>(a.out);
  const int first_row = a.B > 0 ? starts[0] : a.n, last_row = a.B > 0 ? starts[a.B] : a.n;
  if (first_row > 0 || last_row < a.n || over_s) {
#pragma unroll 1
    for (int b = over_s ? -1 : a.B - 1; b <= a.B; ++b) {
      int lo, hi;
      if (b < 0 || (b == a.B - 1 && !over_s)) {
        lo = 0;
        hi = first_row;
      } else if (b == a.B) {
        lo = last_row;
        hi = a.n;
      } else {
        if (pre[b + 1] != pre[b]) continue;
        lo = starts[b];
        hi = starts[b + 1];
      }
      zero_rows<C>(out, a.ld_out, a.q_heads, a.lse, lo < 0 ? 0 : lo, hi < a.n ? hi : a.n, cta, n_ctas);
    }
  }

  // this CTA's range
  const int total = pre[a.B] * a.heads;
  int t0, t1, chunk;
  if (a.B * a.heads <= n_ctas && max_s <= min_units) {  // a CTA a (request, head)
    chunk = 0;
    t0 = t1 = total;
    const int b = cta / a.heads;
    if (b < a.B) {
      const int cost = pre[b + 1] - pre[b];
      t0 = pre[b] * a.heads + (cta - b * a.heads) * cost;
      t1 = t0 + cost - (cost ? kItemCost : 0);
    }
  } else {
    chunk = (total + n_ctas - 1) / n_ctas;
    if (chunk < C::NW) chunk = C::NW;
    t0 = (int64_t)cta * chunk < total ? cta * chunk : total;
    t1 = total - t0 < chunk ? total : t0 + chunk;
  }
  if (t0 >= t1) return;
  const int part = (t1 - t0 + C::NW - 1) / C::NW;
  const int w0 = t0 + warp * part < t1 ? t0 + warp * part : t1;
  const int w1 = w0 + part < t1 ? w0 + part : t1;

  auto find = [&](int f) { return dec_find(a, pre, f); };
  auto next_item = [&](DecPlace& p) {  // (there is one)
    p.u = 0;
    if (++p.h < a.heads) return;
    p.h = 0;
    do ++p.b; while (pre[p.b + 1] == pre[p.b]);
  };

  uint32_t unused = 0;
  auto request = [&](int b) { return dec_request(a, starts[b], starts[b + 1], seqs[b], C::ROWS, unused); };
  DecState<C> st;
  int f = w0;
  DecPlace at = {0, 0, 0};
  DecReq r = {};
  if (f < w1) {
    at = find(f);
    r = request(at.b);
    if (at.u >= r.units) {  // the part begins in the cost of an item's end
      f += r.units + kItemCost - at.u;
      if (f < w1) {
        next_item(at);
        r = request(at.b);
      }
    }
  }
  if (f < w1) {
    // q of an item to shared memory: rows of D values
    auto fetch_q = [&](const DecReq& rq, int h) {
#pragma unroll
      for (int i = 0; i < C::QROW / 512; ++i) {  // (where q's operands stay in registers)
        const int x = i * 32 + lane, rr = x / (C::D / 8), d8 = x % (C::D / 8), j = div_group(a, rr);
        if (rr < rq.rows)
          cp_async16(q_next + x * 16, reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(rq.row0 + j) * a.ld_q +
                                          (h * a.group + rr - j * a.group) * C::D + d8 * 8);
      }
    };
    fetch_q(r, at.h);
    // the producer's place; the addresses of its next 32 tiles, one a lane
    DecPlace pp = at;
    DecReq pr = r;
    int pf = f, pblk = 0;
    const uint8_t* src = nullptr;
    uint32_t there = 0;  // which of the 32 are read
    bool fresh = true;
    uint32_t phase = 0, have = 0;  // parities of the stages' barriers; the tiles of them that are read, two bits each
    const int tpp = a.page_size / kKvTile;
    auto issue = [&](int stage) {  // the next unit of the part into a stage
      if (pf >= w1) return;
      if (fresh || pp.u - pblk == 16) {
        pblk = pp.u;
        fresh = false;
        const int t = pr.tile0 + 2 * pp.u + lane;
        src = nullptr;
        if (2 * pp.u + lane < 2 * pr.units && t * kKvTile < pr.seq) {
          const int nth = page_of_tile(a, t), page = a.table[(int64_t)pp.b * a.ld_table + nth];
          if (page >= 0 && page < a.num_pages)
            src = a.pages + (((int64_t)page * a.heads + pp.h) * tpp + (t - nth * tpp)) * C::TILE;
          else if (pf + (lane >> 1) < w1)  // (reported by the warp that would read it)
            set_error(a.err, LORA_DEV_ERR_PAGE);
        }
        there = __ballot_sync(0xffffffffu, src != nullptr);
      }
      const int k = 2 * (pp.u - pblk);
      const uint32_t got = (there >> k) & 3u;
      if (got && lane == k) mbar_arrive_expect_tx(&bars[warp][stage], (got == 3u ? 2 : 1) * C::TILE);
      __syncwarp();
      if (lane >> 1 == k >> 1 && src)
        bulk_g2s(ring + (stage * 2 + (lane & 1)) * C::TILE, src, C::TILE, &bars[warp][stage]);
      have |= got << (2 * stage);
      ++pf;
      if (++pp.u == pr.units) {
        pf += kItemCost;
        fresh = true;
        if (pf < w1) {
          next_item(pp);
          pr = request(pp.b);
        }
      }
    };
    int stage = 0;
#pragma unroll 1
    for (; stage < stages; ++stage) issue(stage);
    stage = 0;

    while (f < w1) {
      const int item0 = f - at.u, item1 = item0 + r.units;
      const int u_end = item1 < w1 ? r.units : w1 - item0;
      // q of the item: the lane's row g of each column tile, dims of its c
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      uint32_t qf[C::QSMEM ? 1 : C::NT][C::QSMEM ? 1 : C::QREGS];
      float qa[C::NT][2], qb[C::NT][C::G][2], thr[C::NT][2];  // of the lane's columns
#pragma unroll
      for (int n = 0; n < C::NT; ++n) {
        const int rr = n * 8 + g, j = div_group(a, rr);
        uint4 raw[C::G][2];
        float top = 0.0f, sum[C::G];
#pragma unroll
        for (int q = 0; q < C::G; ++q) {
          sum[q] = 0.0f;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            raw[q][x] = make_uint4(0, 0, 0, 0);
            if (rr < r.rows) {
              if (C::QSMEM)
                raw[q][x] = ldg_nc_v4(reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(r.row0 + j) * a.ld_q +
                                      (at.h * a.group + rr - j * a.group) * C::D + q * 64 + c * 16 + x * 8);
              else
                raw[q][x] = *reinterpret_cast<const uint4*>(q_next + (rr * C::D + q * 64 + c * 16 + x * 8) * 2);
            }
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[q][x]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = unpack2<C::BF16>(w[i]);
              top = fmaxf(top, fmaxf(fabsf(v.x), fabsf(v.y)));
              sum[q] += v.x + v.y;
            }
          }
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
          for (int q = 0; q < C::G; ++q) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], d);
        }
        // q 2^(14 - e) with 2^e <= top < 2^(e + 1) is at most 2^15; the
        // scale's sign goes with q, so that a larger product is a larger score
        int e = (int)((__float_as_uint(top) >> 23) & 255u) - 127;
        e = e < -100 ? -100 : e;
        const float mul = a.scale_log2 < 0.0f ? -pow2i(14 - e) : pow2i(14 - e);
#pragma unroll
        for (int q = 0; q < C::G; ++q)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[q][y]);
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = unpack2<C::BF16>(w[i]);
              x[2 * i] = v.x * mul;
              x[2 * i + 1] = v.y * mul;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float k = i % 2 ? 0.0625f : 1.0f;
              const uint32_t v = half2_bits(x[i] * k, x[4 + i] * k);
              const int to = (q * 2 + y) * 4 + i;
              if (C::QSMEM)
                q_s[(n * C::QREGS + to) * 32] = v;
              else
                qf[C::QSMEM ? 0 : n][C::QSMEM ? 0 : to] = v;
            }
          }
        const float fa = fabsf(a.scale_log2) * pow2i(e) * 1024.0f;  // 2^24 / 2^14
        const float fb = mul * 5.9604644775390625e-8f;              // 2^-24, as the codes have
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // the column 2 c + k is lane group 2 c + k's row
          qa[n][k] = __shfl_sync(0xffffffffu, fa, (2 * c + k) * 4);
          thr[n][k] = -INFINITY;
#pragma unroll
          for (int q = 0; q < C::G; ++q)
            qb[n][q][k] = __shfl_sync(0xffffffffu, sum[q] * fb, (2 * c + k) * 4);
        }
      }
      __syncwarp();
      // the item after this one
      const int f_next = item1 + kItemCost;
      if (f_next < w1) {
        DecPlace nx = at;
        next_item(nx);
        fetch_q(request(nx.b), nx.h);
      }
      dec_reset(st);
      // every row sees the tokens [see0, see1)
      const int pos1 = r.pos0 + div_group(a, r.rows - 1);
      const int see1 = r.pos0 + 1 < r.seq ? r.pos0 + 1 : r.seq;
      const int see0 = a.window > 0 && pos1 + 1 - a.window > 0 ? pos1 + 1 - a.window : 0;

#pragma unroll 1
      for (int u = at.u; u < u_end; ++u) {
        const uint32_t got = (have >> (2 * stage)) & 3u;
        if (got) {
          if (!__all_sync(0xffffffffu,
                          mbar_wait_soon(&bars[warp][stage], (phase >> stage) & 1u, a.wait_ns))) {
            // given up: the copies in flight still write to this CTA's memory,
            // so they are waited for; the rest of the part is not read
            if (lane == 0) {
              set_error(a.err, LORA_DEV_ERR_TIMEOUT);
              for (int x = 0; x < stages; ++x)
                if ((have >> (2 * x)) & 3u) mbar_wait_soon(&bars[warp][x], (phase >> x) & 1u, kWaitLimitNs);
            }
            __syncwarp();
            have = 0;
            pf = w1;
            continue;
          }
          phase ^= 1u << stage;
          have &= ~(3u << (2 * stage));
          const int tok0 = (r.tile0 + 2 * u) * kKvTile;
          uint8_t* unit = ring + stage * 2 * C::TILE;
          const bool edge = got != 3u || tok0 < see0 || tok0 + C::UNIT > see1;
          dec_unit<C>(a, r, st, unit, tok0, got, edge, pos1, q_s, qf, qa, qb, thr, lane);
          __syncwarp();
        }
        issue(stage);
        stage = stage + 1 == stages ? 0 : stage + 1;
      }
      dec_finish(st, qa, thr);
      if (item0 >= w0 && item1 <= w1) {
        dec_write(a, request(at.b), at.h, st, lane);
      } else {
        // a part of an item: the warp's first goes to memory, where its ring
        // is still in use; its last to the ring, which has served
        const bool last = f_next >= w1;
        if (lane == 0) {
          sh.seg_b[warp][last] = at.b;
          sh.seg_h[warp][last] = at.h;
          sh.seg_lo[warp][last] = item0;
          sh.seg_hi[warp][last] = item1;
        }
        dec_save(st, last ? reinterpret_cast<float*>(ring)
                          : a.partials + (2 * kAttnMaxCtas + cta * C::NW + warp) * (int64_t)C::SLOT, lane);
      }
      f = f_next;
      if (f < w1) {
        next_item(at);
        r = request(at.b);
      }
    }
  }
  __syncthreads();

  dec_join_all<C>(a, sh, dec_smem, ring_bytes, starts, seqs, pre, t0, t1, part, chunk);
}

}  // namespace lora
