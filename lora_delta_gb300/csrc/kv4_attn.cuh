// Attention over the 4-bit key/value cache for few query rows per request and
// key/value head (single tokens, a few tokens): the cache is read once and
// codes go from shared memory into matrix-instruction operands with one AND.
//
// Per 16-token tile and (request, head), with R = 8 NT query rows as columns:
//   S^T = K Q^T    A = codes of 16 tokens x 16 dims, B = q of 16 dims x 8 rows
//   O^T = V^T P^T  A = codes of 16 dims x 16 tokens, B = p of 16 tokens x 8 rows
// A code c in bits 0-3 of a 16-bit half is the f16 subnormal c 2^-24 and in
// bits 4-7 c 2^-20.  Keys: the operand's odd code pairs are the latter, so q is
// laid out with 2^-4 on the dims they meet.  Values: the odd pairs are rows
// 8-15 of the product, which take 2^-4 at the end.  Scales and least values:
//   s_t,g sum_d q_d c_d + m_t,g sum_d q_d    per group g of 64 dims (float32)
//   sum_t (p_t s_t,g) c_t + sum_t p_t m_t,g  the first sum's weights in f16
// q is brought to f16 by a power of two of its row (exact: 8 or 11 significant
// bits), p s to f16 by a power of two of the largest s so far, with p <= 2^8
// of a running maximum that follows lazily: 11 bits where f16 is normal, down
// to 2^-21 of the largest weight.  Sums, maxima and the m terms are float32.
#pragma once

#include "kv4.cuh"

namespace lora {

constexpr int kAttnMaxReqs = 4096;

struct AttnArgs {
  void* out;
  const void* q;
  int64_t ld_out, ld_q;
  int n, q_heads, heads, group;  // group = q_heads / heads
  const uint8_t* pages;
  int64_t num_pages;
  int page_size;
  const int32_t* table;
  int64_t ld_table;
  int max_pages;
  const int32_t* row_start;
  const int32_t* seq_len;
  int B, max_q_len, window;
  float scale_log2;  // softmax scale * log2(e)
  float* lse;
  uint32_t* err;
  uint64_t wait_ns;
  uint32_t* counters;  // [kAttnMaxCtas], zero between calls
  float* partials;     // [kAttnMaxCtas][2] slots, then [kAttnMaxCtas * warps] slots
};

constexpr int kAttnMaxCtas = 256;
constexpr float kNoMax = -1e30f;  // running maximum before any token

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
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

template <int D_, bool BF16_, int NT_, int NW_, int STAGES_>
struct Dec {
  static constexpr int D = D_, NT = NT_, NW = NW_, STAGES = STAGES_;
  static constexpr bool BF16 = BF16_;
  static constexpr int G = D / 64, W = D < 128 ? D : 128, NP = D / W, WD = W / 32;
  static constexpr int MM = D / 16;  // matrix products of a tile's values
  static constexpr int TILE = kv4_tile_bytes(D), HALF = kv4_half_bytes(D);
  static constexpr int ROWS = 8 * NT;
  static constexpr int QREGS = D / 8;  // q operands of one column tile
  // operands of q stay in registers where there is room beside the sums
  static constexpr bool QSMEM = QREGS * NT > 32;
  static constexpr int SLOT = 32 * (MM * 4 + 4) * NT;  // floats of a partial result
  static constexpr int RING = STAGES * TILE > SLOT * 4 ? STAGES * TILE : SLOT * 4;
  static constexpr int QBYTES = QSMEM ? QREGS * NT * 32 * 4 : 0;
  static constexpr int THREADS = NW * 32;
  static constexpr size_t smem(int B) {
    return (size_t)NW * (RING + QBYTES) + (size_t)(B + 1) * 4 + 16;
  }
};

// Running state of one (request, head): O^T sums, the p m sums, denominators
// and maxima of the lane's columns (2 c and 2 c + 1 of each column tile).
template <class C>
struct DecState {
  float o[C::NT][C::MM][4];
  float z[C::NT][C::G][2];
  float l[C::NT][2], m[C::NT][2];
  int fexp;  // the f16 weights are p s 2^fexp
};

template <class C>
__device__ __forceinline__ void dec_reset(DecState<C>& st) {
#pragma unroll
  for (int n = 0; n < C::NT; ++n) {
#pragma unroll
    for (int i = 0; i < C::MM; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[n][i][j] = 0.0f;
#pragma unroll
    for (int g = 0; g < C::G; ++g) st.z[n][g][0] = st.z[n][g][1] = 0.0f;
    st.l[n][0] = st.l[n][1] = 0.0f;
    st.m[n][0] = st.m[n][1] = kNoMax;
  }
  st.fexp = 126;
}

// Sums over the lanes that share columns; o becomes the sum of p v in float32.
template <class C>
__device__ __forceinline__ void dec_finish(DecState<C>& st) {
  const float f0 = pow2i(-st.fexp < -126 ? -126 : -st.fexp) * 16777216.0f, f1 = f0 * 0.0625f;
#pragma unroll
  for (int n = 0; n < C::NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) st.l[n][e] += __shfl_xor_sync(0xffffffffu, st.l[n][e], d);
#pragma unroll
      for (int g = 0; g < C::G; ++g) {
        float z = st.z[n][g][e];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) z += __shfl_xor_sync(0xffffffffu, z, d);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          st.o[n][4 * g + i][e] = fmaf(st.o[n][4 * g + i][e], f0, z);
          st.o[n][4 * g + i][2 + e] = fmaf(st.o[n][4 * g + i][2 + e], f1, z);
        }
      }
    }
}

// A finished state to / added from a slot (float4s of the 32 lanes).
template <class C>
__device__ __forceinline__ void dec_save(const DecState<C>& st, float* slot, int lane) {
  float4* p = reinterpret_cast<float4*>(slot) + lane;
#pragma unroll
  for (int n = 0; n < C::NT; ++n) {
#pragma unroll
    for (int i = 0; i < C::MM; ++i)
      p[(n * C::MM + i) * 32] = make_float4(st.o[n][i][0], st.o[n][i][1], st.o[n][i][2], st.o[n][i][3]);
    p[(C::NT * C::MM + n) * 32] = make_float4(st.m[n][0], st.m[n][1], st.l[n][0], st.l[n][1]);
  }
}
template <class C>
__device__ __forceinline__ void dec_add(DecState<C>& st, const float* slot, int lane) {
  const float4* p = reinterpret_cast<const float4*>(slot) + lane;
#pragma unroll
  for (int n = 0; n < C::NT; ++n) {
    const float4 ml = p[(C::NT * C::MM + n) * 32];
    const float m0 = fmaxf(st.m[n][0], ml.x), m1 = fmaxf(st.m[n][1], ml.y);
    const float a0 = exp2_fast(st.m[n][0] - m0), a1 = exp2_fast(st.m[n][1] - m1);
    const float b0 = exp2_fast(ml.x - m0), b1 = exp2_fast(ml.y - m1);
    st.m[n][0] = m0;
    st.m[n][1] = m1;
    st.l[n][0] = st.l[n][0] * a0 + ml.z * b0;
    st.l[n][1] = st.l[n][1] * a1 + ml.w * b1;
#pragma unroll
    for (int i = 0; i < C::MM; ++i) {
      const float4 v = p[(n * C::MM + i) * 32];
      st.o[n][i][0] = st.o[n][i][0] * a0 + v.x * b0;
      st.o[n][i][1] = st.o[n][i][1] * a1 + v.y * b1;
      st.o[n][i][2] = st.o[n][i][2] * a0 + v.z * b0;
      st.o[n][i][3] = st.o[n][i][3] * a1 + v.w * b1;
    }
  }
}

// What a (request, head) is: its rows, and the tiles that they see.
struct DecReq {
  int row0, rows;     // first row of the batch; query rows (tokens * group)
  int pos0;           // position of the first row
  int seq;            // tokens that may be seen (clipped to the table)
  int tile0, tiles;   // first tile and number of tiles, 0 for a request without rows here
};

__device__ __forceinline__ DecReq dec_request(const AttnArgs& a, int b, int max_rows, uint32_t& bad) {
  DecReq r;
  const int start = a.row_start[b], end = a.row_start[b + 1];
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  const int seq = a.seq_len[b];
  r.row0 = start;
  r.rows = 0;
  r.pos0 = 0;
  r.seq = 0;
  r.tile0 = 0;
  r.tiles = 0;
  if (end <= start) return r;
  if (start < 0 || end > a.n || end - start > a.max_q_len) {
    bad |= LORA_DEV_ERR_LENGTH;
    return r;
  }
  const int64_t rows = (int64_t)(end - start) * a.group;
  if (rows > max_rows) return r;
  r.rows = (int)rows;
  if (seq < 0 || seq > cap) bad |= LORA_DEV_ERR_LENGTH;
  r.pos0 = seq - (end - start);
  r.seq = seq < 0 ? 0 : (seq > cap ? (int)cap : seq);
  const int first = a.window > 0 && r.pos0 + 1 - a.window > 0 ? r.pos0 + 1 - a.window : 0;
  r.tile0 = first / kKvTile;
  const int last = (r.seq + kKvTile - 1) / kKvTile;
  // (a request that sees nothing keeps one tile, all of it masked)
  r.tiles = last > r.tile0 ? last - r.tile0 : 1;
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
      const int j = rr / a.group, head = h * a.group + rr - j * a.group;
      const float l = st.l[n][e], inv = l != 0.0f ? 1.0f / l : 0.0f;
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

// Zeros to the rows of a range.
template <bool BF16, int D>
__device__ void zero_rows(const AttnArgs& a, int lo, int hi, int part, int parts) {
  const int per = a.q_heads * (D / 8);
  for (int64_t i = (int64_t)part * blockDim.x + threadIdx.x; i < (int64_t)(hi - lo) * per;
       i += (int64_t)parts * blockDim.x) {
    const int64_t row = lo + i / per;
    const int k = (int)(i % per);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + row * a.ld_out + k * 8) =
        make_uint4(0, 0, 0, 0);
    if (a.lse && k % (D / 8) == 0) a.lse[row * a.q_heads + k / (D / 8)] = -INFINITY;
  }
}

// The tiles of all (request, head)s, laid end to end, are shared out evenly:
// a CTA takes a contiguous range and its warps contiguous parts of that.  A
// warp streams its tiles through a ring of bulk copies of its own.  Where a
// (request, head) ends inside a warp's part it is written; what crosses parts
// is joined over the CTA's warps, and over CTAs by the last of them to arrive,
// in the order of the tiles (so results do not depend on the order of events).
template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) kv4_decode_kernel(const AttnArgs a, int min_tiles,
                                                                   int only) {
  extern __shared__ __align__(128) uint8_t dec_smem[];
  __shared__ uint64_t bars[C::NW][C::STAGES];
  __shared__ int scan_s[C::NW];
  __shared__ int max_s, over_s, last_s;
  __shared__ int seg_b[C::NW][2], seg_h[C::NW][2];  // partial results of the warps (-1: none)
  __shared__ int64_t seg_lo[C::NW][2], seg_hi[C::NW][2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  uint8_t* ring = dec_smem + warp * C::RING;
  uint32_t* q_s = reinterpret_cast<uint32_t*>(dec_smem + C::NW * C::RING + warp * C::QBYTES) + lane;
  int32_t* pre = reinterpret_cast<int32_t*>(dec_smem + C::NW * (C::RING + C::QBYTES));
  const int cta = blockIdx.x, n_ctas = gridDim.x;

  if (lane < C::STAGES) mbar_init(&bars[warp][lane], 1);
  if (tid == 0) max_s = over_s = 0;
  fence_barrier_init();
  __syncthreads();
  // tiles of one head, summed over the requests
  uint32_t bad = 0;
  {
    const int per = (a.B + C::THREADS - 1) / C::THREADS;
    int sum = 0, most = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= a.B) break;
      const DecReq r = dec_request(a, b, C::ROWS, bad);
      pre[b] = r.tiles;
      sum += r.tiles;
      most = most > r.tiles ? most : r.tiles;
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
  if (only) {  // rows that no request here covers
    const int r0 = a.B > 0 ? a.row_start[0] : 0, r1 = a.B > 0 ? a.row_start[a.B] : 0;
    if (r0 > 0) zero_rows<C::BF16, C::D>(a, 0, r0 < a.n ? r0 : a.n, cta, n_ctas);
    if (r1 < a.n) zero_rows<C::BF16, C::D>(a, r1 < 0 ? 0 : r1, a.n, cta, n_ctas);
    if (over_s)
      for (int b = 0; b < a.B; ++b)
        if (pre[b + 1] == pre[b]) {
          const int lo = a.row_start[b], hi = a.row_start[b + 1];
          zero_rows<C::BF16, C::D>(a, lo < 0 ? 0 : lo, hi < a.n ? hi : a.n, cta, n_ctas);
        }
  }

  // this CTA's range of tiles
  const int64_t total = (int64_t)pre[a.B] * a.heads;
  int64_t t0, t1, chunk;
  if (a.B * a.heads <= n_ctas && max_s <= min_tiles) {  // a CTA a (request, head)
    chunk = 0;
    t0 = t1 = total;
    const int b = cta / a.heads;
    if (b < a.B) {
      const int tiles = pre[b + 1] - pre[b];
      t0 = (int64_t)pre[b] * a.heads + (int64_t)(cta - b * a.heads) * tiles;
      t1 = t0 + tiles;
    }
  } else {
    chunk = (total + n_ctas - 1) / n_ctas;
    if (chunk < C::NW) chunk = C::NW;
    t0 = cta * chunk < total ? cta * chunk : total;
    t1 = t0 + chunk < total ? t0 + chunk : total;
  }
  if (t0 >= t1) return;
  const int part = (int)((t1 - t0 + C::NW - 1) / C::NW);
  const int64_t w0 = t0 + (int64_t)warp * part < t1 ? t0 + (int64_t)warp * part : t1;
  const int64_t w1 = w0 + part < t1 ? w0 + part : t1;

  float* my_first = a.partials + ((int64_t)2 * kAttnMaxCtas + (int64_t)cta * C::NW + warp) * C::SLOT;
  float* my_last = reinterpret_cast<float*>(ring);
  if (lane < 2) seg_b[warp][lane] = -1;
  __syncwarp();

  // the (request, head, tile) of a flat number; the request's first tile in pre
  auto find = [&](int64_t f, int& b, int& h, int& tile) {
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if ((int64_t)pre[mid] * a.heads <= f) lo = mid; else hi = mid;
    }
    b = lo;
    const int tiles = pre[b + 1] - pre[b];
    const int64_t rest = f - (int64_t)pre[b] * a.heads;
    h = (int)(rest / tiles);
    tile = (int)(rest - (int64_t)h * tiles);
  };

  DecState<C> st;
  if (w0 < w1) {
    uint32_t unused = 0;
    // the producer's place: request pb, head ph, tile pt of it; pages of the
    // next 32 tiles are held one a lane
    int pb, ph, pt, pblk = 0;
    int64_t pf = w0;
    find(w0, pb, ph, pt);
    DecReq pr = dec_request(a, pb, C::ROWS, unused);
    int page_reg = -1;
    bool fresh = true;
    uint32_t held = 0, phase = 0;  // stages with a tile; their barriers' parities
    const int tpp = a.page_size / kKvTile;
    auto issue = [&](int stage) {  // the next tile of the part into a stage
      if (pf >= w1) return;
      if (fresh || pt - pblk == 32) {
        pblk = pt;
        fresh = false;
        const int t = pt + lane;
        page_reg = -1;
        if (t < pr.tiles && (pr.tile0 + t) * kKvTile < pr.seq) {
          page_reg = a.table[(int64_t)pb * a.ld_table + (pr.tile0 + t) / tpp];
          if (page_reg < 0 || page_reg >= a.num_pages) {
            // (reported by the warp that would read it)
            if (pf + lane < w1) set_error(a.err, LORA_DEV_ERR_PAGE);
            page_reg = -1;
          }
        }
      }
      const int page = __shfl_sync(0xffffffffu, page_reg, pt - pblk);
      if (page >= 0) {
        if (lane == 0) {
          const int64_t tile = ((int64_t)page * a.heads + ph) * tpp + (pr.tile0 + pt) % tpp;
          mbar_arrive_expect_tx(&bars[warp][stage], C::TILE);
          bulk_g2s(ring + stage * C::TILE, a.pages + tile * C::TILE, C::TILE, &bars[warp][stage]);
        }
        held |= 1u << stage;
      }
      ++pf;
      if (++pt == pr.tiles) {
        pt = 0;
        fresh = true;
        if (++ph == a.heads && pf < w1) {
          ph = 0;
          do ++pb; while (pre[pb + 1] == pre[pb]);
          pr = dec_request(a, pb, C::ROWS, unused);
        }
      }
    };
#pragma unroll 1
    for (int s = 0; s < C::STAGES; ++s) issue(s);

    int b, h, t;
    find(w0, b, h, t);
    int64_t f = w0;
    int stage = 0;
    while (f < w1) {
      const DecReq r = dec_request(a, b, C::ROWS, unused);
      const int64_t item0 = f - t, item1 = item0 + r.tiles;
      const int t_end = item1 < w1 ? r.tiles : (int)(w1 - item0);
      // q of the item: the lane's row g of each column tile, dims of its c
      uint32_t qf[C::QSMEM ? 1 : C::NT][C::QSMEM ? 1 : C::QREGS];
      float qa[C::NT][2], qb[C::NT][C::G][2];  // factors of the lane's columns
#pragma unroll
      for (int n = 0; n < C::NT; ++n) {
        const int rr = n * 8 + g;
        uint4 raw[C::G][2];
        float top = 0.0f, sum[C::G];
        const int j = rr / a.group;
        const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q) +
                             (int64_t)(r.row0 + j) * a.ld_q + (h * a.group + rr - j * a.group) * C::D;
#pragma unroll
        for (int q = 0; q < C::G; ++q) {
          sum[q] = 0.0f;
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            raw[q][u] = rr < r.rows ? ldg_nc_v4(qp + q * 64 + c * 16 + u * 8) : make_uint4(0, 0, 0, 0);
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[q][u]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 x = unpack2<C::BF16>(w[i]);
              top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
              sum[q] += x.x + x.y;
            }
          }
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
#pragma unroll
          for (int q = 0; q < C::G; ++q) sum[q] += __shfl_xor_sync(0xffffffffu, sum[q], d);
        }
        // q 2^(14 - e) with 2^e <= top < 2^(e + 1) is at most 2^15
        int e = (int)((__float_as_uint(top) >> 23) & 255u) - 127;
        e = e < -100 ? -100 : e;
        const float up = pow2i(14 - e);
#pragma unroll
        for (int q = 0; q < C::G; ++q)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[q][u]);
            float x[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 v = unpack2<C::BF16>(w[i]);
              x[2 * i] = v.x * up;
              x[2 * i + 1] = v.y * up;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float k = i % 2 ? 0.0625f : 1.0f;
              const uint32_t v = half2_bits(x[i] * k, x[4 + i] * k);
              const int at = (q * 2 + u) * 4 + i;
              if (C::QSMEM)
                q_s[(n * C::QREGS + at) * 32] = v;
              else
                qf[C::QSMEM ? 0 : n][C::QSMEM ? 0 : at] = v;
            }
          }
        const float fa = a.scale_log2 * pow2i(e) * 1024.0f;  // 2^24 / 2^14
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // the column 2 c + k is lane group 2 c + k's row
          qa[n][k] = __shfl_sync(0xffffffffu, fa, (2 * c + k) * 4);
#pragma unroll
          for (int q = 0; q < C::G; ++q)
            qb[n][q][k] = a.scale_log2 * __shfl_sync(0xffffffffu, sum[q], (2 * c + k) * 4);
        }
      }
      if (C::QSMEM) __syncwarp();
      dec_reset(st);

#pragma unroll 1
      for (; t < t_end; ++t) {
        if (held & (1u << stage)) {
          if (!__all_sync(0xffffffffu,
                          mbar_wait_bounded(&bars[warp][stage], (phase >> stage) & 1u, a.wait_ns))) {
            // given up: the copies in flight still write to this CTA's memory,
            // so they are waited for; the rest of the part is not read
            if (lane == 0) {
              set_error(a.err, LORA_DEV_ERR_TIMEOUT);
              for (int x = 0; x < C::STAGES; ++x)
                if (held & (1u << x)) mbar_wait_bounded(&bars[warp][x], (phase >> x) & 1u, kWaitLimitNs);
            }
            __syncwarp();
            held = 0;
            pf = w1;
            continue;
          }
          phase ^= 1u << stage;
          held &= ~(1u << stage);
          const uint8_t* tile = ring + stage * C::TILE;
          const int tok0 = (r.tile0 + t) * kKvTile;  // token of row 0
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
#pragma unroll
                for (int n = 0; n < C::NT; ++n) {
                  const int at = (p * C::WD + w) * 4 + 2 * u;
                  const uint32_t b0 = C::QSMEM ? q_s[(n * C::QREGS + at) * 32] : qf[C::QSMEM ? 0 : n][C::QSMEM ? 0 : at];
                  const uint32_t b1 = C::QSMEM ? q_s[(n * C::QREGS + at + 1) * 32] : qf[C::QSMEM ? 0 : n][C::QSMEM ? 0 : at + 1];
                  mma_f16(sc[n][(p * C::WD + w) / 2], a0, a1, a2, a3, b0, b1);
                }
              }
          }
          // scales and least values of tokens g and g + 8
          float2 ks[2][C::G], vs[2][C::G];
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < C::G; ++q) {
              const int at = 8 * C::D + ((g + 8 * u) * C::G + q) * 4;
              ks[u][q] = __half22float2(*reinterpret_cast<const __half2*>(tile + at));
              vs[u][q] = __half22float2(*reinterpret_cast<const __half2*>(tile + C::HALF + at));
            }
          // tokens past the last row's position, or before the first row's
          // window, are not read at all; rows in between are masked one by one
          const int pos1 = r.pos0 + (r.rows - 1) / a.group;
          const bool edge = tok0 + kKvTile > r.pos0 + 1 || tok0 + kKvTile > r.seq ||
                            (a.window > 0 && tok0 <= pos1 - a.window);
          float s[C::NT][4];
#pragma unroll
          for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int u = i >> 1, k = i & 1;
              float v = 0.0f, z = 0.0f;
#pragma unroll
              for (int q = 0; q < C::G; ++q) {
                v = fmaf(ks[u][q].x, sc[n][q][i], v);
                z = fmaf(ks[u][q].y, qb[n][q][k], z);
              }
              s[n][i] = fmaf(v, qa[n][k], z);
            }
          if (edge) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int tok = tok0 + g + 8 * u;
              // (a token that no row sees may hold anything)
              const bool any = tok < r.seq && tok <= pos1 &&
                               (a.window <= 0 || tok > r.pos0 - a.window);
#pragma unroll
              for (int q = 0; q < C::G; ++q)
                if (!any) vs[u][q] = make_float2(0.0f, 0.0f);
#pragma unroll
              for (int n = 0; n < C::NT; ++n)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int pos = r.pos0 + (n * 8 + 2 * c + k) / a.group;
                  if (!any || tok > pos || (a.window > 0 && tok <= pos - a.window))
                    s[n][2 * u + k] = -INFINITY;
                }
            }
          }
          // maxima: a new one only where a score is 2^8 above the old, or the
          // weights would leave f16
          bool up = false;
          float smax = 0.0f;
#pragma unroll
          for (int n = 0; n < C::NT; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k)
              up |= fmaxf(s[n][k], s[n][2 + k]) > st.m[n][k] + 8.0f;
#pragma unroll
          for (int q = 0; q < C::G; ++q)  // (a scale that is not finite poisons its own rows only)
            smax = fmaxf(smax, fmaxf(vs[0][q].x <= 65504.0f ? vs[0][q].x : 0.0f,
                                     vs[1][q].x <= 65504.0f ? vs[1][q].x : 0.0f));
          const float fcur = pow2i(st.fexp);
          up |= smax * fcur > 128.0f;
          if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) smax = fmaxf(smax, __shfl_xor_sync(0xffffffffu, smax, d));
            // 2^e <= smax < 2^(e + 1); s 2^f < 2^7 with f = 6 - e
            int fe = 6 - ((int)((__float_as_uint(smax) >> 23) & 255u) - 127);
            fe = fe < st.fexp ? fe : st.fexp;
            const float fold = pow2i(fe - st.fexp < -126 ? -126 : fe - st.fexp);
            st.fexp = fe;
#pragma unroll
            for (int n = 0; n < C::NT; ++n)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float top = fmaxf(s[n][k], s[n][2 + k]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float m1 = fmaxf(st.m[n][k], top), keep = exp2_fast(st.m[n][k] - m1);
                st.m[n][k] = m1;
                st.l[n][k] *= keep;
#pragma unroll
                for (int q = 0; q < C::G; ++q) st.z[n][q][k] *= keep;
                const float ko = keep * fold;
#pragma unroll
                for (int i = 0; i < C::MM; ++i) {
                  st.o[n][i][k] *= ko;
                  st.o[n][i][2 + k] *= ko;
                }
              }
          }
          const float f16f = pow2i(st.fexp);
          uint32_t pw[C::NT][C::G][2];  // weights of the values' products
#pragma unroll
          for (int n = 0; n < C::NT; ++n) {
            float pr4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pr4[i] = exp2_fast(s[n][i] - st.m[n][i & 1]);
            st.l[n][0] += pr4[0] + pr4[2];
            st.l[n][1] += pr4[1] + pr4[3];
#pragma unroll
            for (int q = 0; q < C::G; ++q) {
              const float f0 = vs[0][q].x * f16f, f1 = vs[1][q].x * f16f;
              float w[4] = {pr4[0] * f0, pr4[1] * f0, pr4[2] * f1, pr4[3] * f1};
              float y[4] = {pr4[0] * vs[0][q].y, pr4[1] * vs[0][q].y, pr4[2] * vs[1][q].y,
                            pr4[3] * vs[1][q].y};
              if (edge) {  // (0 x inf, where one row sees the token and another does not)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (pr4[i] == 0.0f) w[i] = y[i] = 0.0f;
              }
              st.z[n][q][0] += y[0] + y[2];
              st.z[n][q][1] += y[1] + y[3];
              pw[n][q][0] = transpose8(half2_bits(w[0], w[1]));
              pw[n][q][1] = transpose8(half2_bits(w[2], w[3]));
            }
          }
#pragma unroll
          for (int p = 0; p < C::NP; ++p) {
            uint32_t v0[C::WD], v1[C::WD];  // tokens 2 c, + 1 and 2 c + 8, + 9
            const uint8_t* vp = tile + C::HALF + p * 8 * C::W + g * (C::W / 2) + c * (C::W / 8);
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
                const uint32_t a0 = x0 & 0x000f000fu, a1 = x0 & 0x00f000f0u;
                const uint32_t a2 = x1 & 0x000f000fu, a3 = x1 & 0x00f000f0u;
                const int q = (p * C::WD + w) / 2;
#pragma unroll
                for (int n = 0; n < C::NT; ++n)
                  mma_f16(st.o[n][(p * C::WD + w) * 2 + u], a0, a1, a2, a3, pw[n][q][0], pw[n][q][1]);
              }
          }
          __syncwarp();
        }
        issue(stage);
        stage = stage + 1 == C::STAGES ? 0 : stage + 1;
      }
      f = item0 + t_end;
      dec_finish(st);
      if (item0 >= w0 && item1 <= w1) {
        dec_write(a, r, h, st, lane);
      } else {
        // a part of an item: the warp's first goes to memory, where its ring
        // is still in use; its last stays in registers until the end
        const int which = f >= w1 ? 1 : 0;
        if (lane == 0) {
          seg_b[warp][which] = b;
          seg_h[warp][which] = h;
          seg_lo[warp][which] = item0;
          seg_hi[warp][which] = item1;
        }
        if (which == 0) dec_save(st, my_first, lane);
      }
      t = 0;
      if (f < w1 && ++h == a.heads) {
        h = 0;
        do ++b; while (pre[b + 1] == pre[b]);
      }
    }
    __syncwarp();
    if (seg_b[warp][1] >= 0) dec_save(st, my_last, lane);
  }
  __syncthreads();

  // the CTA's parts of items: the warp that holds an item's first part here
  // adds the parts of the warps after it
  auto slot_of = [&](int w, int which) -> float* {
    return which ? reinterpret_cast<float*>(dec_smem + w * C::RING)
                 : a.partials + ((int64_t)2 * kAttnMaxCtas + (int64_t)cta * C::NW + w) * C::SLOT;
  };
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    const int b = seg_b[warp][which];
    if (b < 0) continue;
    const int64_t lo = seg_lo[warp][which], hi = seg_hi[warp][which];
    // the item's first part in this CTA is its own first tile, or the CTA's
    const int64_t from = which == 0 || lo < w0 ? w0 : lo;
    if (from > t0 && lo < from) continue;
    const DecReq r = dec_request(a, b, C::ROWS, bad);
    const int h = seg_h[warp][which];
    // this warp's own part, then those that follow
    dec_reset(st);
    dec_add(st, slot_of(warp, which), lane);
    for (int w = warp + 1; w < C::NW; ++w) {
      const int64_t at = t0 + (int64_t)w * part;
      if (at >= hi || at >= t1) break;
      dec_add(st, slot_of(w, seg_b[w][0] >= 0 && seg_lo[w][0] == lo ? 0 : 1), lane);
    }
    if (lo >= t0 && hi <= t1)
      dec_write(a, r, h, st, lane);
    else
      dec_save(st, a.partials + ((int64_t)2 * cta + (lo > t0 ? 1 : 0)) * C::SLOT, lane);
  }
  if (chunk == 0) return;

  // items that cross CTAs: at most two here, the one that the CTA's first tile
  // is part of and the one that its last is part of
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    int b, h, t;
    find(side == 0 ? t0 : t1 - 1, b, h, t);
    const int64_t lo = (side == 0 ? t0 : t1 - 1) - t, hi = lo + pre[b + 1] - pre[b];
    if (lo >= t0 && hi <= t1) continue;
    if (side == 1 && lo <= t0) continue;  // (the same item, seen on side 0)
    const int c0 = (int)(lo / chunk), c1 = (int)((hi - 1) / chunk);
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const uint32_t before = atomicAdd(&a.counters[c0], 1u);
      last_s = before == (uint32_t)(c1 - c0);
      if (last_s) a.counters[c0] = 0;
    }
    __syncthreads();
    if (!last_s) continue;
    __threadfence();
    if (warp == 0) {
      const DecReq r = dec_request(a, b, C::ROWS, bad);
      dec_reset(st);
      for (int i = c0; i <= c1; ++i)
        dec_add(st, a.partials + ((int64_t)2 * i + (lo > i * chunk ? 1 : 0)) * C::SLOT, lane);
      dec_write(a, r, h, st, lane);
    }
  }
}

}  // namespace lora
