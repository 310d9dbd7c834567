// Attention over the 4-bit key/value cache for many query rows per request and
// key/value head, on the tensor cores (tcgen05).
//
// An item is up to 256 query rows (a request's tokens x the heads that share a
// key/value head; 128 rows at head_dim 256) and the tokens that they see, in
// tiles of 128 (64).  Roles of a CTA, handing over through mbarriers:
//   load warp       bulk copies of the tile's packed 16-token blocks
//   guard warp      whether the tile's keys need two operands
//   8 expand warps  codes to f16 values s c + m in the operands' 128-byte
//                   swizzled layout, keys [token][dim], values [dim][token]
//   an MMA warp     for each row half in turn: O += P V with P read from tensor
//                   memory, then S = Q K^T of the next tile (128 x 128) in its
//                   place
//   4 softmax warps a row half: a thread a row; scores to weights in place of
//                   S, running maximum (followed lazily: O is scaled only when
//                   a row's maximum grew by 2^8), denominator, the final O / l
// The two row halves alternate, so the MMAs of one run while the other's
// weights are computed; tiles are expanded once for both.
// Keys and values are rounded to f16 (2^-12 relative) where tiles are expanded:
// two packed instructions a pair of codes.  Scaling S instead would cost one
// per score, group and query row.  Where that rounding could show, a tile's
// keys come in two operands, the second holding what the first lost, and S is the
// sum of two products; ordinary tiles do without.  A rounding is some 2^-12.3 |k|, so
// a score's error has the variance 2^-24.6 sum_d (scale q_d k_d)^2, at most the sum
// over groups of 64 dims of |scale q_g|^2 max k_g^2.  The guard bounds that for
// every row of the item and every token of the tile that some row sees: above 384
// the keys are two, so that no score is off by more than 2^-8 (one standard
// deviation), whatever the data; of normal keys with a few strong dims that bound is
// about 85 and the largest true sum about 8, an error of 2^-10.8.  (384 takes one
// such tile in 3000, and one in 200 at head_dim 64; 2^8 one in 140 and one in 23,
// and 271 us where a prompt's chunks have such a head for 247; 2^7 a quarter, 2^6 most:
// one prompt of 8192 tokens 720 and 990 us for 477; two operands always take 1057.)
// Queries are brought to f16 by a power of two of their row (exact), weights are
// 2^7 p with p <= 2^8.
//
// Bound: the chain of a half's softmax, its two products and the expansion that
// refills their operands; issue slots are 60% full, the tensor cores 40%.  bf16, 8
// heads of 128, 4 query heads each: one prompt of 8192 tokens 479 us (1148
// TFLOP/s), 32 prompts 110 us, chunks behind 16 thousand tokens 247 us (687 TFLOP/s).
// An item's first keys wait for the guard and so for its q, about 1 us an item (32
// prompts 104 us without); the MMA warp's first product ahead of the guard's word took
// 590 us of the first case, its loop no longer uniform.  Two places of 64 columns of
// scores a half, so that its softmax need not wait, took 650 us of the first where this
// took 531: with more roles at once a third of the warps waited for instructions; an
// MMA warp a half, or one each for S and O, took no less; four operands in flight 600
// us against 575.
#pragma once

#include "kv4_attn.cuh"
#include "tc.cuh"

namespace lora {

template <int D_, bool BF16_>
struct Pre {
  static constexpr int D = D_;
  static constexpr bool BF16 = BF16_;
  static constexpr int G = D / 64, W = D < 128 ? D : 128, NP = D / W, WD = W / 32;
  static constexpr int TILE = kv4_tile_bytes(D), HALF = kv4_half_bytes(D);
  static constexpr int MT = D == 256 ? 1 : 2;       // row halves of 128
  static constexpr int NKV = D == 256 ? 64 : 128;   // tokens of a tile
  static constexpr int TPK = NKV / kKvTile;
  static constexpr int ROWS = MT * 128;
  static constexpr int LPR = D / 8, RPL = 32 / LPR;  // lanes a row of q (16 bytes each), rows a load of a warp
  // blocks lie 16 bytes apart modulo 128, so that lanes reading the same place
  // of neighbouring blocks do not meet in a bank
  static constexpr int RSTRIDE = TILE + 16;
  static constexpr int RAW = TPK * RSTRIDE;
  static constexpr int KV = NKV * D * 2;            // an expanded operand
  static constexpr int KVB = D == 64 ? 6 : 3;       // expanded operands in flight
  static constexpr int Q = ROWS * D * 2;
  static constexpr int INFO = 8;                    // tiles described at once
  // Warps: guard 1, load 2, MMA 3, then softmax and expand from whole warpgroups on
  // (0 only helps at the start).
  static constexpr int SOFT_WARPS = 4 * MT, EXP_WARPS = 8;
  static constexpr int MMA_WARP = 3, LOAD_WARP = 2, GUARD_WARP = 1, SOFT_WARP = 4, EXP_WARP = SOFT_WARP + SOFT_WARPS;
  static constexpr int THREADS = (EXP_WARP + EXP_WARPS) * 32;
  // Registers a thread: 20 warps start with 96.  The expand warps give 24 each
  // to the softmax warps (8 x 72 + 8 x 120 = 16 x 96), which hold 32 words of
  // weights.  16 warps have 128 each anyway.
  static constexpr int REGS = MT == 2 ? 96 : 0, SOFT_REGS = 120, EXP_REGS = 72;
  static_assert(MT != 2 || EXP_WARPS * EXP_REGS + SOFT_WARPS * SOFT_REGS <= (EXP_WARPS + SOFT_WARPS) * REGS,
                "a split beyond the registers at launch would wait for ever");
  static constexpr size_t smem(int B) {
    return 1024 + (size_t)Q + KVB * KV + 2 * RAW + (size_t)(B + 1) * 4;
  }
};

constexpr float kKeyLimit = 384.0f;  // of the guard's bound, as above

// A row's frame: its weights and their sums are exp2((score - base) qa + off), in
// log2 units qa score.  base is 0 and off 7 less the row's maximum, as one product
// and sum a score is least, until the maximum passes 2^12, of which float32 keeps
// too little; then base is that score itself and off 7, so that its weight is 2^7
// at any size.  Kept as the largest score of the frame and `off`, which is
// kNoOffset for a row that takes a base and for one that has seen no token: it makes
// the common pass overflow, so that such rows take the other.
struct PreFrame {
  float top, off;
};
__device__ __forceinline__ float2 frame_terms(const PreFrame& f) {  // (base, off)
  const bool far = f.off == kNoOffset && f.top > -INFINITY;
  return make_float2(far ? f.top : 0.0f, far ? 7.0f : f.off);
}
// What a weight of frame `from` is in frame `to`.
__device__ __forceinline__ float frame_ratio(const PreFrame& from, const PreFrame& to, float qa) {
  const float2 a = frame_terms(from), b = frame_terms(to);
  return exp2_fast(fmaf(a.x - b.x, qa, b.y - a.y));
}

// An item: `rows` of the request's (token, head) rows.
struct PreItem {
  int b, h, rows;
  int tok0, rem0;       // the first row's token and place among the heads of its group
  int row0, pos0, seq;  // first row of the batch, its position, visible tokens
  int kv0, lo, hi, tiles;  // first token copied; tokens [lo, hi) are seen by some row
  int parts;  // of the item, this one among them if sp.part is below
};

__device__ __forceinline__ int pre_rows(const AttnArgs& a, int b, int min_rows, uint32_t& bad) {
  const int start = a.row_start[b], end = a.row_start[b + 1];
  if (end <= start) return 0;
  if (start < 0 || end > a.n || end - start > a.max_q_len) return 0;  // (reported by the decode kernel)
  if ((end - start) * a.group <= min_rows) return 0;
  if (a.seq_len[b] < 0 || a.seq_len[b] > a.cap) bad |= LORA_DEV_ERR_LENGTH;
  return (int)(end - start);
}

// SPLIT: where items are so few that half the CTAs or more had none, each item's
// tiles are shared out over `parts` CTAs, whose results the last of them joins (48
// rows over 65536 tokens: 939 -> 101 us; 512 tokens over 16384: 272 -> 162).  A
// kernel of its own, since what it adds costs the other 15%.
struct PreSplit {
  int parts, part;
};
constexpr int kPartTiles = 4;  // tiles of a part, at least (fewer gain less than the join takes)

// A CTA's items: one of each gridDim.x in turn, forwards and backwards
// alternately, since a prompt's items come by falling work; or a part of one.
template <bool SPLIT>
__device__ __forceinline__ int pre_nth(const PreSplit& sp, int round) {
  if (SPLIT && sp.parts > 1) return round == 0 ? blockIdx.x / sp.parts : INT32_MAX;
  return round * gridDim.x + (round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}

template <class C, bool SPLIT>
__device__ __forceinline__ PreItem pre_item(const AttnArgs& a, const int32_t* pre, const PreSplit& sp, int item) {
  PreItem it;
  const int total = pre[a.B];
  it.h = item % a.heads;
  const int rt = total - 1 - item / a.heads;  // a prompt's last rows see most: first
  int lo = 0, hi = a.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= rt) lo = mid; else hi = mid;
  }
  it.b = lo;
  it.row0 = a.row_start[lo];
  const int tokens = a.row_start[lo + 1] - it.row0;
  const int rows = tokens * a.group;
  const int seq = a.seq_len[lo];
  const int r0 = (rt - pre[lo]) * C::ROWS;
  it.rows = rows - r0 < C::ROWS ? rows - r0 : C::ROWS;
  it.tok0 = r0 / a.group;
  it.rem0 = r0 - it.tok0 * a.group;
  it.pos0 = seq - tokens;
  it.seq = seq < 0 ? 0 : (seq > a.cap ? a.cap : seq);
  const int pos_lo = it.pos0 + it.tok0, pos_hi = pos_lo + div_group(a, it.rem0 + it.rows - 1);
  it.lo = a.window > 0 && pos_lo + 1 - a.window > 0 ? pos_lo + 1 - a.window : 0;
  it.hi = pos_hi + 1 < it.seq ? pos_hi + 1 : it.seq;
  it.kv0 = it.lo / kKvTile * kKvTile;
  // (rows that see nothing keep one tile, all of it masked)
  it.tiles = it.hi > it.kv0 ? (it.hi - it.kv0 + C::NKV - 1) / C::NKV : 1;
  it.parts = 1;
  if (SPLIT && sp.parts > 1) {
    it.parts = it.tiles / kPartTiles;
    it.parts = it.parts < 1 ? 1 : (it.parts < sp.parts ? it.parts : sp.parts);
    const int t0 = sp.part * it.tiles / it.parts;
    it.tiles = (sp.part + 1) * it.tiles / it.parts - t0;
    it.kv0 += t0 * C::NKV;
  }
  return it;
}

// Four packed pairs of codes (two words' places) to values: bits 0-3 and 4-7
// of each half, exact integers first, then one rounding of s c + m.
__device__ __forceinline__ uint32_t code_lo(uint32_t w) {
  const uint32_t x = (w & 0x000f000fu) | 0x64006400u;  // 1024 + c
  const __half2 h = __hsub2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(1024.0f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t code_hi(uint32_t w) {
  const uint32_t x = (w & 0x00f000f0u) | 0x64006400u;  // 1024 + 16 c
  const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(0.0625f),
                            __float2half2_rn(-64.0f));
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t code_value(uint32_t c, __half2 s, __half2 m) {
  const __half2 h = __hfma2(*reinterpret_cast<const __half2*>(&c), s, m);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// Two float32 values worked on by one instruction.
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f32x2_split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <class C, bool SPLIT>
__global__ void __launch_bounds__(C::THREADS, 1) kv4_prefill_kernel(const AttnArgs a, int min_rows) {
  extern __shared__ uint8_t pre_smem_raw[];
  __shared__ uint64_t raw_full[2], raw_empty[2], kv_full[C::KVB], kv_empty[C::KVB];
  __shared__ uint64_t q_full[2], s_full[2], p_full[2], pv_done[2], two_full[2], drain_bar;
  __shared__ float size_s[C::SOFT_WARPS][C::G];    // of a warp's rows of q: the largest |scale q_g|^2
  __shared__ int exp_s[C::SOFT_WARPS][32];         // of q's rows: 2^e <= the largest |q|
  __shared__ uint32_t taddr_s;
  __shared__ uint32_t info_pages[C::INFO];             // blocks of a tile that were copied
  __shared__ uint32_t info_two[C::INFO];               // keys in two operands
  __shared__ uint32_t info_bad[C::INFO][C::G][C::NKV / 32];  // tokens whose values are not finite, by group
  __shared__ int scan_s[32];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (known to be the same in a warp)
  uint8_t* smem = pre_smem_raw + ((1024 - (smem_addr(pre_smem_raw) & 1023)) & 1023);
  uint8_t* q_s = smem;
  uint8_t* kv_s = smem + C::Q;
  uint8_t* raw_s = kv_s + C::KVB * C::KV;
  int32_t* pre = reinterpret_cast<int32_t*>(raw_s + 2 * C::RAW);

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], C::EXP_WARPS);
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
      mbar_init(&two_full[i], 1);
    }
    mbar_init(&drain_bar, 1);
    for (int i = 0; i < C::KVB; ++i) {
      mbar_init(&kv_full[i], C::EXP_WARPS);
      mbar_init(&kv_empty[i], 1);
    }
    fence_barrier_init();
  }
  // row tiles of the requests, summed
  uint32_t bad = 0;
  {
    const int per = (a.B + C::THREADS - 1) / C::THREADS;
    int sum = 0;
    for (int i = 0; i < per; ++i) {
      const int b = tid * per + i;
      if (b >= a.B) break;
      const int rows = pre_rows(a, b, min_rows, bad) * a.group;
      pre[b] = (rows + C::ROWS - 1) / C::ROWS;
      sum += pre[b];
    }
    int inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += u;
    }
    if (lane == 31) scan_s[warp] = inc;
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
  if (warp == C::MMA_WARP) tc::tmem_alloc(&taddr_s, 512);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (bad && blockIdx.x == 0) set_error(a.err, bad);
  const uint32_t tmem = taddr_s;
  int items = pre[a.B] * a.heads;
  PreSplit sp = {1, 0};
  if (SPLIT && items > 0 && 2 * items <= (int)gridDim.x) {
    sp.parts = gridDim.x / items;
    sp.part = blockIdx.x % sp.parts;
    if ((int)blockIdx.x >= items * sp.parts || sp.part >= pre_item<C, SPLIT>(a, pre, sp, blockIdx.x / sp.parts).parts) items = 0;
  }
  constexpr uint32_t kO = 256;  // first tensor-memory column of the sums
  bool ok = true;
  bool issued = false;  // (by the MMA warp)

  if (warp == C::LOAD_WARP) {
    // ------------------------------------------------------------------ load
    uint32_t n = 0;  // tiles so far
    auto prefetch = [&](int round) {  // an item's q on its way to L2
      const int i = pre_nth<SPLIT>(sp, round);
      if (i >= items) return;
      const PreItem it = pre_item<C, SPLIT>(a, pre, sp, i);
      for (int x = lane; x < it.rows * (C::D / 64); x += 32) {
        const int y = it.rem0 + x / (C::D / 64), t = div_group(a, y);
        asm volatile("prefetch.global.L2 [%0];" ::"l"(
            reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(it.row0 + it.tok0 + t) * a.ld_q +
            (it.h * a.group + y - t * a.group) * C::D + x % (C::D / 64) * 64));
      }
    };
    for (int round = 0, i; (i = pre_nth<SPLIT>(sp, round)) < items && ok; ++round) {
      const PreItem it = pre_item<C, SPLIT>(a, pre, sp, i);
      const int32_t* table = a.table + (int64_t)it.b * a.ld_table;
      for (int j = 0; j < it.tiles && ok; ++j, ++n) {
        const int st = n & 1;
        const int tok = it.kv0 + j * C::NKV + lane * kKvTile;
        int page = -1;
        if (lane < C::TPK && tok < it.hi) {
          page = table[page_of_tile(a, tok / kKvTile)];
          if (page < 0 || page >= a.num_pages) {
            set_error(a.err, LORA_DEV_ERR_PAGE);
            page = -1;
          }
        }
        if (n >= 2) ok = mbar_wait_soon(&raw_empty[st], ((n >> 1) - 1) & 1, a.wait_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t got = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) {
          info_pages[n % C::INFO] = got;
          for (int w = 0; w < C::G * C::NKV / 32; ++w) (&info_bad[n % C::INFO][0][0])[w] = 0;
          if (got)
            mbar_arrive_expect_tx(&raw_full[st], __popc(got) * C::TILE);
          else
            mbar_arrive(&raw_full[st]);
        }
        __syncwarp();
        if (page >= 0) {
          const int tpp = a.page_size / kKvTile, t = tok / kKvTile;
          const int64_t tile = ((int64_t)page * a.heads + it.h) * tpp + (t - page_of_tile(a, t) * tpp);
          bulk_g2s(raw_s + st * C::RAW + lane * C::RSTRIDE, a.pages + tile * C::TILE, C::TILE,
                   &raw_full[st]);
        }
        if (j == 0) prefetch(round + 1);  // (behind the first tile's copies)
      }
    }
    // (the copies still in flight write to this CTA's memory)
    for (uint32_t k = n >= 2 ? n - 2 : 0; k < n; ++k)
      if (!mbar_wait_soon(&raw_full[k & 1], (k >> 1) & 1, kWaitLimitNs)) ok = false;
  } else if (warp == C::GUARD_WARP) {
    // ----------------------------------------------------------------- guard
    uint32_t n = 0, q_ph = 0;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_soon(bar, parity, a.wait_ns));
    };
    for (int round = 0, i; (i = pre_nth<SPLIT>(sp, round)) < items && ok; ++round) {
      const PreItem it = pre_item<C, SPLIT>(a, pre, sp, i);
      const int mt = it.rows > 128 ? 2 : 1;
      float size[C::G];
      for (int j = 0; j < it.tiles && ok; ++j, ++n) {
        const int st = n & 1, tok0 = it.kv0 + j * C::NKV;
        wait(&raw_full[st], (n >> 1) & 1);
        if (!ok) break;
        const uint32_t pages = info_pages[n % C::INFO];
        float k2[C::NKV / 32][C::G];  // the largest k^2 of each group, of tokens that some row sees
#pragma unroll
        for (int x = 0; x < C::NKV / 32; ++x) {
          const int t = x * 32 + lane;
          const uint8_t* pairs = raw_s + st * C::RAW + (t / kKvTile) * C::RSTRIDE + 8 * C::D + (t % kKvTile) * C::G * 4;
          const bool use = ((pages >> (t / kKvTile)) & 1u) && tok0 + t >= it.lo && tok0 + t < it.hi;
#pragma unroll
          for (int q = 0; q < C::G; ++q) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(pairs + 4 * q));
            const float k = fmaxf(fabsf(f.y), fabsf(fmaf(15.0f, f.x, f.y)));
            k2[x][q] = use ? k * k : 0.0f;
          }
        }
        if (j == 0) {  // (as late as can be: the rows' warps load q after the last item's end)
          for (int m = 0; m < mt; ++m) {
            wait(&q_full[m], (q_ph >> m) & 1);
            q_ph ^= 1u << m;
          }
          if (!ok) break;
#pragma unroll
          for (int q = 0; q < C::G; ++q)
            size[q] = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < 4 * mt ? __float_as_uint(size_s[lane][q]) : 0u));
        }
        bool large = false;
#pragma unroll
        for (int x = 0; x < C::NKV / 32; ++x) {
          float sum = 0.0f;
#pragma unroll
          for (int q = 0; q < C::G; ++q) sum = fmaf(size[q], k2[x][q], sum);
          large |= !(sum <= kKeyLimit);  // (and what is not a number)
        }
        large = __any_sync(0xffffffffu, large);
        if (lane == 0) {
          info_two[n % C::INFO] = large;
          mbar_arrive(&two_full[st]);
        }
      }
    }
  } else if (warp == C::MMA_WARP) {
    // ------------------------------------------------------------------- MMA
    // The warp runs whole, so that descriptors stay in uniform registers; one
    // lane is elected at each product and commit.
    const uint32_t id_qk = tc::idesc_f16_f32(128, C::NKV), id_pv = tc::idesc_f16_f32(128, C::D);
    // (start addresses are in 16-byte units in a descriptor's low bits, and no
    // sum below carries out of them)
    const uint64_t q_desc = tc::sw128_desc(smem_addr(q_s)), kv_desc = tc::sw128_desc(smem_addr(kv_s));
    uint32_t k = 0, k_ph = 0, n = 0;  // place and parity of the next operand; tiles so far
    uint32_t q_ph = 0, p_ph = 0;      // a bit a half: parities of q_full and p_full
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait_soon(bar, parity, a.wait_ns));
    };
    auto take = [&]() -> uint32_t {  // waits for the next operand and returns its place
      wait(&kv_full[k], k_ph);
      const uint32_t x = k;
      k = k + 1 == C::KVB ? 0 : k + 1;
      k_ph ^= k == 0;
      return x;
    };
    auto commit = [&](uint64_t* bar) {
      if (tc::elect_one()) tc::mma_commit(bar);
    };
    for (int round = 0, i; (i = pre_nth<SPLIT>(sp, round)) < items && ok; ++round) {
      const PreItem it = pre_item<C, SPLIT>(a, pre, sp, i);
      const int mt = it.rows > 128 ? 2 : 1;
      // step -1: S of the first tile; step j: O of tile j, S of the next.  The
      // halves take turns, so that one's products run while the other's weights
      // are computed.
      for (int j = -1; j < it.tiles && ok; ++j) {
        const bool more = j + 1 < it.tiles;
        uint32_t v = 0, x = 0, y = 0;
        if (j >= 0) v = take();
        // (operands are waited for ahead of the weights: 573 -> 542 us)
        if (more) {  // the keys in operand x, and y where they are two
          x = y = take();
          if (ok && __shfl_sync(0xffffffffu, info_two[(n + (j >= 0)) % C::INFO], 0)) y = take();
        }
#pragma unroll 1
        for (int m = 0; m < mt; ++m) {
          const uint32_t t_s = tmem + m * 128, t_o = tmem + kO + m * 128;
          if (j < 0) {
            wait(&q_full[m], (q_ph >> m) & 1);
            q_ph ^= 1u << m;
          } else {
            wait(&p_full[m], (p_ph >> m) & 1);
            p_ph ^= 1u << m;
          }
          if (!ok) break;
          tc::fence_after_sync();
          issued = true;
          if (j >= 0) {
            const uint64_t vd = kv_desc + (uint64_t)(v * (C::KV / 16));
#pragma unroll
            for (int t = 0; t < C::NKV / 16; ++t)
              if (tc::elect_one())
                tc::mma_f16_ts(t_o, t_s + t * 8, vd + ((t / 4) * C::D * 128 + (t % 4) * 32) / 16, id_pv, t > 0 || j > 0);
            commit(&pv_done[m]);
            if (m == mt - 1) commit(&kv_empty[v]);
          }
          if (more) {
            const uint64_t qd = q_desc + (uint64_t)(m * 128 * C::D * 2 / 16);
#pragma unroll 1
            for (uint32_t add = 0, z = x;; add = 1, z = y) {
              const uint64_t kd = kv_desc + (uint64_t)(z * (C::KV / 16));
#pragma unroll
              for (int d = 0; d < C::D / 16; ++d)
                if (tc::elect_one())
                  tc::mma_bf16(t_s, qd + ((d / 4) * 16384 + (d % 4) * 32) / 16,
                               kd + ((d / 4) * C::NKV * 128 + (d % 4) * 32) / 16, id_qk, d > 0 || add);
              if (add || x == y) break;
            }
            commit(&s_full[m]);
            if (m == mt - 1) {
              commit(&kv_empty[x]);
              if (y != x) commit(&kv_empty[y]);
            }
          }
        }
        n += j >= 0;
      }
    }
  } else if (warp >= C::EXP_WARP) {
    // ---------------------------------------------------------------- expand
    if constexpr (C::REGS > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::EXP_REGS));
    const int et = tid - C::EXP_WARP * 32, ew = et >> 5;
    uint32_t n = 0, k = 0;  // tiles and operands so far
    auto wait_free = [&]() {
      if (k >= C::KVB)
        ok = ok && mbar_wait_soon(&kv_empty[k % C::KVB], (k / C::KVB - 1) & 1, a.wait_ns);
      ok = __all_sync(0xffffffffu, ok);
    };
    auto filled = [&]() {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&kv_full[k % C::KVB]);
      ++k;
    };
    for (int round = 0, i; (i = pre_nth<SPLIT>(sp, round)) < items && ok; ++round) {
      const PreItem it = pre_item<C, SPLIT>(a, pre, sp, i);
      const int pos_lo = it.pos0 + it.tok0, pos_hi = pos_lo + div_group(a, it.rem0 + it.rows - 1);
      for (int j = 0; j < it.tiles && ok; ++j, ++n) {
        const int st = n & 1, tok0 = it.kv0 + j * C::NKV;
        ok = __all_sync(0xffffffffu, mbar_wait_soon(&raw_full[st], (n >> 1) & 1, a.wait_ns));
        if (!ok) break;
        const uint32_t pages = info_pages[n % C::INFO];
        // tiles of which some row does not see some token
        const bool edge = tok0 + C::NKV > it.seq || tok0 + C::NKV > pos_lo + 1 ||
                          (a.window > 0 && tok0 <= pos_hi - a.window) || pages != (1u << C::TPK) - 1u;
        uint8_t* raw = raw_s + st * C::RAW;
        if (edge) {
          // Values' scales of tokens that no row sees may hold anything, and a
          // group's that is not finite would reach rows that do not see it: both
          // are set to 0, the latter noted for the softmax.  (Each warp does it
          // for what it reads, noting before it clears.)
          const int tb = C::NKV == 128 ? (ew >> 1) & 1 : 0;
#pragma unroll 1
          for (int t = tb * 64 + lane; t < tb * 64 + 64; t += 32) {
            uint32_t* sp = reinterpret_cast<uint32_t*>(raw + (t / kKvTile) * C::RSTRIDE + C::HALF + 8 * C::D) + (t % kKvTile) * C::G;
            const bool use = ((pages >> (t / kKvTile)) & 1u) && tok0 + t >= it.lo && tok0 + t < it.hi;
#pragma unroll
            for (int q = 0; q < C::G; ++q) {
              const bool odd = (sp[q] & 0x7c00u) == 0x7c00u || (sp[q] & 0x7c000000u) == 0x7c000000u;
              if (use && odd) atomicOr(&info_bad[n % C::INFO][q][t / 32], 1u << (t % 32));
              if (!use || odd) sp[q] = 0;
            }
          }
          fence_proxy_async_smem();  // (the block is next written by a bulk copy)
          __syncwarp();
        }
        wait_free();
        if (!ok) break;
        bool two;
        {
          uint8_t* kb = kv_s + (k % C::KVB) * C::KV;
#pragma unroll
          for (int s = 0; s < C::NKV * 4 * C::NP / (32 * C::EXP_WARPS); ++s) {
            const int u = et + 32 * C::EXP_WARPS * s, p = u / (C::NKV * 4), t = (u / 4) % C::NKV, c = u % 4;
            const uint8_t* tile = raw + (t / kKvTile) * C::RSTRIDE;
            const int tt = t % kKvTile;
            uint32_t w[C::WD];
            const uint8_t* kp = tile + p * 8 * C::W + tt * (C::W / 2) + c * (C::W / 8);
            if (C::WD == 4)
              *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(kp);
            else
              *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(kp);
#pragma unroll
            for (int q = 0; q < C::WD / 2; ++q) {
              const int gq = p * (C::WD / 2) + q;
              const __half2 sm = *reinterpret_cast<const __half2*>(tile + 8 * C::D + (tt * C::G + gq) * 4);
              const __half2 s2 = __low2half2(sm), m2 = __high2half2(sm);
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t v = w[2 * q + x], v8 = v >> 8;
                // dims 0 4 1 5 2 6 3 7 of the word, the order that q is laid out in
                const uint4 o = make_uint4(code_value(code_lo(v), s2, m2), code_value(code_hi(v), s2, m2),
                                           code_value(code_lo(v8), s2, m2), code_value(code_hi(v8), s2, m2));
                *reinterpret_cast<uint4*>(kb + gq * C::NKV * 128 + t * 128 + (((2 * c + x) ^ (t & 7)) << 4)) = o;
              }
            }
          }
          // (the MMA warp reads the guard's word too, by way of these keys)
          ok = __all_sync(0xffffffffu, mbar_wait_soon(&two_full[st], (n >> 1) & 1, a.wait_ns));
          if (!ok) break;
          two = info_two[n % C::INFO];
          filled();
        }
        wait_free();
        if (!ok) break;
        if (two) {  // what the keys' rounding left
          uint8_t* kb = kv_s + (k % C::KVB) * C::KV;
#pragma unroll 1
          for (int u = et; u < C::NKV * 4 * C::NP * C::WD; u += 32 * C::EXP_WARPS) {
            const int w = u % C::WD, c = u / C::WD % 4, t = u / (4 * C::WD) % C::NKV, p = u / (4 * C::WD * C::NKV);
            const int gq = p * (C::WD / 2) + w / 2, tt = t % kKvTile;
            const uint8_t* tile = raw + (t / kKvTile) * C::RSTRIDE;
            const uint32_t v = *reinterpret_cast<const uint32_t*>(tile + p * 8 * C::W + tt * (C::W / 2) + c * (C::W / 8) + w * 4);
            const __half2 sm = *reinterpret_cast<const __half2*>(tile + 8 * C::D + (tt * C::G + gq) * 4);
            const float2 f = __half22float2(sm);
            uint32_t o[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t code = x % 2 ? code_hi(x > 1 ? v >> 8 : v) : code_lo(x > 1 ? v >> 8 : v);
              const uint32_t val = code_value(code, __low2half2(sm), __high2half2(sm));
              const float2 cf = __half22float2(*reinterpret_cast<const __half2*>(&code));
              const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&val));
              o[x] = half2_bits(fmaf(f.x, cf.x, f.y) - vf.x, fmaf(f.x, cf.y, f.y) - vf.y);
            }
            *reinterpret_cast<uint4*>(kb + gq * C::NKV * 128 + t * 128 + (((2 * c + w % 2) ^ (t & 7)) << 4)) =
                make_uint4(o[0], o[1], o[2], o[3]);
          }
          filled();
          wait_free();
          if (!ok) break;
        }
        {
          uint8_t* vb = kv_s + (k % C::KVB) * C::KV;
          // a warp takes 64 tokens' half of the dims of every group's eighths: words
          // [x0, x0 + WH) of each lane place, all of one group where W is 128
          constexpr int WH = C::WD / 2;
          const int odd = ew & 1, tb = C::NKV == 128 ? (ew >> 1) & 1 : 0, p = C::NKV == 128 ? 0 : (ew >> 1) & 1;
          const int x0 = (ew >> 2) * WH, gq = p * (C::WD / 2) + x0 / 2;
          const int tile4 = lane & 3, u = (lane >> 2) & 1, g = 2 * (lane >> 3) + u, h = u ^ odd;
          const uint8_t* tile = raw + (tb * 4 + tile4) * C::RSTRIDE + C::HALF;
          const uint8_t* vp = tile + p * 8 * C::W + h * 4 * C::W + g * (C::W / 2) + x0 * 4;
          __half2 s2[4], m2[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            __half2 sm[2];
#pragma unroll
            for (int e = 0; e < 2; ++e)
              sm[e] = *reinterpret_cast<const __half2*>(tile + 8 * C::D + ((8 * h + 2 * c + e) * C::G + gq) * 4);
            s2[c] = __lows2half2(sm[0], sm[1]);
            m2[c] = __highs2half2(sm[0], sm[1]);
          }
          uint8_t* to = vb + tb * C::D * 128;
#pragma unroll 1
          for (int x = 0; x < WH; ++x) {
            uint32_t w[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) w[c] = *reinterpret_cast<const uint32_t*>(vp + c * (C::W / 8) + x * 4);
            const int d0 = gq * 64 + 8 * g + 4 * ((x0 + x) % 2);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              uint32_t o[4];
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t v = jj >= 2 ? w[c] >> 8 : w[c];
                o[c] = code_value(jj % 2 ? code_hi(v) : code_lo(v), s2[c], m2[c]);
              }
              const int d = d0 + jj;
              *reinterpret_cast<uint4*>(to + d * 128 + (((tile4 * 2 + h) ^ (d & 7)) << 4)) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
          filled();
          if (lane == 0) mbar_arrive(&raw_empty[st]);
        }
      }
    }
  } else if (warp >= C::SOFT_WARP) {
    // --------------------------------------------------------------- softmax
    if constexpr (C::REGS > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFT_REGS));
    const int m = (warp - C::SOFT_WARP) >> 2, wl = warp & 3, r_l = wl * 32 + lane;
    const uint32_t t_s = tmem + m * 128 + ((uint32_t)(wl * 32) << 16);
    const uint32_t t_o = tmem + kO + m * 128 + ((uint32_t)(wl * 32) << 16);
    uint32_t n = 0, n_t = 0;  // tiles of all items; tiles of this half
    // (a scale of 0 goes with q too, so that masked scores times qa stay -inf)
    const float sign = a.scale_log2 < 0.0f ? -1.0f : a.scale_log2 > 0.0f ? 1.0f : 0.0f;
    uint8_t* q_half = q_s + m * 128 * C::D * 2;
    // the place of 16 bytes of a row of q, and of out on its way to memory
    auto q_place = [&](int row, int chunk) {
      return reinterpret_cast<uint4*>(q_half + (chunk / 8) * 16384 + row * 128 + (((chunk % 8) ^ (row & 7)) << 4));
    };
    // (of a part: to be counted in, whatever happens, so that the count returns to 0)
    uint32_t* count = nullptr;
    int parts = 1;
    [[maybe_unused]] auto arrive = [&]() -> bool {  // whether all the others had
      bool last = false;
      if (lane == 0) {
        last = atomicAdd(count, 1u) == (uint32_t)parts - 1u;
        if (last) *count = 0;
      }
      count = nullptr;
      return __shfl_sync(0xffffffffu, last, 0);
    };
    for (int round = 0, i; (i = pre_nth<SPLIT>(sp, round)) < items && ok; ++round) {
      const PreItem it = pre_item<C, SPLIT>(a, pre, sp, i);
      if (SPLIT && it.parts > 1 && m * 128 < it.rows) {
        parts = it.parts;
        count = a.counters + i * C::SOFT_WARPS + (warp - C::SOFT_WARP);
      }
      if (m * 128 >= it.rows) {  // this half sits the item out
        n += it.tiles;
        continue;
      }
      const bool live = m * 128 + r_l < it.rows;
      const int in_item = it.rem0 + m * 128 + r_l, tok = div_group(a, in_item);  // (tokens from tok0)
      const int head = it.h * a.group + in_item - tok * a.group;
      // q of the warp's rows, 16 bytes a lane (earlier products with this
      // half's q are done), a batch of loads at once
      const int chunk = lane % C::LPR;
      constexpr int kBatch = C::LPR < 16 ? 8 : 16;
      float largest = 0.0f;  // |q_g|^2 of the lane's group of dims
#pragma unroll 1
      for (int y0 = 0; y0 < 32 / C::RPL; y0 += kBatch) {
        uint4 raw[kBatch];
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
          const int row = m * 128 + wl * 32 + (y0 + y) * C::RPL + lane / C::LPR;
          const int x = it.rem0 + row, t = div_group(a, x);
          raw[y] = row < it.rows ? ldg_nc_v4(reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(it.row0 + it.tok0 + t) * a.ld_q +
                                             (it.h * a.group + x - t * a.group) * C::D + chunk * 8)
                                 : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int y = 0; y < kBatch; ++y) {
          const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[y]);
          float f[8], top = 0.0f, sq = 0.0f;
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 z = unpack2<C::BF16>(w[x]);
            f[2 * x] = z.x;
            f[2 * x + 1] = z.y;
            top = fmaxf(top, fmaxf(fabsf(z.x), fabsf(z.y)));
            sq = fmaf(z.x, z.x, fmaf(z.y, z.y, sq));
          }
#pragma unroll
          for (int d = 1; d < 8; d <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
          largest = fmaxf(largest, sq);
#pragma unroll
          for (int d = 1; d < C::LPR; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          int e = (int)((__float_as_uint(top) >> 23) & 255u) - 127;
          e = e < -100 ? -100 : e;
          const float up = pow2i(14 - e) * sign;
          const int row = (y0 + y) * C::RPL + lane / C::LPR;
          if (chunk == 0) exp_s[warp - C::SOFT_WARP][row] = e;
          // (dims 0 4 1 5 2 6 3 7, as the keys lie)
          *q_place(wl * 32 + row, chunk) = make_uint4(half2_bits(f[0] * up, f[4] * up), half2_bits(f[1] * up, f[5] * up),
                                                      half2_bits(f[2] * up, f[6] * up), half2_bits(f[3] * up, f[7] * up));
        }
      }
#pragma unroll
      for (int d = C::LPR; d < 32; d <<= 1) largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, d));
      const float sc = a.scale_log2 * 0.69314718055994531f;
      if (lane < C::LPR && lane % 8 == 0) size_s[warp - C::SOFT_WARP][lane / 8] = largest * (sc * sc);
      fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[m]);
      const float qa = sign == 0.0f ? 1.0f : fabsf(a.scale_log2) * pow2i(exp_s[warp - C::SOFT_WARP][lane]) * (1.0f / 16384.0f);

      const int pos = it.pos0 + it.tok0 + tok;
      const int see_hi = live ? (pos + 1 < it.seq ? pos + 1 : it.seq) : -1;
      const int see_lo = a.window > 0 ? pos + 1 - a.window : 0;
      const int last = it.rows < m * 128 + 128 ? it.rows : m * 128 + 128;
      const int pos_lo = it.pos0 + it.tok0 + div_group(a, it.rem0 + m * 128);
      const int pos_hi = it.pos0 + it.tok0 + div_group(a, it.rem0 + last - 1);
      PreFrame fr = {-INFINITY, kNoOffset};
      float l = 0.0f;
      uint32_t lost = 0;  // groups of 64 dims of which the row has seen a value that is not finite
      auto spoil = [&](auto& v, int group) {
        if (__any_sync(0xffffffffu, lost)) {
          const float add = (lost >> group) & 1u ? __int_as_float(0x7fffffff) : 0.0f;
#pragma unroll
          for (float& x : v) x += add;
        }
      };
      for (int j = 0; j < it.tiles; ++j, ++n, ++n_t) {
        ok = __all_sync(0xffffffffu, mbar_wait_soon(&s_full[m], n_t & 1, a.wait_ns));
        if (!ok) break;
        tc::fence_after_sync();
        const int tok0 = it.kv0 + j * C::NKV;
        const uint32_t pages = info_pages[n % C::INFO];
        const bool edge = tok0 + C::NKV > it.seq || tok0 + C::NKV > pos_lo + 1 ||
                          (a.window > 0 && tok0 <= pos_hi - a.window) || pages != (1u << C::TPK) - 1u;
        // columns that the row sees, and the blocks of 16 that were not read
        const int c_lo = see_lo - tok0, c_hi = see_hi - tok0;
        auto seen32 = [&](int col) -> uint32_t {  // of the 32 columns from col
          const int lo = c_lo - col > 0 ? c_lo - col : 0, hi = c_hi - col < 32 ? c_hi - col : 32;
          uint32_t s = hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
          const uint32_t two_blocks = pages >> (col / kKvTile);
          if (!(two_blocks & 1u)) s &= 0xffff0000u;
          if (!(two_blocks & 2u)) s &= 0x0000ffffu;
          return s;
        };
        // 32 columns at a time: weights by the maximum so far, kept in registers
        // until their sum shows that none is above 2^15, which f16 holds (32 at
        // the maximum make 2^12); else once more in a new frame.  (64 at a
        // time, with one wait for more loads but twice the instructions to
        // fetch: 32 prompts 108.5 us for 105.7, one of 8192 tokens as long.)
        const uint64_t qa2 = f32x2(qa, qa);
        auto scores = [&](int col, float* v) {
          tc::tmem_ld32(t_s + col, v);
          if (edge) {
            __syncwarp();  // (a branch, not 32 selections each time)
            const uint32_t s = seen32(col);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (!(s & (1u << x))) v[x] = -INFINITY;
          }
        };
#pragma unroll 1
        for (int part = 0; part < C::NKV / 32; ++part) {
          uint32_t w[16];
          float v[32], l0, l1;
          const uint64_t off2 = f32x2(fr.off, fr.off);
          uint64_t l2 = f32x2(0.0f, 0.0f);
          scores(part * 32, v);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            float e0, e1;
            f32x2_split(fma_f32x2(f32x2(v[2 * x], v[2 * x + 1]), qa2, off2), e0, e1);
            e0 = exp2_fast(e0);
            e1 = exp2_fast(e1);
            l2 = add_f32x2(l2, f32x2(e0, e1));
            w[x] = half2_bits(e0, e1);
          }
          f32x2_split(l2, l0, l1);
          if (__any_sync(0xffffffffu, l0 + l1 > 32768.0f)) {
            float mx = -INFINITY;
            scores(part * 32, v);
#pragma unroll
            for (int x = 0; x < 32; ++x) mx = fmaxf(mx, v[x]);
            const PreFrame old = fr;
            if (mx > fr.top) {
              fr.top = mx;
              fr.off = fabsf(mx * qa) > kFarScore ? kNoOffset : 7.0f - mx * qa;
            }
            const float keep = frame_ratio(old, fr, qa);
            if (__any_sync(0xffffffffu, keep != 1.0f)) {
              // the sums so far by that, in O after the product that is under way,
              // and the weights of this tile already written
              l *= keep;
              const __half2 keep2 = __float2half2_rn(keep);
              tc::tmem_wait_st();
#pragma unroll 1
              for (int x = 0; x < part; ++x) {
                float z[16];
                tc::tmem_ld16(t_s + x * 16, z);
#pragma unroll
                for (int y = 0; y < 16; ++y) {
                  const __half2 t = __hmul2(*reinterpret_cast<__half2*>(&z[y]), keep2);
                  z[y] = *reinterpret_cast<const float*>(&t);
                }
                tc::tmem_st16(t_s + x * 16, reinterpret_cast<const uint32_t*>(z));
              }
              if (j > 0) {
                ok = __all_sync(0xffffffffu, mbar_wait_soon(&pv_done[m], (n_t - 1) & 1, a.wait_ns));
                if (!ok) break;
                tc::fence_after_sync();
#pragma unroll 1
                for (int x = 0; x < C::D / 16; ++x) {
                  float z[16];
                  tc::tmem_ld16(t_o + x * 16, z);
#pragma unroll
                  for (int y = 0; y < 16; ++y) z[y] *= keep;
                  tc::tmem_st16(t_o + x * 16, reinterpret_cast<const uint32_t*>(z));
                }
              }
            }
            // no weight is above 2^8 now
            const float2 f = frame_terms(fr);
            scores(part * 32, v);
            l0 = l1 = 0.0f;
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              const float e0 = exp2_fast(fmaf(v[2 * x] - f.x, qa, f.y)), e1 = exp2_fast(fmaf(v[2 * x + 1] - f.x, qa, f.y));
              l0 += e0;
              l1 += e1;
              w[x] = half2_bits(e0, e1);
            }
          }
          l += l0 + l1;
          tc::tmem_st16(t_s + part * 16, w);  // (over columns read already)
        }
        if (!ok) break;
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[m]);
        // (tokens noted where the tile is an edge of the item, be it one of this
        // half's rows or not)
        uint32_t noted = 0;
#pragma unroll
        for (int w = 0; w < C::G * C::NKV / 32; ++w) noted |= (&info_bad[n % C::INFO][0][0])[w];
        if (noted) {
          for (int w = 0; w < C::G * C::NKV / 32; ++w)
            if ((&info_bad[n % C::INFO][0][0])[w] & seen32(w % (C::NKV / 32) * 32)) lost |= 1u << w / (C::NKV / 32);
        }
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, mbar_wait_soon(&pv_done[m], (n_t - 1) & 1, a.wait_ns));
      if (!ok) break;
      tc::fence_after_sync();
      // a part's sums, its frame and l first, four columns of the rows side by side;
      // the parts' in their order by whoever comes last
      const float4* from = nullptr;
      if (SPLIT && it.parts > 1) {
        constexpr int kSlot = C::ROWS * (1 + C::D / 4);  // float4s
        float4* slot = reinterpret_cast<float4*>(a.partials) + (int64_t)blockIdx.x * kSlot + m * 128 + r_l;
        __stcg(slot, make_float4(fr.top, fr.off, l, 0.0f));
#pragma unroll 1
        for (int ch = 0; ch < C::D / 16; ++ch) {
          float v[16];
          tc::tmem_ld16(t_o + ch * 16, v);
          spoil(v, ch / 4);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            __stcg(slot + (1 + ch * 4 + x) * C::ROWS, make_float4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]));
        }
        __threadfence();
        __syncwarp();
        if (!arrive()) {
          __syncwarp();
          continue;
        }
        __threadfence();
        from = reinterpret_cast<const float4*>(a.partials) + (int64_t)(blockIdx.x - sp.part) * kSlot + m * 128 + r_l;
        for (int s = 0; s < it.parts; ++s) {
          const float4 f = __ldcg(from + (int64_t)s * kSlot);
          if (f.x > fr.top) fr = PreFrame{f.x, f.y};
        }
        l = 0.0f;
        for (int s = 0; s < it.parts; ++s) {
          const float4 f = __ldcg(from + (int64_t)s * kSlot);
          l = fmaf(frame_ratio(PreFrame{f.x, f.y}, fr, qa), f.z, l);
        }
      }
      const float inv = l != 0.0f ? 1.0f / l : 0.0f;
      // the warp's rows through the place of its rows of q, so that a row's
      // bytes are stored by neighbouring lanes
#pragma unroll 1
      for (int ch = 0; ch < C::D / 32; ++ch) {
        float v[32];
        if (SPLIT && from) {
          constexpr int kSlot = C::ROWS * (1 + C::D / 4);
#pragma unroll
          for (int x = 0; x < 32; ++x) v[x] = 0.0f;
#pragma unroll 1
          for (int s = 0; s < it.parts; ++s) {
            const float4* f = from + (int64_t)s * kSlot;
            const float4 first = __ldcg(f);
            const float w = frame_ratio(PreFrame{first.x, first.y}, fr, qa);
#pragma unroll
            for (int x = 0; x < 8; ++x) {
              const float4 z = __ldcg(f + (1 + ch * 8 + x) * C::ROWS);
              v[4 * x] = fmaf(w, z.x, v[4 * x]);
              v[4 * x + 1] = fmaf(w, z.y, v[4 * x + 1]);
              v[4 * x + 2] = fmaf(w, z.z, v[4 * x + 2]);
              v[4 * x + 3] = fmaf(w, z.w, v[4 * x + 3]);
            }
          }
        } else {
          tc::tmem_ld32(t_o + ch * 32, v);
          spoil(v, ch / 2);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          *q_place(r_l, ch * 4 + x) =
              make_uint4(pack2<C::BF16>(v[8 * x] * inv, v[8 * x + 1] * inv),
                         pack2<C::BF16>(v[8 * x + 2] * inv, v[8 * x + 3] * inv),
                         pack2<C::BF16>(v[8 * x + 4] * inv, v[8 * x + 5] * inv),
                         pack2<C::BF16>(v[8 * x + 6] * inv, v[8 * x + 7] * inv));
      }
      tc::fence_before_sync();
      __syncwarp();
#pragma unroll 4
      for (int y = 0; y < 32 / C::RPL; ++y) {
        const int row = wl * 32 + y * C::RPL + lane / C::LPR;
        const int x = it.rem0 + m * 128 + row, t = div_group(a, x);
        if (m * 128 + row < it.rows)
          *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + (int64_t)(it.row0 + it.tok0 + t) * a.ld_out +
                                    (it.h * a.group + x - t * a.group) * C::D + chunk * 8) = *q_place(row, chunk);
      }
      if (live && a.lse) {
        const float2 f = frame_terms(fr);
        a.lse[(int64_t)(it.row0 + it.tok0 + tok) * a.q_heads + head] =
            l != 0.0f ? (fmaf(f.x, qa, -f.y) + log2f(l)) * 0.69314718055994531f : -INFINITY;
      }
      __syncwarp();  // (before the next item's q goes there)
    }
    if (SPLIT && count) arrive();
  }
  if (!ok) set_error(a.err, LORA_DEV_ERR_TIMEOUT);
  // After a time-out the products issued last may still run: one more commit
  // tracks them, and tensor memory is freed after it has arrived.
  if (!__syncthreads_and(ok) && issued && tc::elect_one()) {
    tc::mma_commit(&drain_bar);
    mbar_wait_soon(&drain_bar, 0, kWaitLimitNs);
  }
  tc::fence_before_sync();
  __syncthreads();
  if (warp == C::MMA_WARP) tc::tmem_dealloc(tmem, 512);
}

}  // namespace lora
