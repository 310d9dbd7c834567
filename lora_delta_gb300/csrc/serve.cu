// C ABI of the serving-step operators beside the delta: the batch plan, the
// 4-bit key/value cache's store and read, and attention over it.  Host-side
// validation and dispatch onto the caller's stream; nothing here allocates or
// synchronizes, and every failure is a status code.
#include <math.h>

#include <type_traits>

#include "common.cuh"
#include "host.cuh"
#include "kv4.cuh"
#include "kv4_attn.cuh"
#include "kv4_prefill.cuh"
#include "lora_delta.h"
#include "plan.cuh"

using namespace lora;

namespace {

// Whether two arrays share bytes (a NULL one has none).
inline bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && np && nq && a < b + nq && b < a + np;
}
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

int check_page_size(int page_size) {
  if (page_size < 1) return LORA_ERR_ARG;
  return page_size % kKvTile || page_size > 1024 ? LORA_ERR_UNSUPPORTED : LORA_OK;
}

// The cache's own arguments, common to store, read and attention.
int check_cache(const void* pages, int64_t num_pages, int page_size, int heads, int head_dim,
                int dtype) {
  if (!pages || num_pages < 1 || heads < 1) return LORA_ERR_ARG;
  if (dtype != LORA_BF16 && dtype != LORA_F16) return LORA_ERR_ARG;
  if (const int rc = check_page_size(page_size)) return rc;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return LORA_ERR_UNSUPPORTED;
  if (num_pages > INT32_MAX || heads > 1024) return LORA_ERR_UNSUPPORTED;
  return aligned16(pages) ? LORA_OK : LORA_ERR_ALIGN;
}

int check_rows(const void* p, int64_t ld, int n, int width) {
  if (!p) return LORA_ERR_ARG;
  if (n > 1 && ld < width) return LORA_ERR_SHAPE;
  return ld % 8 || !aligned16(p) ? LORA_ERR_ALIGN : LORA_OK;
}

// Dynamic shared memory of an attention CTA: what a CTA may have, less the
// kernels' own variables.
constexpr size_t kAttnMaxSmem = 227 * 1024 - 2048;

// Launch of a kernel that waits for the one before it by griddepcontrol.
template <class... P, class... A>
int launch_after(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t stream,
                 const A&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = use_pdl() ? 1 : 0;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
}

// f(kernel for head_dim and type)
template <class F>
int by_type(int head_dim, int dtype, F f) {
  const bool bf = dtype == LORA_BF16;
  if (head_dim == 64) return bf ? f(std::integral_constant<int, 64>(), std::true_type())
                                : f(std::integral_constant<int, 64>(), std::false_type());
  if (head_dim == 128) return bf ? f(std::integral_constant<int, 128>(), std::true_type())
                                 : f(std::integral_constant<int, 128>(), std::false_type());
  return bf ? f(std::integral_constant<int, 256>(), std::true_type())
            : f(std::integral_constant<int, 256>(), std::false_type());
}

int rows_call(bool store, const void* k, int64_t ld_k, const void* v, int64_t ld_v, void* pages,
              int64_t num_pages, int page_size, int heads, int head_dim, int dtype,
              const int64_t* slot_map, int n, uint32_t* err, cudaStream_t stream) {
  if (n < 0) return LORA_ERR_ARG;
  if (n == 0) return LORA_OK;
  int rc = check_cache(pages, num_pages, page_size, heads, head_dim, dtype);
  if (rc) return rc;
  if (!slot_map) return LORA_ERR_ARG;
  if ((rc = check_rows(k, ld_k, n, heads * head_dim))) return rc;
  if ((rc = check_rows(v, ld_v, n, heads * head_dim))) return rc;
  if (!aligned8(slot_map) || !aligned4(err)) return LORA_ERR_ALIGN;
  Kv4Rows a = {};
  a.k = k;
  a.v = v;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.pages = reinterpret_cast<uint8_t*>(pages);
  a.num_slots = num_pages * page_size;
  a.page_size = page_size;
  a.heads = heads;
  a.slot_map = slot_map;
  a.n = n;
  a.err = err;
  a.page_shift = -1;
  for (int x = 4; x <= 10; ++x)
    if (page_size == 1 << x) a.page_shift = x;
  // a head a task until there are 128 warps for an SM
  const int64_t blocks = ((int64_t)n + 7) / 8, fill = (int64_t)sm_count() * 128;
  int64_t per = blocks * 2 * heads / fill;
  per = per < 1 ? 1 : (per > heads ? heads : per);
  a.task_heads = (int)per;
  const int64_t tasks = blocks * 2 * ((heads + per - 1) / per);
  if (tasks > INT32_MAX) return LORA_ERR_UNSUPPORTED;
  constexpr int kWarps = kKvThreads / 32;
  const int64_t want = (tasks + kWarps - 1) / kWarps, most = (int64_t)sm_count() * 32;
  const unsigned grid = (unsigned)(want < most ? want : most);
  return by_type(head_dim, dtype, [&](auto d, auto bf) {
    constexpr int D = decltype(d)::value;
    constexpr bool BF16 = decltype(bf)::value;
    return store ? launch_after(kv4_rows_kernel<D, BF16, true>, grid, kKvThreads, 0, stream, a)
                 : launch_after(kv4_rows_kernel<D, BF16, false>, grid, kKvThreads, 0, stream, a);
  });
}

// Configurations of the decode kernel: 16 warps where their sums fit 128
// registers, else 8.
template <int D, bool BF16, int NT>
using DecCfg = Dec<D, BF16, NT, (D * NT <= 128 ? 16 : 8)>;

template <class C>
int launch_decode(const AttnArgs& a, cudaStream_t stream) {
  // as many units in flight as shared memory holds
  int stages = C::MAX_STAGES;
  while (stages > C::MIN_STAGES && C::smem(a.B, stages, false) > kAttnMaxSmem) --stages;
  static_assert(C::smem(kAttnMaxReqs, C::MIN_STAGES, false) <= kAttnMaxSmem, "a CTA's shared memory");
  const int cached = C::smem(a.B, stages, true) <= kAttnMaxSmem;
  const int smem = (int)C::smem(a.B, stages, cached != 0);
  if (prepare_kernel(kv4_decode_kernel<C>, smem, false) != cudaSuccess) return LORA_ERR_CUDA;
  int ctas = sm_count();
  if (ctas > kAttnMaxCtas) ctas = kAttnMaxCtas;
  // Items of at most this many units stay whole where there is a CTA for each: no
  // joins over CTAs against fewer of them (8 heads of 128; whole, shared out).  One
  // request of 300 tokens 9.9, 14.2 us; 1000 12.9, 15.8; 2000 (63 units) 16.5, 16.1;
  // 4000 24.4, 14.5.  16 requests of 2000 18.0, 22.9; of 4000 26.2, 29.6.
  static const int alone = env_int("LORA_ATTN_ALONE", 64);
  return launch_after(kv4_decode_kernel<C>, (unsigned)ctas, C::THREADS, (size_t)smem, stream, a, stages, cached, alone);
}

template <class C, bool SPLIT>
int launch_prefill_as(const AttnArgs& a, int min_rows, cudaStream_t stream) {
  const int smem = (int)C::smem(a.B);
  if (prepare_kernel(kv4_prefill_kernel<C, SPLIT>, smem, false) != cudaSuccess) return LORA_ERR_CUDA;
  // (the kernel hands registers from warp to warp, out of those that it was
  // built to start with)
  static const bool regs_ok = [] {
    cudaFuncAttributes fa;
    return cudaFuncGetAttributes(&fa, kv4_prefill_kernel<C, SPLIT>) == cudaSuccess && fa.numRegs >= C::REGS;
  }();
  if (!regs_ok) return LORA_ERR_CUDA;
  const int ctas = sm_count() < kAttnMaxCtas ? sm_count() : kAttnMaxCtas;
  kv4_prefill_kernel<C, SPLIT><<<ctas, C::THREADS, smem, stream>>>(a, min_rows);
  return cuda_status(cudaGetLastError());
}

// Items are split along the tokens where, by the rows of the batch, there are
// at most half as many as CTAs, and contexts may be long enough for two parts.
template <class C>
int launch_prefill(const AttnArgs& a, int min_rows, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.n * a.group, reqs = rows / (min_rows + 1);
  const int64_t items = (rows / C::ROWS + (reqs < a.B ? reqs : a.B)) * a.heads;
  const bool split = 2 * items <= sm_count() && a.cap >= 2 * kPartTiles * C::NKV;
  return split ? launch_prefill_as<C, true>(a, min_rows, stream) : launch_prefill_as<C, false>(a, min_rows, stream);
}

// Floats of the partial results of every configuration.
template <class C>
constexpr size_t dec_partials() {
  return (size_t)kAttnMaxCtas * (2 + C::NW) * C::SLOT;
}
constexpr size_t max2(size_t x, size_t y) { return x > y ? x : y; }
constexpr size_t kPartialFloats =
    max2(max2(max2(dec_partials<DecCfg<64, true, 1>>(), dec_partials<DecCfg<64, true, 2>>()),
              max2(dec_partials<DecCfg<64, true, 4>>(), dec_partials<DecCfg<128, true, 1>>())),
         max2(max2(dec_partials<DecCfg<128, true, 2>>(), dec_partials<DecCfg<128, true, 4>>()),
              max2(dec_partials<DecCfg<256, true, 1>>(), dec_partials<DecCfg<256, true, 2>>())));
constexpr size_t kCounterBytes = (size_t)kAttnMaxCtas * 16;
// (a part of a prefill item a CTA; a count for each of 8 warps of at most half as
// many items)
static_assert(kPartialFloats >= (size_t)kAttnMaxCtas * 256 * (128 + 4) && kPartialFloats >= (size_t)kAttnMaxCtas * 128 * (256 + 4),
              "the parts of the prefill kernel's items");

}  // namespace

extern "C" {

int lora_batch_plan_bounded(const int32_t* ctx_len, const int32_t* new_len, const int32_t* req_slot,
                            int n_reqs, int n_rows, int page_size, int32_t* block_table,
                            int64_t ld_table, int max_pages, const int32_t* free_pages, int free_cap,
                            const int32_t* free_count, int32_t* free_left, int32_t* row_start,
                            int32_t* seq_len, int32_t* row_req, int32_t* position,
                            int64_t* slot_map, int32_t* seq_slot, uint32_t* err_word,
                            lora_stream_t stream) {
  if (n_reqs < 0 || n_rows < 0 || max_pages < 0 || free_cap < 0 || !row_start) return LORA_ERR_ARG;
  if (n_reqs > 0 && (!ctx_len || !new_len || !block_table || !seq_len)) return LORA_ERR_ARG;
  if (n_rows > 0 && (!row_req || !position || !slot_map || !seq_slot)) return LORA_ERR_ARG;
  if ((free_pages != nullptr) != (free_count != nullptr) ||
      (free_pages != nullptr) != (free_left != nullptr))
    return LORA_ERR_ARG;
  if (const int rc = check_page_size(page_size)) return rc;
  if (n_reqs > kPlanMaxReqs || (int64_t)n_reqs * max_pages > INT32_MAX ||
      (int64_t)max_pages * page_size > (1 << 29))
    return LORA_ERR_UNSUPPORTED;
  if (n_reqs > 1 && ld_table < max_pages) return LORA_ERR_SHAPE;
  if (!aligned16(row_req) || !aligned16(position) || !aligned16(slot_map) || !aligned16(seq_slot))
    return LORA_ERR_ALIGN;
  // the one input that may be replaced is ctx_len, by seq_len
  const size_t reqs = (size_t)n_reqs * 4, rows = (size_t)n_rows * 4;
  const struct {
    const void* p;
    size_t bytes;
  } ins[] = {{ctx_len, reqs}, {new_len, reqs}, {req_slot, reqs}, {free_count, 4}},
    outs[] = {{row_start, reqs + 4}, {seq_len, reqs}, {row_req, rows}, {position, rows}, {seq_slot, rows}, {slot_map, 2 * rows}};
  for (const auto& in : ins)
    for (const auto& out : outs)
      if (overlap(in.p, in.bytes, out.p, out.bytes) && !(in.p == ctx_len && out.p == seq_len && in.p == out.p)) return LORA_ERR_ARG;
  for (int i = 0; i < 3; ++i)
    if (overlap(ins[i].p, ins[i].bytes, free_left, 4)) return LORA_ERR_ARG;
  PlanArgs a = {ctx_len,    new_len,   req_slot, n_reqs,   n_rows,   page_size, max_pages,
                block_table, ld_table, free_pages, free_cap, free_count, free_left, row_start, seq_len,
                row_req,    position,  slot_map, seq_slot, err_word};
  const int smem = (int)plan_smem_bytes(n_reqs);
  if (prepare_kernel(batch_plan_kernel, smem, false) != cudaSuccess) return LORA_ERR_CUDA;
  const int64_t per_cta = kPlanThreads * kPlanRowsPerThread;
  // (one cluster where the free count or the lengths are replaced in place)
  const bool cluster = (free_left != nullptr && free_left == free_count) || (n_reqs > 0 && seq_len == ctx_len);
  const int64_t want = (n_rows + per_cta - 1) / per_cta, most = cluster ? kPlanMaxCluster : sm_count();
  const int ctas = want < 1 ? 1 : (int)(want < most ? want : most);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = use_pdl() ? attr : attr + 1;
  cfg.numAttrs = (use_pdl() ? 1 : 0) + (cluster && ctas > 1 ? 1 : 0);
  return cuda_status(cudaLaunchKernelEx(&cfg, batch_plan_kernel, (const PlanArgs)a, cluster && ctas > 1 ? 1 : 0));
}

int lora_batch_plan(const int32_t* ctx_len, const int32_t* new_len, const int32_t* req_slot,
                    int n_reqs, int n_rows, int page_size, int32_t* block_table, int64_t ld_table,
                    int max_pages, const int32_t* free_pages, const int32_t* free_count,
                    int32_t* free_left, int32_t* row_start, int32_t* seq_len, int32_t* row_req,
                    int32_t* position, int64_t* slot_map, int32_t* seq_slot, uint32_t* err_word,
                    lora_stream_t stream) {
  return lora_batch_plan_bounded(ctx_len, new_len, req_slot, n_reqs, n_rows, page_size, block_table,
                                 ld_table, max_pages, free_pages, INT32_MAX, free_count, free_left,
                                 row_start, seq_len, row_req, position, slot_map, seq_slot,
                                 err_word, stream);
}

int lora_pages_release(const int32_t* done, const int32_t* seq_len, int n_reqs, int page_size,
                       int32_t* block_table, int64_t ld_table, int max_pages, int32_t* free_pages,
                       int free_cap, int32_t* free_count, uint32_t* err_word,
                       lora_stream_t stream) {
  if (n_reqs < 0 || max_pages < 0 || free_cap < 0) return LORA_ERR_ARG;
  if (n_reqs == 0 || max_pages == 0) return LORA_OK;
  if (!done || !seq_len || !block_table || !free_pages || !free_count) return LORA_ERR_ARG;
  if (const int rc = check_page_size(page_size)) return rc;
  if (n_reqs > kPlanMaxReqs || (int64_t)n_reqs * max_pages > INT32_MAX) return LORA_ERR_UNSUPPORTED;
  if (n_reqs > 1 && ld_table < max_pages) return LORA_ERR_SHAPE;
  pages_release_kernel<<<1, kPlanThreads, 0, (cudaStream_t)stream>>>(
      done, seq_len, n_reqs, page_size, block_table, ld_table, max_pages, free_pages, free_cap,
      free_count, err_word);
  return cuda_status(cudaGetLastError());
}

size_t lora_kv4_page_bytes(int page_size, int kv_heads, int head_dim) {
  if (check_page_size(page_size) || kv_heads < 1) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return (size_t)kv_heads * (page_size / kKvTile) * kv4_tile_bytes(head_dim);
}

int lora_kv4_append(void* pages, int64_t num_pages, int page_size, int kv_heads, int head_dim,
                    int dtype, const void* k, int64_t ld_k, const void* v, int64_t ld_v,
                    const int64_t* slot_map, int n, uint32_t* err_word, lora_stream_t stream) {
  return rows_call(true, k, ld_k, v, ld_v, pages, num_pages, page_size, kv_heads, head_dim, dtype,
                   slot_map, n, err_word, (cudaStream_t)stream);
}

int lora_kv4_read(const void* pages, int64_t num_pages, int page_size, int kv_heads, int head_dim,
                  int dtype, void* k, int64_t ld_k, void* v, int64_t ld_v, const int64_t* slot_map,
                  int n, uint32_t* err_word, lora_stream_t stream) {
  return rows_call(false, k, ld_k, v, ld_v, const_cast<void*>(pages), num_pages, page_size,
                   kv_heads, head_dim, dtype, slot_map, n, err_word, (cudaStream_t)stream);
}

size_t lora_kv4_attention_workspace_size(void) { return kCounterBytes + kPartialFloats * 4; }
size_t lora_kv4_attention_zeroed_bytes(void) { return kCounterBytes; }

int lora_kv4_attention(void* out, int64_t ld_out, const void* q, int64_t ld_q, int n, int q_heads,
                       const void* pages, int64_t num_pages, int page_size, int kv_heads,
                       int head_dim, int dtype, const int32_t* block_table, int64_t ld_table,
                       int max_pages, const int32_t* row_start, const int32_t* seq_len, int n_reqs,
                       int max_q_len, float scale, int window, float* lse, void* workspace,
                       size_t ws_bytes, uint32_t* err_word, lora_stream_t stream) {
  if (n < 0 || n_reqs < 0 || max_pages < 0 || window < 0 || q_heads < 1 || max_q_len < 0)
    return LORA_ERR_ARG;
  if (n == 0) return LORA_OK;
  int rc = check_cache(pages, num_pages, page_size, kv_heads, head_dim, dtype);
  if (rc) return rc;
  if (q_heads % kv_heads) return LORA_ERR_SHAPE;
  if (!row_start || (n_reqs > 0 && (!seq_len || !block_table))) return LORA_ERR_ARG;
  if (n_reqs > kAttnMaxReqs || (int64_t)max_pages * page_size > (1 << 29) || q_heads > 65535)
    return LORA_ERR_UNSUPPORTED;
  if ((rc = check_rows(out, ld_out, n, q_heads * head_dim))) return rc;
  if ((rc = check_rows(q, ld_q, n, q_heads * head_dim))) return rc;
  if (n_reqs > 1 && ld_table < max_pages) return LORA_ERR_SHAPE;
  if (!workspace || ws_bytes < lora_kv4_attention_workspace_size()) return LORA_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LORA_ERR_ALIGN;
  if (n_reqs * ((int64_t)max_pages * (page_size / kKvTile) + kItemCost) * kv_heads > INT32_MAX ||
      (int64_t)n * (q_heads / kv_heads) > INT32_MAX)
    return LORA_ERR_UNSUPPORTED;
  AttnArgs a = {};
  a.out = out;
  a.q = q;
  a.ld_out = ld_out;
  a.ld_q = ld_q;
  a.n = n;
  a.q_heads = q_heads;
  a.heads = kv_heads;
  a.group = q_heads / kv_heads;
  a.group_inv = (uint32_t)(((1ull << 31) + a.group - 1) / a.group);
  a.pages = reinterpret_cast<const uint8_t*>(pages);
  a.num_pages = num_pages;
  a.page_size = page_size;
  a.table = block_table;
  a.ld_table = ld_table;
  a.cap = max_pages * page_size;
  a.tpp_inv = (uint32_t)(((1ull << 31) + page_size / kKvTile - 1) / (page_size / kKvTile));
  a.row_start = row_start;
  a.seq_len = seq_len;
  a.B = n_reqs;
  a.max_q_len = max_q_len;
  a.window = window;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  a.lse = lse;
  a.err = err_word;
  a.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  a.counters = reinterpret_cast<uint32_t*>(workspace);
  a.partials = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + kCounterBytes);
  const int64_t rows = (int64_t)max_q_len * a.group;
  return by_type(head_dim, dtype, [&](auto d, auto bf) {
    constexpr int D = decltype(d)::value;
    constexpr bool BF16 = decltype(bf)::value;
    if (rows <= 8) return launch_decode<DecCfg<D, BF16, 1>>(a, (cudaStream_t)stream);
    if (rows <= 16) return launch_decode<DecCfg<D, BF16, 2>>(a, (cudaStream_t)stream);
    // the most rows that the decode kernel takes; requests with more go to the
    // tensor cores
    constexpr int NT = D == 256 ? 2 : 4;
    const int rc = launch_decode<DecCfg<D, BF16, NT>>(a, (cudaStream_t)stream);
    if (rc || rows <= 8 * NT) return rc;
    return launch_prefill<Pre<D, BF16>>(a, 8 * NT, (cudaStream_t)stream);
  });
}

}  // extern "C"
