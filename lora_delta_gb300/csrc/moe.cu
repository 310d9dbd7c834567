// C ABI of the routed-expert layer around the deltas: tokens sorted by expert
// and back, and products with an epilogue.  Host-side validation and dispatch
// onto the caller's stream; nothing here allocates or synchronizes, and every
// failure is a status code.
#include "common.cuh"
#include "host.cuh"
#include "linear.cuh"
#include "lora_delta.h"
#include "moe.cuh"

using namespace lora;

namespace {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// A matrix of 16-bit values, n rows of `width` that lie `ld` apart.
struct Mat {
  const void* p;
  int64_t ld, n, width;
};

int check_mat(const Mat& m) {
  if (!m.p) return LORA_ERR_ARG;
  if (m.n > 1 && m.ld < m.width) return LORA_ERR_SHAPE;
  return (m.n > 1 && m.ld % 8) || !aligned16(m.p) ? LORA_ERR_ALIGN : LORA_OK;
}

// Whether two matrices share elements.  Columns of one buffer, at the same row
// distance, may interleave.
bool share(const Mat& a, const Mat& b) {
  if (!a.p || !b.p || a.n < 1 || b.n < 1) return false;
  const int64_t pa = (int64_t)reinterpret_cast<uintptr_t>(a.p), pb = (int64_t)reinterpret_cast<uintptr_t>(b.p);
  const int64_t end_a = pa + 2 * ((a.n - 1) * a.ld + a.width), end_b = pb + 2 * ((b.n - 1) * b.ld + b.width);
  if (pa >= end_b || pb >= end_a) return false;
  const int64_t ld = a.n > 1 ? a.ld : b.ld;
  if ((a.n > 1 && b.n > 1 && a.ld != b.ld) || ld < 1) return true;
  int64_t d = (pb - pa) % (2 * ld);  // b's columns relative to a's
  if (d < 0) d += 2 * ld;
  return d < 2 * a.width || d + 2 * b.width > 2 * ld;
}

bool shares_words(const Mat& a, const void* p, int64_t words) {
  return share(a, Mat{p, 0, words > 0 ? 1 : 0, 2 * words});
}

template <class... P, class... A>
int launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster, const A&... args) {
  cudaLaunchAttribute attr[2];
  int attrs = 0;
  if (use_pdl()) {
    attr[attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[attrs++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (cluster > 1) {
    attr[attrs].id = cudaLaunchAttributeClusterDimension;
    attr[attrs].val.clusterDim.x = (unsigned)cluster;
    attr[attrs].val.clusterDim.y = 1;
    attr[attrs++].val.clusterDim.z = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = (unsigned)attrs;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
}

int check_moe(int T, int top_k, int H) {
  if (T < 0 || top_k < 1 || H < 1) return LORA_ERR_ARG;
  if (H % 8) return LORA_ERR_ALIGN;
  return (int64_t)T * top_k > INT32_MAX / 2 || top_k > LORA_MOE_MAX_TOP_K ? LORA_ERR_UNSUPPORTED : LORA_OK;
}

int check_dtype(int dtype) { return dtype == LORA_BF16 || dtype == LORA_F16 ? LORA_OK : LORA_ERR_ARG; }

// Tensor maps of 64 columns of K (128 bytes, swizzled): rows of x, and the rows
// of W that a CTA's tile has of the matrix or, gated, of a half.
bool encode_map(CUtensorMap* m, bool bf16, int dims, const void* base, const cuuint64_t* size, const cuuint64_t* stride,
                const cuuint32_t* box) {
  const PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return enc && enc(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)dims,
                    const_cast<void*>(base), size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                    CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_x(RowMaps* m, const LinearArgs& a, bool bf16, int first, int last) {
  const cuuint64_t size[2] = {(cuuint64_t)a.K, (cuuint64_t)a.n}, stride[1] = {(cuuint64_t)(a.n > 1 ? a.ld_x : a.K) * 2};
  for (int i = first; i <= last; ++i) {
    const cuuint32_t box[2] = {64, 16u << i};
    if (!encode_map(&m->box[i], bf16, 2, a.x, size, stride, box)) return false;
  }
  return true;
}
bool encode_w(CUtensorMap* m, const LinearArgs& a, bool bf16) {
  const cuuint64_t K = (cuuint64_t)a.K, row = (cuuint64_t)a.ld_w * 2, groups = (cuuint64_t)a.groups;
  const cuuint64_t group = a.groups > 1 ? (cuuint64_t)a.stride_w * 2 : row * (cuuint64_t)a.N;
  const cuuint64_t size[3] = {K, (cuuint64_t)a.N, groups}, stride[2] = {row, group};
  const cuuint32_t box[3] = {64, a.gated ? 64u : 128u, 1};
  return encode_map(m, bf16, 3, a.w, size, stride, box);
}

template <bool BF16, int NT>
int launch_few(const LinearArgs& a, cudaStream_t stream) {
  using C = Few<NT>;
  CUtensorMap map_w;
  RowMaps maps_x = {};
  if (!encode_w(&map_w, a, BF16) || !encode_x(&maps_x, a, BF16, 0, row_box(NT))) return LORA_ERR_CUDA;
  if (prepare_kernel(linear_few_kernel<BF16, C>, (int)C::smem(), false) != cudaSuccess) return LORA_ERR_CUDA;
  const int per = a.gated ? 64 : 128, features = (a.n_out + per - 1) / per, blocks = (a.K + 63) / 64;
  const int64_t row_tiles = ((int64_t)a.n + NT - 1) / NT;
  const int z = (int)(a.seg_start ? (row_tiles < 2 ? row_tiles : 2) : (row_tiles < 65535 ? row_tiles : 65535));
  // K in as many parts as give an SM 1.6 CTAs (48 tiles of 1 row and K = 4096, parts
  // of K: 1 23.2 us, 2 14.9, 3 13.2, 4 12.7, 5 13.0, 6 19.2; 32 tiles of 64 rows and
  // K = 14336: 1 93.8, 4 29.7, 5 28.3, 8 28.3)
  const int64_t tiles = (int64_t)features * a.groups * (a.seg_start ? 1 : z);
  int64_t split = sm_count() * 8 / 5 / tiles;
  split = split < 1 ? 1 : (split > 8 ? 8 : split);
  if (split > blocks) split = blocks;
  return launch(linear_few_kernel<BF16, C>, dim3((unsigned)(features * split), (unsigned)a.groups, (unsigned)z), C::THREADS,
                C::smem(), stream, (int)split, a, map_w, maps_x, (int)split);
}

template <bool BF16, bool GATED, int EXTRA>
int launch_pair(const LinearArgs& a, cudaStream_t stream) {
  CUtensorMap map_w;
  RowMaps maps_x = {};
  if (!encode_w(&map_w, a, BF16) || !encode_x(&maps_x, a, BF16, 1, 3)) return LORA_ERR_CUDA;
  const size_t smem = Pair::smem(a.groups);
  const auto kernel = linear_pair_kernel<BF16, GATED, EXTRA>;
  if (prepare_kernel(kernel, (int)smem, false) != cudaSuccess) return LORA_ERR_CUDA;
  int pairs = sm_count() / 2;
  if (pairs > Pair::MAX) pairs = Pair::MAX;
  return launch(kernel, dim3(2u * (unsigned)pairs), Pair::THREADS, smem, stream, 2, a, map_w, maps_x);
}

template <bool BF16, bool GATED>
int launch_pair_form(const LinearArgs& a, cudaStream_t stream) {
  if (a.delta && a.residual) return launch_pair<BF16, GATED, 3>(a, stream);
  if (a.residual) return launch_pair<BF16, GATED, 2>(a, stream);
  return a.delta ? launch_pair<BF16, GATED, 1>(a, stream) : launch_pair<BF16, GATED, 0>(a, stream);
}

// Up to how many rows of a group, on average, the kernel for few rows takes.  Few rows,
// many rows: 128 by 4096 x 28672 47 us, 59; 128 by 4096 x 6144 17, 28; experts of 64
// rows (2048 x 1536 gated) 80, 83; of 80 rows 109, 84.
constexpr int kFewRows = 64, kFewRowsAlone = 128;
int64_t mean_rows(int n, int groups) { return ((int64_t)n + groups - 1) / groups; }

template <bool BF16>
int linear_launch(const LinearArgs& a, cudaStream_t stream) {
  const int64_t rows = mean_rows(a.n, a.groups);
  const bool few = rows <= (a.groups > 1 ? kFewRows : kFewRowsAlone);
  if (!few) {
    return a.gated ? launch_pair_form<BF16, true>(a, stream) : launch_pair_form<BF16, false>(a, stream);
  }
  const int64_t want = a.groups > 1 ? 2 * rows : rows;
  if (want <= 16) return launch_few<BF16, 16>(a, stream);
  if (want <= 32) return launch_few<BF16, 32>(a, stream);
  if (want <= 64) return launch_few<BF16, 64>(a, stream);
  return launch_few<BF16, 128>(a, stream);
}

int linear_call(LinearArgs& a, int dtype, void* workspace, size_t ws_bytes, cudaStream_t stream) {
  if (a.n < 0 || a.K < 1 || a.N < 1 || a.groups < 1) return LORA_ERR_ARG;
  if (a.act < LORA_ACT_NONE || a.act > LORA_ACT_GELU_TANH || (a.gated != 0 && a.gated != 1)) return LORA_ERR_ARG;
  int rc = check_dtype(dtype);
  if (rc) return rc;
  if (a.K % 8 || a.N % (a.gated ? 16 : 8)) return LORA_ERR_ALIGN;
  if (a.groups > kMoeMaxExperts || a.n > (1 << 30) || a.K > (1 << 24) || a.N > (1 << 24) || (int64_t)a.groups * a.N > INT32_MAX) return LORA_ERR_UNSUPPORTED;
  if (a.n == 0) return LORA_OK;
  a.n_out = a.gated ? a.N / 2 : a.N;
  const Mat out = {a.out, a.ld_out, a.n, a.n_out}, x = {a.x, a.ld_x, a.n, a.K}, w = {a.w, a.ld_w, a.N, a.K},
            delta = {a.delta, a.ld_delta, a.n, a.N}, res = {a.residual, a.ld_residual, a.n, a.n_out};
  if ((rc = check_mat(out)) || (rc = check_mat(x)) || (rc = check_mat(w))) return rc;
  if (a.delta && (rc = check_mat(delta))) return rc;
  if (a.residual && (rc = check_mat(res))) return rc;
  if (a.groups > 1 && a.stride_w < (int64_t)(a.N - 1) * a.ld_w + a.K) return LORA_ERR_SHAPE;
  if (a.groups > 1 && a.stride_w % a.ld_w) return LORA_ERR_SHAPE;
  if (!aligned16(a.bias) || !aligned4(a.seg_start) || !aligned4(a.err)) return LORA_ERR_ALIGN;
  const bool in_place = a.residual == a.out && (a.ld_residual == a.ld_out || a.n == 1);
  const Mat all_w = {a.w, 0, 1, (int64_t)(a.groups - 1) * a.stride_w + (int64_t)(a.N - 1) * a.ld_w + a.K};
  const Mat in[] = {x, a.groups > 1 ? all_w : w, delta, {a.bias, 0, 1, (int64_t)a.groups * a.N}, {a.seg_start, 0, 1, 2 * (a.groups + 1)}};
  const Mat err = {a.err, 0, 1, 2};
  for (const Mat& m : in)
    if (share(out, m) || share(err, m)) return LORA_ERR_ARG;
  if ((!in_place && share(out, res)) || share(err, res) || share(err, out)) return LORA_ERR_ARG;
  if (workspace) {
    const size_t need = lora_linear_workspace_size(a.n, a.groups);
    if (ws_bytes < need) return LORA_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LORA_ERR_ALIGN;
    const Mat ws = {workspace, 0, need > 0, (int64_t)(need / 2)};
    for (const Mat& m : in)
      if (share(ws, m)) return LORA_ERR_ARG;
    if (share(ws, res) || share(ws, out) || share(ws, err)) return LORA_ERR_ARG;
    a.counters = reinterpret_cast<uint32_t*>(workspace);
    a.parts = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + kLinearCounterBytes);
  }
  a.wait_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  return dtype == LORA_BF16 ? linear_launch<true>(a, stream) : linear_launch<false>(a, stream);
}

}  // namespace

extern "C" {

int lora_moe_dispatch(void* rows, int64_t ld_rows, int32_t* seg_start, int32_t* row_pair, int32_t* pair_row,
                      int32_t* row_expert, int32_t* row_lora, const void* x, int64_t ld_x, const int32_t* topk_ids,
                      const int32_t* lora_ids, const int32_t* expert_map, int n_global_experts, int T, int top_k, int E,
                      int H, uint32_t* err_word, lora_stream_t stream) {
  int rc = check_moe(T, top_k, H);
  if (rc) return rc;
  if (E < 1 || !seg_start || (expert_map && n_global_experts < 1)) return LORA_ERR_ARG;
  if (E > kMoeMaxExperts) return LORA_ERR_UNSUPPORTED;
  const int P = T * top_k;
  if (T > 0) {
    if (!row_pair || !pair_row || !row_expert || !row_lora || !topk_ids) return LORA_ERR_ARG;
    if ((rc = check_mat(Mat{rows, ld_rows, P, H})) || (rc = check_mat(Mat{x, ld_x, T, H}))) return rc;
  }
  const void* words[] = {seg_start, row_pair, pair_row, row_expert, row_lora, topk_ids, lora_ids, expert_map, err_word};
  const int64_t sizes[] = {E + 1, P, P, P, P, P, T, n_global_experts, 1};
  for (int i = 0; i < 9; ++i) {
    if (!aligned4(words[i])) return LORA_ERR_ALIGN;
    if (T > 0 && shares_words(Mat{rows, ld_rows, P, H}, words[i], sizes[i])) return LORA_ERR_ARG;
    for (int j = 0; j < i; ++j)  // an output of the plan, or the error word, and any other array
      if ((j < 5 || i == 8) && words[i] && words[j] && sizes[j] > 0 && shares_words(Mat{words[i], 0, sizes[i] > 0, 2 * sizes[i]}, words[j], sizes[j]))
        return LORA_ERR_ARG;
    if ((i < 5 || i == 8) && T > 0 && shares_words(Mat{x, ld_x, T, H}, words[i], sizes[i])) return LORA_ERR_ARG;
  }
  if (T > 0 && share(Mat{rows, ld_rows, P, H}, Mat{x, ld_x, T, H})) return LORA_ERR_ARG;
  const MoePlanArgs p = {{topk_ids, expert_map, n_global_experts, E}, lora_ids, P, top_k, seg_start, row_pair, pair_row,
                         row_expert, row_lora, err_word};
  MoveArgs a = {};
  a.out = rows;
  a.ld_out = ld_rows;
  a.x = x;
  a.ld_x = ld_x;
  a.pair_row = pair_row;
  a.T = T;
  a.top_k = top_k;
  a.H = H;
  a.P = P;
  if (T > 0 && P <= kMoeFewPairs) {
    const size_t smem = (size_t)(E + 1) * 4 + (size_t)P * 2;
    return launch(moe_dispatch_few_kernel, dim3((unsigned)T), kMoeThreads, smem, (cudaStream_t)stream, 1, p, a);
  }
  const int smem = (int)moe_sort_smem(E);
  if (prepare_kernel(moe_sort_kernel, smem, true) != cudaSuccess) return LORA_ERR_CUDA;
  const int want = P / 2048 + 1, ctas = want < kMoeSortCluster ? want : kMoeSortCluster;
  if ((rc = launch(moe_sort_kernel, dim3((unsigned)ctas), kRouteThreads, (size_t)smem, (cudaStream_t)stream, ctas, p))) return rc;
  if (T == 0) return LORA_OK;
  return launch(moe_scatter_kernel, dim3((unsigned)T), kMoeThreads, 0, (cudaStream_t)stream, 1, a);
}

int lora_moe_combine(void* out, int64_t ld_out, const void* rows, int64_t ld_rows, const int32_t* pair_row,
                     const float* weights, const void* residual, int64_t ld_residual, int T, int top_k, int H, int dtype,
                     lora_stream_t stream) {
  int rc = check_moe(T, top_k, H);
  if (rc || (rc = check_dtype(dtype))) return rc;
  if (T == 0) return LORA_OK;
  const int P = T * top_k;
  const Mat o = {out, ld_out, T, H}, y = {rows, ld_rows, P, H}, res = {residual, ld_residual, T, H};
  if (!pair_row) return LORA_ERR_ARG;
  if ((rc = check_mat(o)) || (rc = check_mat(y)) || (residual && (rc = check_mat(res)))) return rc;
  if (!aligned4(pair_row) || !aligned4(weights)) return LORA_ERR_ALIGN;
  const bool in_place = residual == out && (ld_residual == ld_out || T == 1);
  if (share(o, y) || (residual && !in_place && share(o, res)) || shares_words(o, pair_row, P) || shares_words(o, weights, P))
    return LORA_ERR_ARG;
  MoveArgs a = {};
  a.out = out;
  a.ld_out = ld_out;
  a.rows = rows;
  a.ld_rows = ld_rows;
  a.residual = residual;
  a.ld_residual = ld_residual;
  a.pair_row = pair_row;
  a.weights = weights;
  a.T = T;
  a.top_k = top_k;
  a.H = H;
  a.P = P;
  return dtype == LORA_BF16 ? launch(moe_combine_kernel<true>, dim3((unsigned)T), kMoeThreads, 0, (cudaStream_t)stream, 1, a)
                            : launch(moe_combine_kernel<false>, dim3((unsigned)T), kMoeThreads, 0, (cudaStream_t)stream, 1, a);
}

int lora_moe_combine_grad(void* grad_rows, int64_t ld_grad_rows, float* grad_weights, const void* grad_out,
                          int64_t ld_grad_out, const void* rows, int64_t ld_rows, const int32_t* pair_row,
                          const float* weights, int T, int top_k, int H, int dtype, lora_stream_t stream) {
  int rc = check_moe(T, top_k, H);
  if (rc || (rc = check_dtype(dtype))) return rc;
  if (T == 0) return LORA_OK;
  const int P = T * top_k;
  const Mat gr = {grad_rows, ld_grad_rows, P, H}, go = {grad_out, ld_grad_out, T, H}, y = {rows, ld_rows, P, H};
  if (!pair_row) return LORA_ERR_ARG;
  if ((rc = check_mat(gr)) || (rc = check_mat(go)) || (rc = check_mat(y))) return rc;
  if (!aligned4(pair_row) || !aligned4(weights) || !aligned4(grad_weights)) return LORA_ERR_ALIGN;
  const Mat gw = {grad_weights, 0, 1, 2 * (int64_t)P};
  if (share(gr, go) || share(gr, y) || shares_words(gr, pair_row, P) || shares_words(gr, weights, P) || share(gr, gw) ||
      share(gw, go) || share(gw, y) || shares_words(gw, pair_row, P) || shares_words(gw, weights, P))
    return LORA_ERR_ARG;
  MoveArgs a = {};
  a.out = grad_rows;
  a.ld_out = ld_grad_rows;
  a.x = grad_out;
  a.ld_x = ld_grad_out;
  a.rows = rows;
  a.ld_rows = ld_rows;
  a.pair_row = pair_row;
  a.weights = weights;
  a.grad_weights = grad_weights;
  a.T = T;
  a.top_k = top_k;
  a.H = H;
  a.P = P;
  return dtype == LORA_BF16
             ? launch(moe_combine_grad_kernel<true>, dim3((unsigned)T), kMoeThreads, 0, (cudaStream_t)stream, 1, a)
             : launch(moe_combine_grad_kernel<false>, dim3((unsigned)T), kMoeThreads, 0, (cudaStream_t)stream, 1, a);
}

size_t lora_linear_workspace_size(int n, int groups) {
  const bool few = groups < 1 || mean_rows(n, groups) <= (groups > 1 ? kFewRows : kFewRowsAlone);
  return few ? 0 : kLinearCounterBytes + kLinearPartFloats * 4;
}
size_t lora_linear_zeroed_bytes(void) { return kLinearCounterBytes; }

int lora_linear(void* out, int64_t ld_out, const void* x, int64_t ld_x, int n, int k_in, const void* w, int64_t ld_w,
                int n_out, const void* bias, const void* delta, int64_t ld_delta, const void* residual,
                int64_t ld_residual, int activation, int gated, int dtype, void* workspace, size_t ws_bytes,
                uint32_t* err_word, lora_stream_t stream) {
  LinearArgs a = {out, ld_out, x, ld_x, w, ld_w, 0, bias, delta, ld_delta, residual, ld_residual, nullptr, 1, n, k_in, n_out,
                  0, activation, gated, err_word, 0, nullptr, nullptr};
  return linear_call(a, dtype, workspace, ws_bytes, (cudaStream_t)stream);
}

int lora_moe_linear(void* out, int64_t ld_out, const void* rows, int64_t ld_rows, int n, int k_in, const int32_t* seg_start,
                    int E, const void* w, int64_t ld_w, int64_t stride_w, int n_out, const void* bias, const void* delta,
                    int64_t ld_delta, const void* residual, int64_t ld_residual, int activation, int gated, int dtype,
                    void* workspace, size_t ws_bytes, uint32_t* err_word, lora_stream_t stream) {
  if (!seg_start) return LORA_ERR_ARG;
  LinearArgs a = {out, ld_out, rows, ld_rows, w, ld_w, stride_w, bias, delta, ld_delta, residual, ld_residual, seg_start, E, n,
                  k_in, n_out, 0, activation, gated, err_word, 0, nullptr, nullptr};
  return linear_call(a, dtype, workspace, ws_bytes, (cudaStream_t)stream);
}

}  // extern "C"
