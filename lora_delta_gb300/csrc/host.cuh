// Host-side helpers that the C-ABI translation units share: alignment tests,
// environment levers, per-kernel launch attributes, the wait limit and the
// SM count.  Nothing here allocates device memory or synchronizes.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <stdlib.h>

#include <atomic>
#include <mutex>
#include <unordered_map>

#include "common.cuh"

namespace lora {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }

inline int env_int(const char* name, int dflt) {
  const char* v = getenv(name);
  if (!v || !*v) return dflt;
  char* end = nullptr;
  long x = strtol(v, &end, 10);
  return (end && *end == 0) ? (int)x : dflt;
}

inline bool use_pdl() {
  static const bool on = env_int("LORA_PDL", 1) != 0;
  return on;
}

// Limit of the kernels' bounded waits, read at each launch
// (lora_set_wait_limit_ns).
inline std::atomic<uint64_t> g_wait_limit_ns{kWaitLimitNs};

// Per-(kernel, device) function attributes, set once: the dynamic shared
// memory opt-in (to the largest size requested so far) and the non-portable
// cluster size.
struct KernelAttrCache {
  std::mutex mu;
  std::unordered_map<uint64_t, int> smem;  // (kernel, device) -> bytes granted
  std::unordered_map<uint64_t, bool> cluster;
  std::unordered_map<uint64_t, int> occupancy;  // (kernel, device, smem) -> CTAs per SM
};
inline KernelAttrCache& attr_cache() {
  static KernelAttrCache c;
  return c;
}

template <class K>
cudaError_t prepare_kernel(K kernel, int smem_bytes, bool big_cluster) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t id = (reinterpret_cast<uint64_t>(reinterpret_cast<const void*>(kernel)) << 6) ^
                      (uint64_t)dev;
  KernelAttrCache& c = attr_cache();
  std::lock_guard<std::mutex> lock(c.mu);
  if (smem_bytes > 48 * 1024) {
    auto it = c.smem.find(id);
    if (it == c.smem.end() || it->second < smem_bytes) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes);
      if (e != cudaSuccess) return e;
      // all of the unified L1 as shared memory, so that several such CTAs fit
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
      if (e != cudaSuccess) return e;
      c.smem[id] = smem_bytes;
    }
  }
  if (big_cluster && !c.cluster[id]) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    c.cluster[id] = true;
  }
  return cudaSuccess;
}

inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA; }

inline int sm_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (!cache[dev]) {
    int v = 0;
    cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    cache[dev] = v > 0 ? v : 148;
  }
  return cache[dev];
}

// The driver's encoder of tensor maps, through the runtime, looked up once.
inline PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

}  // namespace lora
