// dspark_attention_host.h -- what the host sides of both paged attentions share: the
// tensor-map encoder, the number of SMs, shared memory per CTA.
#pragma once

#include <cudaTypedefs.h>
#include <mutex>

#include "dspark_attention.cuh"

namespace dspark {

inline std::mutex g_attn_mutex;
inline int g_attn_sms[128];
inline PFN_cuTensorMapEncodeTiled_v12000 g_attn_encode = nullptr;

// Shared memory of a CTA that has its SM to itself (227 KB), or of one of two:
// half of 228 KB, less 1 KB each for the system.
template <int CTAS>
constexpr int kSmemCta = CTAS == 1 ? 232448 : 115712;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

inline int attn_setup(int& sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return DSPARK_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_attn_mutex);
  if (!g_attn_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || !fn)
      return DSPARK_ERR_CUDA;
    g_attn_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  if (g_attn_sms[dev] == 0 &&
      cudaDeviceGetAttribute(&g_attn_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  sms = g_attn_sms[dev];
  return DSPARK_OK;
}

}  // namespace dspark
