// dspark_attention.cu -- dspark_paged_attention: checks, tensor maps, shapes and
// launches (the kernels and their reasons are in dspark_attention.cuh).
#include <algorithm>
#include <cmath>

#include "dspark_attention.cuh"
#include "dspark_attention_host.h"

namespace dspark {
namespace {

// A tensor of 16-bit elements in the 128-byte swizzled layout; dims[0] innermost.
// A row of 128 elements is fetched in two halves, whose 256 bytes come together;
// past a row of 64 lies another head's, which would be fetched for nothing (49%
// more DRAM reads, measured with 24 heads side by side).
bool attn_map(CUtensorMap* map, bool f16, const void* base, int rank, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box) {
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return g_attn_encode(map,
                       f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides, box,
                       one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       dims[0] == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                     : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Launch {
  CUtensorMap q, k, v;
  AttnArgs a;
  JoinArgs j;
  int items;
  cudaStream_t stream;
};

template <class S, bool F16>
int attn_launch(Launch& c, int sms) {
  static bool ready[128];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128) return DSPARK_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(g_attn_mutex);
    if (!ready[dev]) {
      if (cudaFuncSetAttribute(k_attention<S, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kSmemCta<S::CTAS>) != cudaSuccess)
        return DSPARK_ERR_CUDA;
      ready[dev] = true;
    }
  }
  AttnArgs& a = c.a;
  a.ctas = std::max(1, std::min(sms * S::CTAS, DSPARK_PAGED_MAX_CTAS) / a.n_chunks);
  const int grid = a.ctas * a.n_chunks;
  // Shared memory: what the queries and the weights leave is the rings'. A
  // second tile of queries where it costs them no tile.
  constexpr uint32_t kSmem = kSmemCta<S::CTAS>;
  const uint32_t q_bytes = static_cast<uint32_t>(S::HALVES * a.n_cols * 128);
  a.p_bytes = static_cast<uint32_t>(a.n_cols / 16 * 4096);
  auto ring_stages = [&](int q_bufs) {
    a.q_bufs = q_bufs;
    a.p_off = kCtlBytes<S> + q_bufs * q_bytes;
    a.ring_off = a.p_off + S::PBUFS * a.p_bytes;
    return std::min<int>(kMaxStages, (kSmem - a.ring_off) / S::kStage);
  };
  const int stages = ring_stages(1);
  if (ring_stages(2) < stages) ring_stages(1);
  a.k_stages = stages / 2;
  a.v_stages = stages - a.k_stages;  // values wait for the softmax, keys do not
  a.lead = 3;
  const size_t smem = a.ring_off + static_cast<size_t>(stages) * S::kStage;
  if (launch_pdl(k_attention<S, F16>, grid, S::THREADS, smem, c.stream, c.q, c.k, c.v, a) !=
      cudaSuccess)
    return DSPARK_ERR_CUDA;
  JoinArgs& j = c.j;
  j.n = grid;
  j.ctas = a.ctas;
  // Few requests: each is cut into many pieces, which eight warps share per row.
  j.per_row = c.items * 8 <= grid ? kJoinWarps : 1;
  const int rows = kJoinWarps / j.per_row;
  if (launch_pdl(k_attention_join<S::D, F16>,
                 dim3(std::min(c.items, grid), (a.n_cols + rows - 1) / rows), kJoinWarps * 32, 0,
                 c.stream, j) != cudaSuccess ||
      cudaGetLastError() != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

// The smallest row block that holds the rows; keys are copied once for all of them.
template <int D, bool F16>
int attn_shape(Launch& c, int sms) {
  if (c.a.n_cols <= 16) return attn_launch<AttnShape<D, 16, 1, 2, 2>, F16>(c, sms);
  if (c.a.n_cols <= 32) return attn_launch<AttnShape<D, 32, 1, 2, 2>, F16>(c, sms);
  if (c.a.n_cols <= 64) return attn_launch<AttnShape<D, 64, 4, 1, 2>, F16>(c, sms);
  if (c.a.n_cols <= 96) return attn_launch<AttnShape<D, 96, 3, 1, 2>, F16>(c, sms);
  return attn_launch<AttnShape<D, 160, 3, 1, 1>, F16>(c, sms);
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" int dspark_paged_attention(
    const void* q, int64_t q_row_stride, int64_t q_head_stride, const void* k_cache,
    const void* v_cache, int64_t page_stride, int64_t token_stride, int64_t head_stride,
    int32_t page_size, int32_t num_pages, const int32_t* block_table, int64_t table_stride,
    int32_t max_pages, const int32_t* context_len, const int64_t* row_off, int32_t B,
    int32_t n_tokens, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_new, float scale,
    int32_t window, int32_t dtype, void* out, float* lse, int32_t* device_status, void* workspace,
    size_t workspace_bytes, struct CUstream_st* stream) {
  if (B < 0 || n_tokens < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 || Hq > 65536 ||
      (D != 64 && D != 128) || max_new < 1 || max_new > (1 << 20) || !std::isfinite(scale) ||
      !(scale > 0.f) || window < 0 || (dtype != DSPARK_BF16 && dtype != DSPARK_F16) ||
      page_size < 8 || page_size > 1024 || (page_size & (page_size - 1)) != 0 || num_pages < 1 ||
      static_cast<int64_t>(num_pages) * page_size > INT32_MAX || max_pages < 1 ||
      static_cast<int64_t>(max_pages) * page_size > INT32_MAX - 2 * kTileTok ||
      static_cast<int64_t>(max_pages) * page_size / kTileTok * Hkv > INT32_MAX / 2 ||
      table_stride < max_pages || !device_status)
    return DSPARK_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || n_tokens == 0)  // no rows
    return cudaMemsetAsync(device_status, 0, 4, st) == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
  if (!q || !k_cache || !v_cache || !block_table || !context_len || !row_off || !out ||
      !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      q_row_stride < 0 || q_head_stride < 0 || page_stride < 0 || token_stride < 0 ||
      head_stride < 0 ||
      ((q_row_stride | q_head_stride | page_stride | token_stride | head_stride) & 7) != 0)
    return DSPARK_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < DSPARK_PAGED_ATTENTION_WS_BYTES(Hq, Hkv, max_new, D))
    return DSPARK_ERR_WORKSPACE;
  int sms = 0;
  const int rc = attn_setup(sms);
  if (rc != DSPARK_OK) return rc;

  Launch c{};
  AttnArgs& a = c.a;
  a.G = Hq / Hkv;
  a.parts = 1;  // of a group of query heads, if it has more than fit
  while (a.G % a.parts != 0 || a.G / a.parts > DSPARK_PAGED_MAX_ROWS) ++a.parts;
  a.Gs = a.G / a.parts;
  const int fit = DSPARK_PAGED_MAX_ROWS / a.Gs;
  const int t_chunks = (max_new + fit - 1) / fit;
  a.t_chunk = (max_new + t_chunks - 1) / t_chunks;
  a.n_chunks = a.parts * t_chunks;
  if (a.n_chunks > sms) return DSPARK_ERR_INVALID_ARG;
  a.n_cols = (a.Gs * a.t_chunk + 15) / 16 * 16;
  a.table = block_table, a.ctx = context_len, a.row_off = row_off, a.out = out, a.lse = lse;
  a.v_cache = v_cache, a.stride = table_stride, a.page_stride = page_stride;
  a.token_stride = token_stride, a.head_stride = head_stride, a.B = B, a.n_tokens = n_tokens;
  a.Hq = Hq, a.Hkv = Hkv, a.max_new = max_new, a.num_pages = num_pages, a.max_pages = max_pages;
  while ((1 << a.shift) < page_size) ++a.shift;
  a.window = window > 0 ? window : INT_MAX;
  a.c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  a.records = reinterpret_cast<AttnRecord*>(ws);
  ws += DSPARK_ALIGN256(DSPARK_PAGED_MAX_CTAS * sizeof(AttnRecord));
  a.part_ml = reinterpret_cast<float*>(ws);
  ws += static_cast<size_t>(2 * DSPARK_PAGED_MAX_CTAS) * a.n_cols * 8;
  a.part_o = reinterpret_cast<float*>(ws);
  c.j.records = a.records, c.j.part_ml = a.part_ml, c.j.part_o = a.part_o, c.j.out = out;
  c.j.lse = lse, c.j.status = device_status, c.j.n_cols = a.n_cols, c.j.Hq = Hq, c.j.Gs = a.Gs;
  c.items = static_cast<int>(
      std::min<int64_t>(static_cast<int64_t>(B) * Hkv * a.n_chunks, DSPARK_PAGED_MAX_CTAS));
  c.stream = st;

  const bool f16 = dtype == DSPARK_F16;
  const cuuint64_t e = 2;
  const cuuint64_t qd[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq),
                            static_cast<cuuint64_t>(n_tokens)};
  const cuuint64_t qs[2] = {q_head_stride * e, q_row_stride * e};
  const cuuint32_t qb[3] = {64, static_cast<cuuint32_t>(a.Gs), static_cast<cuuint32_t>(a.t_chunk)};
  const cuuint64_t cd[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(page_size),
                            static_cast<cuuint64_t>(Hkv), static_cast<cuuint64_t>(num_pages)};
  const cuuint64_t cs[3] = {token_stride * e, head_stride * e, page_stride * e};
  const cuuint32_t cb[4] = {64, static_cast<cuuint32_t>(std::min(page_size, kTileTok)), 1, 1};
  if (!attn_map(&c.q, f16, q, 3, qd, qs, qb) || !attn_map(&c.k, f16, k_cache, 4, cd, cs, cb) ||
      !attn_map(&c.v, f16, v_cache, 4, cd, cs, cb))
    return DSPARK_ERR_INVALID_ARG;
  if (D == 64) return f16 ? attn_shape<64, true>(c, sms) : attn_shape<64, false>(c, sms);
  return f16 ? attn_shape<128, true>(c, sms) : attn_shape<128, false>(c, sms);
}
