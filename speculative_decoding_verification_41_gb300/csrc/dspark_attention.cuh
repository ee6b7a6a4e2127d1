// dspark_attention.cuh -- attention of each request's newest tokens over its
// pages (dspark_paged_attention, include/dspark_paged.h), sm_103a.
//
// Mathematics. For one request and one key head, R query rows (new tokens x
// query heads of the group) against L cached tokens, in tiles of 128 tokens:
//   S^T = K Q^T           (128 tokens x R rows, tcgen05, f32 in tensor memory)
//   P^T = 2^(c S^T - m)    (c = scale log2 e; m one reference per row)
//   O^T += V^T P^T         (D x R, tcgen05, f32 in tensor memory), l += sum P
// The tokens, of which there are many, are the 128 rows of the instruction and
// the query rows, of which there may be one, its N: a single new token costs
// N = 16 instead of a padded M = 128, and keys and values are used as they lie
// in the cache (K row by row, V as a transposed operand), so no tile is
// rearranged. A thread of the softmax warps owns one token of the tile and
// walks the rows: its weights P land in shared memory as 16-byte stores.
//
// The reference m of a row need not be its running maximum, only near it: a
// tile in which no score exceeds its row's m by 8 (a factor 2^8, which neither
// bf16 nor half precision nor the f32 sums mind) is used as it is, and that is
// one vote per tile instead of a maximum over 128 tokens for every row. Only
// when the vote fails (in a request's first tile, and rarely after it) are the
// maxima taken, m raised and O and l scaled.
//
// Bound. Every cached key and value is read once: 4 D bytes per token and key
// head against 4 D R flops, so up to R of about 280 the copy rate of HBM bounds
// the call. So: (1) a ring of TMA copies that runs ahead of the arithmetic
// across requests; (2) work split evenly over the CTAs whatever the lengths:
// all (request, head, tile) units form one line, CTA c of C takes units
// [cW/C, (c+1)W/C), found from the lengths on the device; a request cut by such
// a border leaves partial (m, l, O) rows that k_attention_join adds up in
// the order of the tiles, so results do not depend on timing.
//
// Warps: 0 copies (TMA), 1 issues the products, the others (one or two groups
// of four, which share the rows) do the softmax and write the results.
#pragma once

#include <climits>

#include "../../include/dspark_paged.h"
#include "dspark_tc.cuh"

namespace dspark {

constexpr int kTileTok = 128;
constexpr float kNoRef = 1e38f;  // minus the reference of a row that has seen no token yet
constexpr float kSlack = 8.f;    // how far (log2) a score may exceed its row's reference

struct AttnArgs {
  const int32_t* table;
  const int32_t* ctx;
  const int64_t* row_off;
  void* out;
  float* lse;
  const void* v_cache;  // for values that a row may not see (see odd_values)
  struct AttnRecord* records;
  float* part_ml;  // [slot][n_cols][2]
  float* part_o;   // [slot][n_cols][D]
  int64_t stride, page_stride, token_stride, head_stride;
  int32_t B, n_tokens, Hq, Hkv, G, Gs, parts, max_new, t_chunk, n_chunks, ctas, n_cols;
  int32_t shift, num_pages, max_pages, window;  // window INT_MAX: none
  float c;  // scale * log2(e)
};

// What CTA c leaves for the join: `first`..c cut one request's tokens among
// them and c has the last; rows of the request.
struct AttnRecord {
  int32_t valid, first, status, rows;
  int64_t row0;
  int32_t head0, lim0;
  int32_t pad[8];
};
static_assert(sizeof(AttnRecord) == 64, "AttnRecord layout");

// One piece of work: tiles [tile0, tile0 + tiles) of a request's key head.
struct AttnItem {
  int64_t row0;            // first row of q and out
  int32_t r, kv_head, head0;
  int32_t tiles, tile0;    // tiles = 0: no row sees a token
  int32_t t_rows;          // new tokens
  int32_t lim0;            // tokens that the first new token sees end here (exclusive)
  int32_t begin, end;      // tokens that some row sees
  int32_t starts, ends;    // has the request's first / last tile
  int32_t first;           // CTA with the request's first tile
  int32_t pad[2];
};
static_assert(sizeof(AttnItem) == 64, "AttnItem layout");

struct AttnReq {  // a request, as the partition sees it
  int64_t row0;
  int32_t units;  // per key head
  int32_t t_rows, lim0, begin, end;
};

__device__ __forceinline__ bool attn_request(const AttnArgs& a, int r, int t0, AttnReq& q) {
  const int64_t o0 = a.row_off[r], o1 = a.row_off[r + 1];
  const int32_t len = a.ctx[r];
  q.units = 0;
  const int64_t T = o1 - o0;
  if (o0 < 0 || T < 0 || T > a.max_new || o1 > a.n_tokens || len < 0 ||
      len > (static_cast<int64_t>(a.max_pages) << a.shift))
    return false;
  if (T <= t0) return true;
  q.row0 = o0 + t0;
  q.t_rows = min(a.t_chunk, static_cast<int32_t>(T) - t0);
  q.lim0 = len - static_cast<int32_t>(T) + t0 + 1;
  q.end = max(0, q.lim0 + q.t_rows - 1);
  q.begin = min(q.end, max(0, q.lim0 > a.window ? q.lim0 - a.window : 0));
  q.units = q.end > 0 ? (q.end + kTileTok - 1) / kTileTok - q.begin / kTileTok : 1;
  return true;
}

// ---------------------------------------------------------------------------
// PTX pieces
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            int z, int w, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_to(uint32_t dst, const CUtensorMap* map, int x, int y,
                                               int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
// 16 consecutive f32 columns of this thread's lane, complete on return
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void bar_sync(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
// barrier among n threads; true for all of them if any passed true
__device__ __forceinline__ bool bar_any(int id, int n, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(n), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void sts_u4(uint32_t addr, uint32_t x, uint32_t y, uint32_t z,
                                       uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z),
               "r"(w)
               : "memory");
}
__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool F16>
__device__ __forceinline__ float half_to_float(uint32_t bits16) {
  if constexpr (F16) {
    float f;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.f32.f16 %0, h;\n\t}"
        : "=f"(f)
        : "r"(bits16));
    return f;
  } else {
    return __uint_as_float(bits16 << 16);
  }
}
// Instruction descriptor: D f32; A and B both bf16 (1) or both f16 (0); ta, tb:
// the operand's rows are contiguous in memory instead of its K (transposed).
__host__ __device__ constexpr uint32_t attn_idesc(bool f16, int M, int N, bool ta, bool tb) {
  return (1u << 4) | ((f16 ? 0u : 1u) << 7) | ((f16 ? 0u : 1u) << 10) | ((ta ? 1u : 0u) << 15) |
         ((tb ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// Shared-memory descriptor without its start address: leading and stride byte
// offsets, swizzle (2: 128 bytes, 6: 32 bytes).
__host__ __device__ constexpr uint64_t attn_desc(uint32_t lbo, uint32_t sbo, uint32_t swizzle) {
  return (static_cast<uint64_t>(lbo >> 4) << 16) | (static_cast<uint64_t>(sbo >> 4) << 32) |
         (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(swizzle) << 61);
}
__device__ __forceinline__ uint64_t at(uint64_t desc, uint32_t saddr) {
  return desc | ((saddr >> 4) & 0x3FFFu);
}

// ---------------------------------------------------------------------------
// shapes
// ---------------------------------------------------------------------------
template <int D_, int NB_, int GROUPS_, int CTAS_, int STAGES_>
struct AttnShape {
  static constexpr int D = D_, NB = NB_, GROUPS = GROUPS_, CTAS = CTAS_, STAGES = STAGES_;
  static constexpr int THREADS = 64 + 128 * GROUPS;
  static constexpr int NC = NB / GROUPS;           // columns (rows of q) of a softmax group
  static constexpr int HALVES = D / 64;            // 128-byte wide slabs of a K, V or Q tile
  static constexpr uint32_t kSlab = kTileTok * 128;
  static constexpr uint32_t kStage = HALVES * kSlab;
  static constexpr uint32_t kQ = 0, kQBytes = HALVES * NB * 128;
  static constexpr uint32_t kP = kQ + kQBytes, kPBytes = NB / 16 * 4096;
  static constexpr uint32_t kRing = kP + kPBytes;
  static constexpr uint32_t kCtl = kRing + STAGES * kStage;
  static constexpr uint32_t kColS = 0, kColO = 2 * NB;
  static constexpr uint32_t kTmem = 3 * NB <= 64 ? 64 : 3 * NB <= 128 ? 128 : 3 * NB <= 256 ? 256 : 512;
};

template <class S>
struct AttnCtl {
  uint64_t full[S::STAGES], empty[S::STAGES];
  uint64_t q_full, q_empty, s_full[2], p_full, pv_done, item_full[2], item_empty[2], drained;
  uint32_t tmem;
  int32_t status, abort, odd_n;
  AttnItem item[2];
  alignas(16) float nref[S::NB];       // minus the rows' references
  alignas(16) int32_t lim[S::NB];      // a row sees the tokens below (and within the window)
  alignas(16) float fac[S::NB];        // a row's factor: of its sums, or of its result
  float red[4][S::NB];                 // per warp: maxima, sums
  int32_t odd[2 * S::NB];              // tokens whose values are not finite and not for all rows
  int64_t scan[S::THREADS / 32];
  int64_t u_total;
  int32_t start_r, start_off;
};

template <class S>
constexpr uint32_t attn_smem() {
  return S::kCtl + static_cast<uint32_t>(sizeof(AttnCtl<S>));
}

template <class S, bool F16>
__global__ void __launch_bounds__(S::THREADS, S::CTAS)
    k_attention(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  AttnCtl<S>& ctl = *reinterpret_cast<AttnCtl<S>*>(smem + S::kCtl);
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < S::STAGES; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.q_full, 1);
    mbar_init(&ctl.q_empty, 1);
    mbar_init(&ctl.p_full, 4 * S::GROUPS);
    mbar_init(&ctl.pv_done, 1);
    mbar_init(&ctl.drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.item_full[i], 1);
      mbar_init(&ctl.item_empty[i], 4 * S::GROUPS);
    }
    ctl.status = DSPARK_OK;
    ctl.abort = 0;
    ctl.odd_n = 0;
    fence_barrier_init();
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  if (warp == 1) {
    tmem_alloc(&ctl.tmem, S::kTmem);
    tmem_relinquish();
  }
  pdl_wait();  // predecessor grid complete, its writes visible
  pdl_trigger();

  // ---- this CTA's part of the line of units ------------------------------
  const int chunk = blockIdx.x % a.n_chunks, cta = blockIdx.x / a.n_chunks;
  const int part = chunk % a.parts, t0 = chunk / a.parts * a.t_chunk;
  {
    const int per = (a.B + S::THREADS - 1) / S::THREADS;
    const int r0 = min(tid * per, a.B), r1 = min(r0 + per, a.B);
    int64_t sum = 0;
    bool bad = false;
    AttnReq q;
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
      bad |= !attn_request(a, r, t0, q);
      sum += static_cast<int64_t>(q.units) * a.Hkv;
    }
    int64_t in = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xFFFFFFFFu, in, o);
      if (lane >= o) in += u;
    }
    if (lane == 31) ctl.scan[warp] = in;
    tc_fence_before();
    const int any_bad = __syncthreads_or(bad);
    tc_fence_after();
    int64_t before = in - sum, total = 0;
    for (int w = 0; w < S::THREADS / 32; ++w) {
      if (w < warp) before += ctl.scan[w];
      total += ctl.scan[w];
    }
    const int64_t g = min(static_cast<int64_t>(a.ctas), total);
    const int64_t u0 = cta < g ? cta * total / g : total;
    if (u0 >= before && u0 < before + sum) {
      int64_t u = before;
      for (int r = r0; r < r1; ++r) {
        attn_request(a, r, t0, q);
        const int64_t n = static_cast<int64_t>(q.units) * a.Hkv;
        if (u0 < u + n) {
          ctl.start_r = r;
          ctl.start_off = static_cast<int32_t>(u0 - u);
          break;
        }
        u += n;
      }
    }
    if (tid == 0) {
      ctl.u_total = total;
      if (any_bad) ctl.status = DSPARK_ERR_BAD_DATA;
    }
  }
  __syncthreads();
  const int64_t W = ctl.u_total;
  const int64_t g = min(static_cast<int64_t>(a.ctas), W);
  const int64_t u_begin = cta < g ? cta * W / g : W, u_end = cta < g ? (cta + 1) * W / g : W;
  const uint32_t tmem = ctl.tmem;
  const int id = chunk * a.ctas + cta;  // of the record and the partial slots
  if (tid == 0 && u_begin == u_end) a.records[id].valid = 0;

  if (warp == 0) {
    // =====================================================================
    // copies
    // =====================================================================
    if (u_begin < u_end) {
      const uint64_t policy = policy_evict_first();
      const int rows_box = min(1 << a.shift, kTileTok);
      const int n_box = kTileTok / rows_box;
      const int box = lane % n_box, half = lane / n_box;
      const bool copier = half < S::HALVES;
      const uint32_t q_bytes = S::HALVES * a.Gs * a.t_chunk * 128;
      int r = ctl.start_r, off = ctl.start_off;
      int64_t u = u_begin;
      // requests r_base .. r_base+31, one per lane
      int r_base = -1000;
      AttnReq mine{};
      AttnItem it{};
      int left = 0, tile = 0;  // tiles of the item that are not generated yet, the next one
      struct Gen {
        int tile, page;
        bool first, any, load;
      };
      bool done = false;
      // the next tile of the line (uniform over the warp but for page and load)
      auto next = [&](AttnItem& item) -> Gen {
        Gen n{0, 0, false, false, false};
        if (left == 0) {
          if (u >= u_end) {
            done = true;
            return n;
          }
          AttnReq q;
          for (;;) {
            if (r >= r_base + 32 || r < r_base) {
              r_base = r;
              mine.units = 0;
              if (r + lane < a.B) attn_request(a, r + lane, t0, mine);
            }
            const int src = r - r_base;
            q.units = __shfl_sync(0xFFFFFFFFu, mine.units, src);
            if (off < q.units * a.Hkv) {
              q.row0 = __shfl_sync(0xFFFFFFFFu, mine.row0, src);
              q.t_rows = __shfl_sync(0xFFFFFFFFu, mine.t_rows, src);
              q.lim0 = __shfl_sync(0xFFFFFFFFu, mine.lim0, src);
              q.begin = __shfl_sync(0xFFFFFFFFu, mine.begin, src);
              q.end = __shfl_sync(0xFFFFFFFFu, mine.end, src);
              break;
            }
            off -= q.units * a.Hkv;
            ++r;
            if (r >= a.B) {  // lengths changed under the call
              u = u_end;
              done = true;
              return n;
            }
          }
          const int h = off / q.units, in_head = off - h * q.units;
          const int take = static_cast<int>(
              min(static_cast<int64_t>(q.units - in_head), u_end - u));
          item.row0 = q.row0;
          item.r = r;
          item.kv_head = h;
          item.head0 = h * a.G + part * a.Gs;
          item.tiles = q.end > 0 ? take : 0;
          item.tile0 = q.begin / kTileTok + in_head;
          item.t_rows = q.t_rows;
          item.lim0 = q.lim0;
          item.begin = q.begin;
          item.end = q.end;
          item.starts = in_head == 0;
          item.ends = in_head + take == q.units;
          item.first = static_cast<int32_t>(((u - in_head + 1) * g - 1) / W);
          u += take;
          off += take;
          left = item.tiles;
          tile = item.tile0;
          n.first = true;
          if (left == 0) return n;
        }
        n.any = true;
        n.tile = tile;
        const int tok = tile * kTileTok + box * rows_box;
        n.load = copier && tok < item.end && tok + rows_box > item.begin;
        if (n.load)
          n.page = a.table[static_cast<int64_t>(item.r) * a.stride + (tok >> a.shift)];
        ++tile;
        --left;
        return n;
      };
      // one outcome for the warp, so that its lanes stay together
      auto all_wait = [](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity)) != 0;
      };
      uint32_t step = 0, items = 0, q_loads = 0;  // ring position; items and Q tiles so far
      bool ok = true;
      AttnItem cur_item{};
      Gen cur = next(it);
      cur_item = it;
      while (ok && (cur.first || cur.any)) {
        // the next tile's page ids are on their way while this one is copied
        Gen nxt = done ? Gen{0, 0, false, false, false} : next(it);
        if (cur.first) {
          const uint32_t slot = items & 1u;
          if (items >= 2) ok = all_wait(&ctl.item_empty[slot], ((items >> 1) - 1u) & 1u);
          if (!ok) break;
          if (lane == 0) {
            ctl.item[slot] = cur_item;
            mbar_arrive(&ctl.item_full[slot]);
          }
          ++items;
          if (cur.any) {
            if (q_loads >= 1) ok = all_wait(&ctl.q_empty, (q_loads - 1u) & 1u);
            if (!ok) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(&ctl.q_full, q_bytes);
              for (int s = 0; s < S::HALVES; ++s)
                tma_load_3d_to(sbase + S::kQ + s * S::NB * 128, &map_q, s * 64, cur_item.head0,
                               static_cast<int>(cur_item.row0), &ctl.q_full);
            }
            ++q_loads;
          }
        }
        if (cur.any) {
          int page = cur.page;
          const bool lost = cur.load && static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages);
          if (lost) {
            atomicCAS(&ctl.status, static_cast<int32_t>(DSPARK_OK),
                      static_cast<int32_t>(DSPARK_ERR_BAD_DATA));
            page = 0;
          }
          const uint32_t loads = __ballot_sync(0xFFFFFFFFu, cur.load);
          const uint32_t bytes = __popc(loads) * rows_box * 128;
          const int y = (cur.tile * kTileTok + box * rows_box) & ((1 << a.shift) - 1);
#pragma unroll
          for (int kv = 0; kv < 2 && ok; ++kv, ++step) {
            const uint32_t s = step % S::STAGES, use = step / S::STAGES;
            if (use >= 1) ok = all_wait(&ctl.empty[s], (use - 1u) & 1u);
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&ctl.full[s], bytes);
            __syncwarp();
            if (cur.load)
              tma_load_4d(sbase + S::kRing + s * S::kStage + half * S::kSlab + box * rows_box * 128,
                          kv == 0 ? &map_k : &map_v, half * 64, y, cur_item.kv_head, page,
                          &ctl.full[s], policy);
          }
        }
        cur = nxt;
        cur_item = it;
      }
      if (!ok) {
        set_status(&ctl.status, DSPARK_ERR_TIMEOUT);
        *reinterpret_cast<volatile int32_t*>(&ctl.abort) = 1;
      }
      // the end of the line
      if (ok) {
        const uint32_t slot = items & 1u;
        if (items >= 2) ok = all_wait(&ctl.item_empty[slot], ((items >> 1) - 1u) & 1u);
        if (ok && lane == 0) {
          ctl.item[slot].tiles = -1;
          mbar_arrive(&ctl.item_full[slot]);
        }
      }
      // leave no copy in flight into this CTA's shared memory
      for (uint32_t i = step > S::STAGES ? step - S::STAGES : 0; i < step; ++i)
        mbar_wait(&ctl.full[i % S::STAGES], (i / S::STAGES) & 1u);
      if (q_loads > 0) mbar_wait(&ctl.q_full, (q_loads - 1u) & 1u);
    }
  } else if (warp == 1) {
    // =====================================================================
    // products
    // =====================================================================
    if (lane == 0 && u_begin < u_end) {
      const uint32_t n = static_cast<uint32_t>(a.n_cols);
      const uint32_t idesc_s = attn_idesc(F16, kTileTok, n, false, false);
      const uint32_t idesc_o = attn_idesc(F16, S::D, n, true, true);
      // K and Q: rows of 128 bytes (64 elements), 8-row groups 1,024 bytes apart
      const uint64_t desc_kq = attn_desc(16, 1024, 2);
      // V: 64 elements of d contiguous per token, slabs of 64 apart, 8-token groups 1,024 apart
      const uint64_t desc_v = attn_desc(S::kSlab, 1024, 2);
      // P: 16 rows of q contiguous per token, 16-row blocks 4,096 apart, 8-token groups 256 apart
      const uint64_t desc_p = attn_desc(4096, 256, 6);
      uint32_t k_step = 0, items = 0, q_loads = 0, tiles = 0;  // ring position of the next K
      bool ok = true;
      auto product_s = [&]() {  // S^T of the next tile
        const uint32_t s = k_step % S::STAGES, buf = (k_step >> 1) & 1u;
        ok = mbar_wait(&ctl.full[s], (k_step / S::STAGES) & 1u);
        if (!ok) return;
        tc_fence_after();
        const uint32_t k0 = sbase + S::kRing + s * S::kStage, q0 = sbase + S::kQ;
#pragma unroll
        for (int k = 0; k < S::D / 16; ++k)
          tc_mma(tmem + S::kColS + buf * S::NB, at(desc_kq, k0 + (k / 4) * S::kSlab + (k % 4) * 32),
                 at(desc_kq, q0 + (k / 4) * S::NB * 128 + (k % 4) * 32), idesc_s, k > 0);
        tc_commit(&ctl.empty[s]);
        tc_commit(&ctl.s_full[buf]);
        k_step += 2;
      };
      while (ok) {
        const uint32_t slot = items & 1u;
        ok = mbar_wait(&ctl.item_full[slot], (items >> 1) & 1u);
        if (!ok) break;
        const int nt = ctl.item[slot].tiles;
        ++items;
        if (nt < 0) break;
        if (nt == 0) continue;
        ok = mbar_wait(&ctl.q_full, q_loads & 1u);
        ++q_loads;
        if (!ok) break;
        product_s();
        for (int i = 0; i < nt && ok; ++i) {
          if (i + 1 < nt) product_s();
          if (!ok) break;
          if (i == max(nt - 2, 0)) tc_commit(&ctl.q_empty);  // after the item's last S
          ok = mbar_wait(&ctl.p_full, tiles & 1u);
          if (!ok) break;
          const uint32_t v_step = 2 * tiles + 1, s = v_step % S::STAGES;
          ok = mbar_wait(&ctl.full[s], (v_step / S::STAGES) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint32_t v0 = sbase + S::kRing + s * S::kStage, p0 = sbase + S::kP;
#pragma unroll
          for (int k = 0; k < kTileTok / 16; ++k)
            tc_mma(tmem + S::kColO, at(desc_v, v0 + k * 2048), at(desc_p, p0 + k * 512), idesc_o,
                   i > 0 || k > 0);
          tc_commit(&ctl.empty[s]);
          tc_commit(&ctl.pv_done);
          ++tiles;
        }
      }
      if (!ok) {
        set_status(&ctl.status, DSPARK_ERR_TIMEOUT);
        *reinterpret_cast<volatile int32_t*>(&ctl.abort) = 1;
        tc_commit(&ctl.drained);  // no product may outlive the CTA
        mbar_wait(&ctl.drained, 0);
      }
    }
    __syncwarp();
  } else if (u_begin < u_end) {
    // =====================================================================
    // softmax, results
    // =====================================================================
    constexpr int kSoft = 128 * S::GROUPS;
    const int group = (warp - 2) >> 2, quarter = warp & 3;
    const int gt = (quarter << 5) | lane;  // this thread's token of a tile, and lane of S and O
    const int blocks = (a.n_cols / 16 + S::GROUPS - 1) / S::GROUPS;  // of 16 columns, per group
    const int c0 = group * blocks * 16;    // the group's first column
    const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;  // (32 * quarter) << 16
    const uint32_t window = static_cast<uint32_t>(a.window);
    volatile int32_t* abort_flag = &ctl.abort;
    uint32_t tiles = 0, items = 0;
    bool recorded = false;
    for (;;) {
      const uint32_t slot = items & 1u;
      bool failed = !mbar_wait(&ctl.item_full[slot], (items >> 1) & 1u);
      if (bar_any(1, kSoft, failed || *abort_flag != 0)) {
        failed = true;
        *abort_flag = 1;
        break;
      }
      const AttnItem it = ctl.item[slot];
      if (it.tiles < 0) break;
      ++items;
      const int rows = it.t_rows * a.Gs;
      const int my_rows = max(0, min(16 * blocks, rows - c0));
      const int nb = (my_rows + 15) >> 4;
      for (int j = c0 + gt; j < min(c0 + 16 * blocks, a.n_cols); j += 128) {
        // a column past the rows takes no part: all its scores are below its reference
        ctl.nref[j] = j < rows ? kNoRef : -INFINITY;
        ctl.lim[j] = j < rows ? it.lim0 + j / a.Gs : INT_MIN / 2;
      }
      if (tid == 64) ctl.odd_n = 0;
      bar_sync(1, kSoft);
      const int lim_last = it.lim0 + it.t_rows - 1;
      float l[S::NC];
#pragma unroll
      for (int j = 0; j < S::NC; ++j) l[j] = 0.f;

      bool leave = false;
      for (int i = 0; i < it.tiles; ++i, ++tiles) {
        const uint32_t buf = tiles & 1u;
        const int tok0 = (it.tile0 + i) * kTileTok, tok = tok0 + gt;
        // every token of the tile visible to every row?
        const bool whole = tok0 + kTileTok <= it.lim0 &&
                           (a.window == INT_MAX || tok0 >= lim_last - a.window);
        failed |= !mbar_wait(&ctl.s_full[buf], (tiles >> 1) & 1u);
        tc_fence_after();
        const uint32_t s_addr = tmem + lanes + S::kColS + buf * S::NB + c0;
        // the scores of columns j .. j+15, -inf where the row does not see the token
        auto scores = [&](int j, float (&x)[16]) {
          tmem_ld16(s_addr + j, x);
          if (!whole) {
            const int4* lim4 = reinterpret_cast<const int4*>(&ctl.lim[c0 + j]);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int4 m = lim4[k];
              if (static_cast<uint32_t>(m.x - 1 - tok) >= window) x[4 * k] = -INFINITY;
              if (static_cast<uint32_t>(m.y - 1 - tok) >= window) x[4 * k + 1] = -INFINITY;
              if (static_cast<uint32_t>(m.z - 1 - tok) >= window) x[4 * k + 2] = -INFINITY;
              if (static_cast<uint32_t>(m.w - 1 - tok) >= window) x[4 * k + 3] = -INFINITY;
            }
          }
        };
        auto exponents = [&](int j, float (&x)[16]) {
          scores(j, x);
          const float4* nr4 = reinterpret_cast<const float4*>(&ctl.nref[c0 + j]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 m = nr4[k];
            x[4 * k] = fmaf(x[4 * k], a.c, m.x);
            x[4 * k + 1] = fmaf(x[4 * k + 1], a.c, m.y);
            x[4 * k + 2] = fmaf(x[4 * k + 2], a.c, m.z);
            x[4 * k + 3] = fmaf(x[4 * k + 3], a.c, m.w);
          }
        };
        // With one block of columns the exponents stay in registers over the
        // vote; with more they are read from tensor memory again.
        float keep[16];
        float top = -INFINITY;
#pragma unroll
        for (int b = 0; b < S::NC / 16; ++b)
          if (b < nb) {
            exponents(16 * b, keep);
#pragma unroll
            for (int k = 0; k < 16; ++k) top = fmaxf(top, keep[k]);
          }
        const uint32_t prev = (tiles - 1u) & 1u;  // phase of the tile before, if there is one
        if (bar_any(1, kSoft, top > kSlack || failed)) {
#pragma unroll 1
          for (int b = 0; b < nb; ++b) {
            float x[16];
            scores(16 * b, x);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              // floats in the order of integers; NaN takes no part
              const int32_t f = __float_as_int(x[k] == x[k] ? x[k] : -INFINITY);
              const int32_t o = __reduce_max_sync(0xFFFFFFFFu, f ^ ((f >> 31) & 0x7FFFFFFF));
              if (lane == k)
                ctl.red[quarter][c0 + 16 * b + k] = __int_as_float(o ^ ((o >> 31) & 0x7FFFFFFF));
            }
          }
          if (bar_any(1, kSoft, failed || *abort_flag != 0)) {
            leave = true;
            break;
          }
          for (int j = c0 + gt; j < c0 + my_rows; j += 128) {
            const float m = a.c * fmaxf(fmaxf(ctl.red[0][j], ctl.red[1][j]),
                                        fmaxf(ctl.red[2][j], ctl.red[3][j]));
            const float old = -ctl.nref[j];
            ctl.fac[j] = m > old ? ex2_approx(old - m) : 1.f;
            if (m > old) ctl.nref[j] = -m;
          }
          bar_sync(1, kSoft);
          if (i > 0) {
            failed |= !mbar_wait(&ctl.pv_done, prev);
            tc_fence_after();
          }
#pragma unroll
          for (int b = 0; b < S::NC / 16; ++b)
            if (b < nb) {
              float f[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                const int j = 16 * b + k;
                f[k] = j < my_rows ? ctl.fac[c0 + j] : 1.f;
                l[j] *= f[k];
              }
              if (i > 0) {
                float o[16];
                tmem_ld16(tmem + lanes + S::kColO + c0 + 16 * b, o);
#pragma unroll
                for (int k = 0; k < 16; ++k) o[k] *= f[k];
                tmem_st16(tmem + lanes + S::kColO + c0 + 16 * b, o);
              }
              if constexpr (S::NC == 16) exponents(0, keep);
            }
          tmem_wait_st();
        }
        // P is free once the tile before it has been multiplied
        if (tiles > 0) failed |= !mbar_wait(&ctl.pv_done, prev);
#pragma unroll
        for (int b = 0; b < S::NC / 16; ++b)
          if (b < nb) {
            if constexpr (S::NC > 16) exponents(16 * b, keep);
            uint32_t p[8];
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float p0 = ex2_approx(keep[k]), p1 = ex2_approx(keep[k + 1]);
              l[16 * b + k] += p0;
              l[16 * b + k + 1] += p1;
              // The weights enter the second product in the inputs' type (half
              // a step of it each, the step at most that of the output); their
              // sum l is of the unrounded ones, whose errors do not add up.
              p[k / 2] = pack2<F16>(p0, p1);
            }
            const uint32_t row = sbase + S::kP + ((c0 >> 4) + b) * 4096 + gt * 32;
            const uint32_t swap = (gt & 4) << 2;  // 32-byte swizzle
            sts_u4(row + swap, p[0], p[1], p[2], p[3]);
            sts_u4(row + (swap ^ 16u), p[4], p[5], p[6], p[7]);
          }
        if (!whole && group == 0) {
          // Zero weights do not silence values that are not finite, and the
          // tile's rest may hold anything: what no row sees is zeroed, and of
          // what only some rows see the non-finite values are taken out here
          // and added to those rows at the end.
          const bool some = tok >= it.begin && tok < it.end;
          const bool all = tok < it.lim0 && (a.window == INT_MAX || tok >= lim_last - a.window);
          const uint32_t v_step = 2 * tiles + 1, s = v_step % S::STAGES;
          failed |= !mbar_wait(&ctl.full[s], (v_step / S::STAGES) & 1u);
          const uint32_t v_row = sbase + S::kRing + s * S::kStage + gt * 128;
          if (!some) {
#pragma unroll
            for (int q = 0; q < S::HALVES; ++q)
#pragma unroll
              for (int k = 0; k < 8; ++k) sts_u4(v_row + q * S::kSlab + k * 16, 0, 0, 0, 0);
          } else if (!all) {
            bool odd = false;
            constexpr uint32_t kExp = F16 ? 0x7C00u : 0x7F80u;
            for (int k = 0; k < 8 * S::HALVES; ++k) {
              const uint32_t addr = v_row + (k >> 3) * S::kSlab + (k & 7) * 16;
              const uint4 v = lds_u4(addr);
              uint32_t w[4] = {v.x, v.y, v.z, v.w};
              bool hit = false;
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                if ((w[q] & kExp) == kExp) w[q] &= 0xFFFF0000u, hit = true;
                if (((w[q] >> 16) & kExp) == kExp) w[q] &= 0x0000FFFFu, hit = true;
              }
              if (hit) sts_u4(addr, w[0], w[1], w[2], w[3]);
              odd |= hit;
            }
            if (odd) ctl.odd[atomicAdd(&ctl.odd_n, 1)] = tok;
          }
        }
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full);
      }
      if (leave) {
        failed = true;
        *abort_flag = 1;
        break;
      }

      // ---- the item's rows ----------------------------------------------
      const bool alone = it.starts && it.ends;
      const int64_t part_row = static_cast<int64_t>(2 * id + (it.starts ? 1 : 0)) * a.n_cols;
      if (it.tiles > 0) {
        failed |= !mbar_wait(&ctl.pv_done, (tiles - 1u) & 1u);
        tc_fence_after();
      }
#pragma unroll
      for (int b = 0; b < S::NC / 16; ++b)
        if (b < nb) {
          // sums over the warp's 32 tokens: halve the columns, double the tokens
#pragma unroll
          for (int h = 8, o = 16; h >= 1; h >>= 1, o >>= 1) {
            const bool upper = (lane & o) != 0;
#pragma unroll
            for (int k = 0; k < h; ++k) {
              const float give = upper ? l[16 * b + k] : l[16 * b + k + h];
              const float have = upper ? l[16 * b + k + h] : l[16 * b + k];
              l[16 * b + k] = have + __shfl_xor_sync(0xFFFFFFFFu, give, o);
            }
          }
          l[16 * b] += __shfl_xor_sync(0xFFFFFFFFu, l[16 * b], 1);
          if ((lane & 1) == 0) ctl.red[quarter][c0 + 16 * b + (lane >> 1)] = l[16 * b];
        }
      if (bar_any(1, kSoft, failed || *abort_flag != 0)) {
        failed = true;
        *abort_flag = 1;
        break;
      }
      for (int j = c0 + gt; j < c0 + my_rows; j += 128) {
        const float sum = (ctl.red[0][j] + ctl.red[1][j]) + (ctl.red[2][j] + ctl.red[3][j]);
        const float m = -ctl.nref[j];
        if (alone) {
          const bool seen = ctl.lim[j] > 0;
          ctl.fac[j] = 1.f / sum;
          if (a.lse)
            a.lse[(it.row0 + j / a.Gs) * a.Hq + it.head0 + j % a.Gs] =
                seen ? (m + log2f(sum)) * 0.69314718055994531f : -INFINITY;
        } else {
          reinterpret_cast<float2*>(a.part_ml)[part_row + j] = make_float2(m, sum);
        }
      }
      bar_sync(1, kSoft);
      const int odd_n = ctl.odd_n;
      const bool writer = S::D == 128 || lane < 16;  // M = 64 fills 16 lanes of each warp's 32
      const int d = S::D == 128 ? gt : quarter * 16 + lane;
      int t = c0 / a.Gs, h = c0 % a.Gs;
#pragma unroll 1
      for (int b = 0; b < nb; ++b) {
        float o[16];
        if (it.tiles > 0) {
          tmem_ld16(tmem + lanes + S::kColO + c0 + 16 * b, o);
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int j = c0 + 16 * b + k;
          if (j < c0 + my_rows && writer) {
            const int lim = ctl.lim[j];
            float v = o[k];
            for (int q = 0; q < odd_n; ++q) {
              const int u = ctl.odd[q];
              if (static_cast<uint32_t>(lim - 1 - u) >= window) continue;
              const int32_t page = a.table[it.r * a.stride + (u >> a.shift)];
              if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) continue;
              const uint16_t bits = static_cast<const uint16_t*>(a.v_cache)[
                  page * a.page_stride + (u & ((1 << a.shift) - 1)) * a.token_stride +
                  it.kv_head * a.head_stride + d];
              constexpr uint32_t kExp = F16 ? 0x7C00u : 0x7F80u;
              if ((bits & kExp) == kExp) v += half_to_float<F16>(bits);
            }
            if (alone) {
              v = lim > 0 ? v * ctl.fac[j] : 0.f;
              const uint32_t w = pack2<F16>(v, 0.f);
              static_cast<uint16_t*>(a.out)[((it.row0 + t) * a.Hq + it.head0 + h) * S::D + d] =
                  static_cast<uint16_t>(w);
            } else {
              a.part_o[(part_row + j) * S::D + d] = v;
            }
          }
          if (++h == a.Gs) h = 0, ++t;
        }
      }
      if (it.ends && !it.starts) {
        recorded = true;
        if (tid == 64) {
          AttnRecord& rec = a.records[id];
          rec.valid = 1;
          rec.first = it.first;
          rec.rows = rows;
          rec.row0 = it.row0;
          rec.head0 = it.head0;
          rec.lim0 = it.lim0;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl.item_empty[slot]);
    }
    if (!recorded && tid == 64) a.records[id].valid = 0;
    if (*abort_flag != 0 && tid == 64) set_status(&ctl.status, DSPARK_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, S::kTmem);
  if (tid == 0) a.records[id].status = ctl.status;
}

// ---------------------------------------------------------------------------
// the rows of requests that were cut between CTAs
// ---------------------------------------------------------------------------
// Block (x, y) takes the x-th cut request and kJoinWarps / per_row of its rows;
// per_row warps share a row's pieces. Sums run in the order of the tiles.
constexpr int kJoinWarps = 8;

struct JoinArgs {
  const AttnRecord* records;
  const float* part_ml;
  const float* part_o;
  void* out;
  float* lse;
  int32_t* status;
  int32_t n, ctas, n_cols, Hq, Gs, per_row;
};

template <int D, bool F16>
__global__ void __launch_bounds__(kJoinWarps * 32) k_attention_join(const JoinArgs a) {
  __shared__ uint32_t s_valid[(DSPARK_PAGED_MAX_CTAS + 31) / 32], s_bad[(DSPARK_PAGED_MAX_CTAS + 31) / 32];
  __shared__ float s_acc[kJoinWarps][D];
  __shared__ float s_sum[kJoinWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  const int words = (a.n + 31) / 32;
  for (int w = warp; w < words; w += kJoinWarps) {
    const int i = w * 32 + lane;
    const bool in = i < a.n;
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, in && a.records[i].valid != 0);
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, in && a.records[i].status != DSPARK_OK);
    if (lane == 0) s_valid[w] = v, s_bad[w] = b;
  }
  __syncthreads();
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) {
    int32_t st = DSPARK_OK;
    for (int w = 0; w < words && st == DSPARK_OK; ++w)
      if (s_bad[w]) st = a.records[w * 32 + __ffs(s_bad[w]) - 1].status;
    *a.status = st;
  }
  int want = blockIdx.x, id = -1;
  for (int w = 0; w < words; ++w) {
    const int c = __popc(s_valid[w]);
    if (want < c) {
      uint32_t m = s_valid[w];
      for (; want > 0; --want) m &= m - 1u;
      id = w * 32 + __ffs(m) - 1;
      break;
    }
    want -= c;
  }
  if (id < 0) return;
  const AttnRecord rec = a.records[id];
  const int chunk0 = id / a.ctas * a.ctas, pieces = id - chunk0 - rec.first + 1;
  const int row = blockIdx.y * (kJoinWarps / a.per_row) + warp / a.per_row;
  const int sub = warp % a.per_row;
  constexpr int V = D / 32;  // floats per lane
  float acc[V], sum = 0.f, top = -INFINITY;
#pragma unroll
  for (int k = 0; k < V; ++k) acc[k] = 0.f;
  auto slot = [&](int k) {
    return (2 * static_cast<int64_t>(chunk0 + rec.first + k) + (k == 0 ? 1 : 0)) * a.n_cols + row;
  };
  const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
  if (row < rec.rows) {
    for (int k = lane; k < pieces; k += 32) top = fmaxf(top, ml[slot(k)].x);
    top = warp_max(top);
#pragma unroll 4
    for (int k = sub; k < pieces; k += a.per_row) {
      const int64_t s = slot(k);
      const float2 p = ml[s];
      const float w = ex2_approx(p.x - top);
      sum = fmaf(w, p.y, sum);
      const float* o = a.part_o + s * D + lane * V;
#pragma unroll
      for (int q = 0; q < V; ++q) acc[q] = fmaf(w, o[q], acc[q]);
    }
  }
  if (a.per_row > 1) {
#pragma unroll
    for (int q = 0; q < V; ++q) s_acc[warp][lane * V + q] = acc[q];
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    if (sub == 0)
      for (int w = 1; w < a.per_row; ++w) {
        sum += s_sum[warp + w];
#pragma unroll
        for (int q = 0; q < V; ++q) acc[q] += s_acc[warp + w][lane * V + q];
      }
  }
  if (row < rec.rows && sub == 0) {
    const bool seen = rec.lim0 + row / a.Gs > 0;
    const int64_t at = (rec.row0 + row / a.Gs) * a.Hq + rec.head0 + row % a.Gs;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at * D + lane * V);
    const float inv = 1.f / sum;
#pragma unroll
    for (int q = 0; q < V; q += 2)
      out[q / 2] = seen ? pack2<F16>(acc[q] * inv, acc[q + 1] * inv) : 0u;
    if (a.lse && lane == 0) a.lse[at] = seen ? (top + log2f(sum)) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace dspark
