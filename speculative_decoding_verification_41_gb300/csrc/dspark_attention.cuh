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
// The reference m of a row need not be its running maximum: any m with 2^(c s - m)
// in range for every score s serves, and one that lies a whole number of powers of
// two from some score keeps that score's weight free of rounding. A tile whose
// scores exceed their rows' references by no more than kHighest (log2) is used as
// it is: that is one vote per tile instead of a maximum over 128 tokens for every
// row. A row starts with its maximum over the first tile (a score of one token
// would do for the range of bf16, and costs as much, but leaves the largest weight
// a rounding that a power of two has not: 1.5 times the output's own rounding error
// in all, against 1.1 to 1.3). When a vote fails, the maxima are taken, m raised
// and O and l scaled.
//
// Bound. Every cached key and value is read once: 4 D bytes per token and key
// head against 4 D R flops, so up to R of about 280 the copy rate of HBM bounds
// the call. So: (1) a ring of TMA copies that runs ahead of the arithmetic
// across requests; (2) work split evenly over the CTAs whatever the lengths:
// all (request, head) items form one line, each as long as its tiles and `lead`
// more for what it costs to begin and end one; CTA c of C takes [cW/C, (c+1)W/C)
// of it, found from the lengths on the device; a request cut by such a border
// leaves partial (m, l, O) rows that k_attention_join adds up in the order of
// the tiles, so results do not depend on timing.
//
// Warps: 0 copies keys, 1 values, 3 queries (TMA), 2 issues the products; from
// the fifth on groups of four, which share the rows among them, do the softmax
// and write the results. S and P have two buffers each (P of the widest block
// one): while a group is at a tile's exponents the products of the next scores
// and of the weights before are under way.
#pragma once

#include <cfloat>
#include <climits>

#include "../../include/dspark_paged.h"
#include "dspark_tc.cuh"

namespace dspark {

constexpr int kTileTok = 128;
constexpr float kNoRef = 1e38f;  // minus the reference of a row that has seen no token yet
// Exponents (log2) of a row's weights: the largest one when its reference is set
// (kBase), and the largest before it is raised (kHighest). Half precision ends at
// 2^16 and has its full 11 bits down to 2^-14, so its weights use the upper end: with a
// largest weight of 1 a row with one token 17 nats above 2,000 others lost 3% of
// their sum in the second product and none of it in l. Seven powers of two of room
// seldom need a raise (136 rows, scores of 2 nats' deviation: 1% of the time, against
// 13% with four), and weights down to 2^-23 of the largest keep their bits. A row
// with a peak, a tile's maximum far above one of its four quarters' (kPeak), is the
// one that needs more, and the one whose maximum is not likely to grow: its weights
// keep theirs down to 2^-28. bf16 has the range of binary32, which the sums of
// weights times values must not leave where the values themselves are near its end:
// no weight exceeds 1, and the room lies below.
template <bool F16>
constexpr float kBase = F16 ? 9.f : -8.f;
template <bool F16>
constexpr float kPeakBase = F16 ? 14.f : -8.f;
constexpr float kPeak = 8.f;
template <bool F16>
constexpr float kHighest = F16 ? 15.9f : 0.f;
// Rows of few, with many tiles to come, take every new maximum: a largest weight
// that is a power of two has no rounding, and the output is off by 1.1 to 1.2 times
// its own rounding (1.25 to 1.4 with the room above). New maxima grow rare along a
// context, and a block of up to 16 rows waits for memory anyway; short pieces and
// wider blocks would pay (measured: a tenth for 9 tiles, 3% for 32 rows, a fifth
// for 64).
constexpr int kExactRows = 16, kExactTiles = 16;
template <bool F16>
constexpr float kExactBase = F16 ? 15.f : 0.f;
// A maximum of this size or more is the reference itself: its product with c is
// rounded to a 64th or less finely, and the room above kBase has to hold that too.
constexpr float kNoShift = 262144.f;

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
  int32_t lead;     // length of an item besides its tiles
  int32_t q_bufs;   // tiles of queries
  int32_t k_stages, v_stages;  // tiles of keys and of values in the rings
  uint32_t p_off, p_bytes, ring_off;  // shared memory: weights, rings
  float c;  // scale * log2(e)
};

// What CTA c leaves for the join: `first`..c cut one request's tokens among
// them and c has the last; rows of the request.
struct AttnRecord {
  int32_t valid, first, status, rows;
  int64_t row0;
  int32_t head0, lim0;
};
static_assert(sizeof(AttnRecord) == 32, "AttnRecord layout");

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
  int32_t units;  // length of the item of a key head; 0: no rows
  int32_t t_rows, lim0, begin, end;
};

// The line of all units, cut into one part per CTA: the first `more` parts are
// one unit longer. CTAs past `parts` have none.
constexpr uint32_t kMaxUnits = INT_MAX;
struct Line {
  uint32_t units = 0, parts = 0, per = 0, more = 0;
  __device__ Line() {}
  __device__ Line(uint32_t n, int ctas) : units(n) {
    parts = min(n, static_cast<uint32_t>(ctas));
    if (parts > 0) per = n / parts, more = n - per * parts;
  }
  __device__ uint32_t begin(uint32_t c) const {
    return c >= parts ? units : c * per + min(c, more);
  }
  __device__ int32_t owner(uint32_t u) const {  // of unit u
    const uint32_t longer = more * (per + 1u);
    return static_cast<int32_t>(u < longer ? u / (per + 1u) : more + (u - longer) / per);
  }
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
  // an item without tiles still has rows to write: it counts as one
  q.units = a.lead + (q.end > 0 ? (q.end + kTileTok - 1) / kTileTok - q.begin / kTileTok : 1);
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
__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}
__device__ __forceinline__ void tma_load_3d_to(uint32_t dst, const CUtensorMap* map, int x, int y,
                                               int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
      : "memory");
}
// 8 consecutive f32 columns of this thread's lane; the values are there after
// tmem_arrived() on them.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// Ties the values of a load to a wait before this statement.
__device__ __forceinline__ void tmem_arrived(float* v) {
  asm volatile(""
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
      : "memory");
}
// Sum or maximum of 8 columns over lanes 4 apart: each step halves the columns
// a lane holds and doubles the lanes they stand for. Lane i returns its part of
// column i / 4.
template <bool MAX>
__device__ __forceinline__ float fold_columns(float (&v)[8], int lane) {
#pragma unroll
  for (int h = 4, o = 16; h >= 1; h >>= 1, o >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int k = 0; k < h; ++k) {
      const float give = upper ? v[k] : v[k + h], have = upper ? v[k + h] : v[k];
      const float got = __shfl_xor_sync(0xFFFFFFFFu, give, o);
      v[k] = MAX ? fmaxf(have, got) : have + got;
    }
  }
  return v[0];
}
// ... and over the four lanes of a column.
template <bool MAX>
__device__ __forceinline__ float over_four(float v) {
#pragma unroll
  for (int o = 2; o >= 1; o >>= 1) {
    const float got = __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = MAX ? fmaxf(v, got) : v + got;
  }
  return v;
}
// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}
// A wait of a whole warp: one outcome, so that its lanes stay together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity)) != 0;
}
// Whether a phase is complete, without waiting; one outcome for the warp.
__device__ __forceinline__ bool warp_test(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return __all_sync(0xFFFFFFFFu, done) != 0;
}
// Pairs of floats: one instruction for two of them.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
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
// m + log2(sum): the sum's exponent joins m, whose opposite it nearly is where the
// reference lies far from the row's largest score.
__device__ __forceinline__ float plus_log2(float m, float sum) {
  const uint32_t bits = __float_as_uint(sum);
  const int e = static_cast<int>(bits >> 23) - 127;
  if (!(sum >= FLT_MIN && sum <= FLT_MAX)) return m + log2f(sum);
  return (m + static_cast<float>(e)) + log2f(__uint_as_float(bits - (static_cast<uint32_t>(e) << 23)));
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
constexpr int kMaxStages = 12;
constexpr uint32_t kItems = 4;  // items planned ahead of their use, at most

template <int D_, int NB_, int GROUPS_, int CTAS_, int PBUFS_>
struct AttnShape {
  static constexpr int D = D_, NB = NB_, GROUPS = GROUPS_, CTAS = CTAS_;
  static constexpr int PBUFS = PBUFS_;          // buffers of weights
  static constexpr int THREADS = 128 + 128 * GROUPS;
  static constexpr int NC = (NB / 8 + GROUPS - 1) / GROUPS * 8;  // columns of a softmax group
  static constexpr int HALVES = D / 64;         // 128-byte wide slabs of a K, V or Q tile
  static constexpr uint32_t kSlab = kTileTok * 128;
  static constexpr uint32_t kStage = HALVES * kSlab;
  static constexpr uint32_t kColS = 0, kColO = 2 * NB;
  static constexpr uint32_t kTmem = 3 * NB <= 64 ? 64 : 3 * NB <= 128 ? 128 : 3 * NB <= 256 ? 256 : 512;
};

template <class S>
struct AttnCtl {
  uint64_t full[kMaxStages], empty[kMaxStages];  // of key tiles, then of value tiles
  uint64_t q_full[2], q_empty[2], s_full[2], p_full[2], pv_done[2];
  uint64_t item_full[kItems], item_empty[kItems];
  uint64_t odd_full, drained;
  uint32_t tmem;
  int32_t status, abort, start_r, start_off;
  uint32_t scan[S::THREADS / 32];
  AttnItem item[kItems];
  // per column (row of q); a group's own. Two of what an item begins with: its
  // slower warps may still write their results when the next one begins.
  alignas(16) float nref[2][S::NB + 8];   // minus the rows' references
  alignas(16) int32_t lim[2][S::NB + 8];  // a row sees the tokens below (and within the window)
  alignas(16) int32_t at[S::NB + 8];      // element of a row in out, from the item's first
  alignas(16) float fac[S::NB + 8];       // factor of a row's sums when its reference rises
  int32_t new_tok[S::NB + 8];             // new token of a column
  float red[4][S::NB + 8];                // per warp: maxima, sums
  int32_t odd_n[2], odd[2][2 * S::NB];  // tokens whose values are not finite and not for all rows
};

template <class S>
constexpr uint32_t kCtlBytes = (static_cast<uint32_t>(sizeof(AttnCtl<S>)) + 1023u) & ~1023u;

template <class S, bool F16>
__global__ void __launch_bounds__(S::THREADS, S::CTAS)
    k_attention(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                const __grid_constant__ CUtensorMap map_v, const __grid_constant__ AttnArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  AttnCtl<S>& ctl = *reinterpret_cast<AttnCtl<S>*>(smem);
  const uint32_t s_q = smem_addr(smem) + kCtlBytes<S>;  // Q; then weights, ring
  const uint32_t s_p = smem_addr(smem) + a.p_off, s_ring = smem_addr(smem) + a.ring_off;
  const uint32_t q_slab = a.n_cols * 128u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < a.k_stages + a.v_stages; ++i) {
      mbar_init(&ctl.full[i], 1);
      mbar_init(&ctl.empty[i], 1);
    }
    mbar_init(&ctl.odd_full, 1);
    mbar_init(&ctl.drained, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl.q_full[i], 1);
      mbar_init(&ctl.q_empty[i], 1);
      mbar_init(&ctl.s_full[i], 1);
      mbar_init(&ctl.p_full[i], 4 * S::GROUPS);
      mbar_init(&ctl.pv_done[i], 1);
    }
    for (uint32_t i = 0; i < kItems; ++i) {
      mbar_init(&ctl.item_full[i], 1);
      mbar_init(&ctl.item_empty[i], 4 * S::GROUPS + 2);  // softmax warps, products, queries
    }
    ctl.status = DSPARK_OK;
    ctl.abort = 0;
    fence_barrier_init();
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  if (warp == 2) {
    tmem_alloc(&ctl.tmem, S::kTmem);
    tmem_relinquish();
  }
  pdl_wait();  // predecessor grid complete, its writes visible
  pdl_trigger();

  // ---- this CTA's part of the line of units ------------------------------
  int chunk = 0, cta = blockIdx.x, part = 0, t0 = 0;
  if (a.n_chunks > 1) {
    chunk = blockIdx.x % a.n_chunks, cta = blockIdx.x / a.n_chunks;
    part = chunk % a.parts, t0 = chunk / a.parts * a.t_chunk;
  }
  Line line;
  {
    const int per = (a.B + S::THREADS - 1) / S::THREADS;  // requests per thread
    const int r0 = min(tid * per, a.B), r1 = min(r0 + per, a.B);
    uint32_t sum = 0;
    bool bad = false;
    AttnReq q{};
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
      bad |= !attn_request(a, r, t0, q);
      sum = min(sum + static_cast<uint32_t>(q.units * a.Hkv), kMaxUnits);
    }
    uint32_t in = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, in, o);
      if (lane >= o) in = min(in + u, kMaxUnits);
    }
    if (lane == 31) ctl.scan[warp] = in;
    tc_fence_before();
    const int any_bad = __syncthreads_or(bad);
    tc_fence_after();
    uint32_t before = in - sum, total = 0;
#pragma unroll
    for (int w = 0; w < S::THREADS / 32; ++w) {
      const uint32_t v = ctl.scan[w];
      if (w < warp) before = min(before + v, kMaxUnits);
      total = min(total + v, kMaxUnits);
    }
    line = Line(total < kMaxUnits ? total : 0u, a.ctas);
    const uint32_t u0 = line.begin(cta);
    if (u0 >= before && u0 < before + sum) {
      uint32_t u = before;
      for (int r = r0; r < r1; ++r) {
        if (per > 1) attn_request(a, r, t0, q);
        const uint32_t n = static_cast<uint32_t>(q.units * a.Hkv);
        if (u0 < u + n) {
          ctl.start_r = r;
          ctl.start_off = static_cast<int32_t>(u0 - u);
          break;
        }
        u += n;
      }
    }
    if (tid == 0) {
      if (total == kMaxUnits) ctl.status = DSPARK_ERR_TOO_LARGE;
      if (any_bad) ctl.status = DSPARK_ERR_BAD_DATA;
    }
  }
  __syncthreads();
  const uint32_t u_begin = line.begin(cta), u_end = line.begin(cta + 1);
  const uint32_t tmem = ctl.tmem;
  const int id = chunk * a.ctas + cta;  // of the record and the partial slots
  if (tid == 0 && u_begin == u_end) a.records[id].valid = 0;

  if (warp < 2) {
    // =====================================================================
    // copies: warp 0 keys and the items' records, warp 1 values. A
    // tile's copies cost a warp some fifty instructions, which share the SM's
    // issue slots with the softmax: with both kinds in one warp and page ids
    // fetched tile by tile the copies fell behind the memory.
    // =====================================================================
    if (u_begin < u_end) {
      const bool keys = warp == 0;
      const uint64_t policy = policy_evict_first();
      const int rows_box = min(1 << a.shift, kTileTok);
      const int n_box = kTileTok / rows_box;
      const int box = lane % n_box, half = lane / n_box;
      const bool copier = half < S::HALVES;
      const uint32_t box_bytes = rows_box * 128;
      const uint32_t first_stage = keys ? 0u : static_cast<uint32_t>(a.k_stages);
      const uint32_t end_stage =
          keys ? static_cast<uint32_t>(a.k_stages) : static_cast<uint32_t>(a.k_stages + a.v_stages);
      const CUtensorMap* const map = keys ? &map_k : &map_v;
      const uint32_t dst0 = s_ring + half * S::kSlab + box * box_bytes;
      int r = ctl.start_r, off = ctl.start_off;
      uint32_t u = u_begin;
      // requests r_base .. r_base+31, one per lane
      int r_base = -1000;
      AttnReq mine{};
      uint32_t items = 0, s = first_stage, wraps = 0;
      bool ok = true;
      while (ok) {
        // ---- the next item of the line
        AttnReq q;
        int h = 0, lead_in = 0, take = 0;
        bool found = false;
        while (u < u_end && r < a.B) {  // (r: lengths that changed under the call)
          if (r >= r_base + 32 || r < r_base) {
            r_base = r;
            mine.units = 0;
            mine.begin = 0;
            if (r + lane < a.B) {
              attn_request(a, r + lane, t0, mine);
              if (mine.units > 0)  // the table rows of requests to come
                prefetch_l2(a.table + (r + lane) * a.stride + (mine.begin >> a.shift));
            }
          }
          const int src = r - r_base;
          q.units = __shfl_sync(0xFFFFFFFFu, mine.units, src);
          if (off >= q.units * a.Hkv) {
            off -= q.units * a.Hkv;
            ++r;
            continue;
          }
          h = off / q.units;
          lead_in = off - h * q.units;
          take = static_cast<int>(min(static_cast<uint32_t>(q.units - lead_in), u_end - u));
          u += take;
          off += take;
          if (lead_in + take > a.lead) {
            q.row0 = __shfl_sync(0xFFFFFFFFu, mine.row0, src);
            q.t_rows = __shfl_sync(0xFFFFFFFFu, mine.t_rows, src);
            q.lim0 = __shfl_sync(0xFFFFFFFFu, mine.lim0, src);
            q.begin = __shfl_sync(0xFFFFFFFFu, mine.begin, src);
            q.end = __shfl_sync(0xFFFFFFFFu, mine.end, src);
            found = true;
            break;
          }  // else nothing but the item's lead: the next CTA begins it
        }
        if (!found) break;
        const int in_head = max(lead_in - a.lead, 0);
        const int tile0 = q.begin / kTileTok + in_head;
        const int tiles = q.end > 0 ? lead_in + take - a.lead - in_head : 0;
        const int32_t* const row = a.table + r * a.stride;
        const int last_page = max(q.end - 1, 0) >> a.shift;
        int page0 = (tile0 * kTileTok) >> a.shift;  // of the 32 ids that the lanes hold
        int ids = 0, next_ids = 0;
        if (tiles > 0) ids = row[min(page0 + lane, last_page)];
        if (keys) {
          const uint32_t slot = items % kItems, use = items / kItems;
          if (use >= 1) ok = warp_wait(&ctl.item_empty[slot], (use - 1u) & 1u);
          if (!ok) break;
          if (lane == 0) {
            AttnItem& item = ctl.item[slot];
            item.row0 = q.row0;
            item.r = r;
            item.kv_head = h;
            item.head0 = h * a.G + part * a.Gs;
            item.tiles = tiles;
            item.tile0 = tile0;
            item.t_rows = q.t_rows;
            item.lim0 = q.lim0;
            item.begin = q.begin;
            item.end = q.end;
            item.starts = in_head == 0;
            item.ends = lead_in + take == q.units;
            item.first = line.owner(u - take - lead_in + a.lead);
            mbar_arrive(&ctl.item_full[slot]);
          }
          ++items;
        }
        // ---- its tiles
        if (tiles > 0) next_ids = row[min(page0 + 32 + lane, last_page)];
        int tok = tile0 * kTileTok + box * rows_box;  // this lane's box of the tile
        for (int i = 0; i < tiles; ++i, tok += kTileTok) {
          int rel = (tok >> a.shift) - page0;
          if (__any_sync(0xFFFFFFFFu, rel >= 32)) {
            page0 += 32;
            rel -= 32;
            ids = next_ids;
            next_ids = row[min(page0 + 32 + lane, last_page)];
          }
          int page = __shfl_sync(0xFFFFFFFFu, ids, rel);
          const bool load = copier && tok < q.end && tok + rows_box > q.begin;
          if (load && static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages)) {
            set_status(&ctl.status, DSPARK_ERR_BAD_DATA);
            page = 0;
          }
          const uint32_t bytes = __popc(__ballot_sync(0xFFFFFFFFu, load)) * box_bytes;
          bool mine_ok = wraps == 0 || mbar_wait(&ctl.empty[s], (wraps - 1u) & 1u);
          if (mine_ok && lane == 0) mbar_arrive_expect_tx(&ctl.full[s], bytes);
          ok = __all_sync(0xFFFFFFFFu, mine_ok) != 0;
          if (!ok) break;
          if (load)
            tma_load_4d(dst0 + s * S::kStage, map, half * 64, tok & ((1 << a.shift) - 1), h, page,
                        &ctl.full[s], policy);
          if (++s == end_stage) s = first_stage, ++wraps;
        }
      }
      // the end of the line
      if (ok && keys) {
        const uint32_t slot = items % kItems, use = items / kItems;
        if (use >= 1) ok = warp_wait(&ctl.item_empty[slot], (use - 1u) & 1u);
        if (ok && lane == 0) {
          ctl.item[slot].tiles = -1;
          mbar_arrive(&ctl.item_full[slot]);
        }
      }
      if (!ok) {
        set_status(&ctl.status, DSPARK_ERR_TIMEOUT);
        *reinterpret_cast<volatile int32_t*>(&ctl.abort) = 1;
      }
      // leave no copy in flight into this CTA's shared memory
      for (uint32_t i = first_stage; i < end_stage; ++i)
        if (i < s || wraps > 0) mbar_wait(&ctl.full[i], (i < s ? wraps : wraps - 1u) & 1u);
    }
  } else if (warp == 2) {
    // =====================================================================
    // products
    // =====================================================================
    // The whole warp walks the line and one elected thread issues: uniform
    // descriptors stay in uniform registers. (Walked by one thread alone an
    // instruction cost about 100 cycles to issue, twice its execution.)
    if (u_begin < u_end) {
      const bool leader = elect_one();
      const uint32_t n = static_cast<uint32_t>(a.n_cols);
      const uint32_t idesc_s = attn_idesc(F16, kTileTok, n, false, false);
      const uint32_t idesc_o = attn_idesc(F16, S::D, n, true, true);
      // K and Q: rows of 128 bytes (64 elements), 8-row groups 1,024 bytes apart
      const uint64_t desc_kq = attn_desc(16, 1024, 2);
      // V: 64 elements of d contiguous per token, slabs of 64 apart, 8-token groups 1,024 apart
      const uint64_t desc_v = attn_desc(S::kSlab, 1024, 2);
      // P: 16 rows of q contiguous per token, 16-row blocks 4,096 apart, 8-token groups 256 apart
      const uint64_t desc_p = attn_desc(4096, 256, 6);
      uint32_t items = 0, tiles = 0, scores = 0;
      struct Ring {
        uint32_t s, phase, first, end;
        __device__ void on() {
          if (++s == end) s = first, phase ^= 1u;
        }
      };
      const uint32_t nk = a.k_stages, nv = a.v_stages;
      Ring rk{0, 0, 0, nk}, rv{nk, 0, nk, nk + nv};
      const uint32_t nq = a.q_bufs;
      Ring rq{nq - 1u, 1u, 0, nq};  // moved on to an item's queries before them
      bool ok = true;
      auto product_s = [&](bool last) {  // S^T of the next tile; the item's last frees Q
        const uint32_t buf = scores & 1u;
        ok = warp_wait(&ctl.full[rk.s], rk.phase);
        if (!ok) return;
        tc_fence_after();
        if (leader) {
          const uint64_t k0 = at(desc_kq, s_ring + rk.s * S::kStage), q0 = at(desc_kq, s_q + rq.s * S::HALVES * q_slab);
#pragma unroll
          for (int k = 0; k < S::D / 16; ++k)
            tc_mma(tmem + S::kColS + buf * S::NB,
                   k0 + static_cast<uint32_t>((k / 4) * (S::kSlab >> 4) + (k % 4) * 2),
                   q0 + ((k / 4) * (q_slab >> 4) + (k % 4) * 2), idesc_s, k > 0);
          tc_commit(&ctl.empty[rk.s]);
          tc_commit(&ctl.s_full[buf]);
          if (last) tc_commit(&ctl.q_empty[rq.s]);
        }
        rk.on();
        ++scores;
      };
      while (ok) {
        const uint32_t slot = items % kItems;
        ok = warp_wait(&ctl.item_full[slot], (items / kItems) & 1u);
        if (!ok) break;
        const int nt = __shfl_sync(0xFFFFFFFFu, ctl.item[slot].tiles, 0);
        int tok0 = __shfl_sync(0xFFFFFFFFu, ctl.item[slot].tile0, 0) * kTileTok;
        const int begin = __shfl_sync(0xFFFFFFFFu, ctl.item[slot].begin, 0);
        const int end = __shfl_sync(0xFFFFFFFFu, ctl.item[slot].end, 0);
        if (nt >= 0 && leader) mbar_arrive(&ctl.item_empty[slot]);
        ++items;
        if (nt < 0) break;
        if (nt == 0) continue;
        rq.on();
        ok = warp_wait(&ctl.q_full[rq.s], rq.phase);
        if (!ok) break;
        product_s(nt == 1);
        for (int i = 0; i < nt && ok; ++i, ++tiles, tok0 += kTileTok) {
          // whichever comes first, the next tile's keys or this one's weights
          const uint32_t buf = tiles % S::PBUFS;
          bool ahead = i + 1 == nt;
          WaitClock clock;
          for (;;) {
            if (!ahead && warp_test(&ctl.full[rk.s], rk.phase)) {
              product_s(i + 2 == nt);
              ahead = true;
            }
            if (warp_test(&ctl.p_full[buf], (tiles / S::PBUFS) & 1u)) break;
            ok = ok && !__any_sync(0xFFFFFFFFu, clock.expired());
            if (!ok) break;
          }
          if (!ok) break;
          // the groups' lists of the item are written
          if (leader && i + 1 == nt) mbar_arrive(&ctl.odd_full);
          ok = warp_wait(&ctl.full[rv.s], rv.phase);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t v0 = at(desc_v, s_ring + rv.s * S::kStage);
            const uint64_t p0 = at(desc_p, s_p + buf * a.p_bytes);
            // the steps of 16 tokens that some row sees
            const int k0 = max(begin - tok0, 0) >> 4, k1 = (min(end - tok0, kTileTok) + 15) >> 4;
            if (k0 == 0 && k1 == kTileTok / 16) {
#pragma unroll
              for (int k = 0; k < kTileTok / 16; ++k)
                tc_mma(tmem + S::kColO, v0 + static_cast<uint32_t>(k * 128),
                       p0 + static_cast<uint32_t>(k * 32), idesc_o, k > 0 ? 1u : i > 0);
            } else {
#pragma unroll 1
              for (int k = k0; k < k1; ++k)
                tc_mma(tmem + S::kColO, v0 + static_cast<uint32_t>(k * 128),
                       p0 + static_cast<uint32_t>(k * 32), idesc_o, i > 0 || k > k0);
            }
            tc_commit(&ctl.empty[rv.s]);
            tc_commit(&ctl.pv_done[buf]);
          }
          rv.on();
          if (!ahead) product_s(i + 2 == nt);
        }
      }
      if (!ok) {
        set_status(&ctl.status, DSPARK_ERR_TIMEOUT);
        *reinterpret_cast<volatile int32_t*>(&ctl.abort) = 1;
        if (leader) tc_commit(&ctl.drained);  // no product may outlive the CTA
        warp_wait(&ctl.drained, 0);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // =====================================================================
    // queries: two tiles of them where there is room, so that an item's are
    // there when the one before it ends
    // =====================================================================
    if (lane == 0 && u_begin < u_end) {
      const uint32_t bytes = S::HALVES * a.Gs * a.t_chunk * 128;
      uint32_t items = 0, b = 0, wraps = 0;
      bool ok = true;
      for (;;) {
        const uint32_t slot = items % kItems;
        ok = mbar_wait(&ctl.item_full[slot], (items / kItems) & 1u);
        if (!ok || ctl.item[slot].tiles < 0) break;
        ++items;
        const int tiles = ctl.item[slot].tiles, head0 = ctl.item[slot].head0;
        const int row0 = static_cast<int>(ctl.item[slot].row0);
        mbar_arrive(&ctl.item_empty[slot]);
        if (tiles == 0) continue;
        if (wraps >= 1) ok = mbar_wait(&ctl.q_empty[b], (wraps - 1u) & 1u);
        if (!ok) break;
        mbar_arrive_expect_tx(&ctl.q_full[b], bytes);
        for (int i = 0; i < S::HALVES; ++i)
          tma_load_3d_to(s_q + (b * S::HALVES + i) * q_slab, &map_q, i * 64, head0, row0,
                         &ctl.q_full[b]);
        if (++b == static_cast<uint32_t>(a.q_bufs)) b = 0, ++wraps;
      }
      if (!ok) {
        set_status(&ctl.status, DSPARK_ERR_TIMEOUT);
        *reinterpret_cast<volatile int32_t*>(&ctl.abort) = 1;
      }
      for (uint32_t i = 0; i < static_cast<uint32_t>(a.q_bufs); ++i)
        if (i < b || wraps > 0) mbar_wait(&ctl.q_full[i], (i < b ? wraps : wraps - 1u) & 1u);
    }
    __syncwarp();
  } else if (u_begin < u_end) {
    // =====================================================================
    // softmax, results
    // =====================================================================
    const int group = (warp - 4) >> 2, quarter = warp & 3, bar = 1 + group;
    const int gt = (quarter << 5) | lane;  // this thread's token of a tile, and lane of S and O
    constexpr int kBlocks = S::NC / 8;     // of 8 columns
    const int cols = a.Gs * a.t_chunk;
    const int blocks = (cols + 8 * S::GROUPS - 1) / (8 * S::GROUPS);  // of the group, in use
    const int c0 = group * blocks * 8;     // the group's first column
    const uint32_t lanes = static_cast<uint32_t>(quarter) << 21;  // (32 * quarter) << 16
    const uint32_t window = static_cast<uint32_t>(a.window);
    volatile int32_t* abort_flag = &ctl.abort;
    uint32_t tiles = 0, items = 0, lists = 0;
    const uint32_t v_end = a.k_stages + a.v_stages;
    uint32_t v_s = a.k_stages, v_phase = 0;  // ring position of the next tile of values
    const uint64_t c2 = pair(a.c, a.c);
    bool recorded = false;
    for (int j = c0 + gt; j < min(c0 + 8 * blocks, S::NB); j += 128) {
      const int t = j / a.Gs;
      ctl.new_tok[j] = t;
      ctl.at[j] = (t * a.Hq + j - t * a.Gs) * S::D;
    }
    bar_sync(bar, 128);
    for (;;) {
      const uint32_t slot = items % kItems, list = lists & 1u;
      bool failed = !mbar_wait(&ctl.item_full[slot], (items / kItems) & 1u);
      const AttnItem& it = ctl.item[slot];
      float* const nref = ctl.nref[items & 1u];
      int32_t* const lims = ctl.lim[items & 1u];
      const int rows = failed ? 0 : max(it.t_rows * a.Gs, 0);
      const int my_rows = max(0, min(8 * blocks, rows - c0));
      const int nb = (my_rows + 7) >> 3;
      for (int j = c0 + gt; j < c0 + 8 * nb; j += 128) {
        // a column past the rows takes no part: all its scores are below its reference
        nref[j] = j < rows ? kNoRef : -INFINITY;
        lims[j] = j < rows ? it.lim0 + ctl.new_tok[j] : INT_MIN / 2;
      }
      if (group == 0 && gt == 0) ctl.odd_n[list] = 0;
      if (bar_any(bar, 128, failed || *abort_flag != 0)) {
        *abort_flag = 1;
        break;
      }
      if (it.tiles < 0) break;
      ++items;
      const int lim_last = it.lim0 + it.t_rows - 1;
      const int lo_last = a.window == INT_MAX ? 0 : max(0, lim_last - a.window);
      // Sums of the columns' weights: a thread's own token's, in pairs; or, where
      // that takes too many registers, folded tile by tile into one per block.
      constexpr bool kPairs = S::NC <= 32;
      uint64_t l[kPairs ? S::NC / 2 : 1];
      float lf[kPairs ? 1 : kBlocks];
      if constexpr (kPairs) {
#pragma unroll
        for (int j = 0; j < S::NC / 2; ++j) l[j] = 0;
      } else {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) lf[b] = 0.f;
      }

      const bool exact = S::NB <= kExactRows && it.tiles >= kExactTiles;
      const float base = exact ? kExactBase<F16> : kBase<F16>;
      const float peak_base = exact ? kExactBase<F16> : kPeakBase<F16>;
      const float highest = exact ? kExactBase<F16> : kHighest<F16>;
      bool leave = false;
      for (int i = 0; i < it.tiles; ++i, ++tiles) {
        const uint32_t buf = tiles & 1u;
        const int tok0 = (it.tile0 + i) * kTileTok, tok = tok0 + gt;
        // every token of the tile visible to every row?
        const bool whole = tok0 + kTileTok <= it.lim0 && tok0 >= lo_last;
        failed |= !mbar_wait(&ctl.s_full[buf], (tiles >> 1) & 1u);
        tc_fence_after();
        // scores, -inf where the row does not see the token
        float x[S::NC];
        const uint32_t s_addr = tmem + lanes + S::kColS + buf * S::NB + c0;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
          if (b < nb) tmem_ld8(s_addr + 8 * b, x + 8 * b);
        tmem_wait_ld();
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
          if (b < nb) {
            tmem_arrived(x + 8 * b);
            if (!whole) {
              const int4* lim4 = reinterpret_cast<const int4*>(&lims[c0 + 8 * b]);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int4 m = lim4[k];
                float* y = x + 8 * b + 4 * k;
                if (static_cast<uint32_t>(m.x - 1 - tok) >= window) y[0] = -INFINITY;
                if (static_cast<uint32_t>(m.y - 1 - tok) >= window) y[1] = -INFINITY;
                if (static_cast<uint32_t>(m.z - 1 - tok) >= window) y[2] = -INFINITY;
                if (static_cast<uint32_t>(m.w - 1 - tok) >= window) y[3] = -INFINITY;
              }
            }
          }
        auto each = [&](auto f) {  // f(b) for every block in use
#pragma unroll
          for (int b = 0; b < kBlocks; ++b)
            if (b < nb) f(b);
        };
        // exponents y = c x - m
        auto exponent = [&](int b, uint64_t (&y)[4]) {
          const ulonglong2* nr = reinterpret_cast<const ulonglong2*>(&nref[c0 + 8 * b]);
          const ulonglong2 m0 = nr[0], m1 = nr[1];
          const float* z = x + 8 * b;
          y[0] = fma2(pair(z[0], z[1]), c2, m0.x);
          y[1] = fma2(pair(z[2], z[3]), c2, m0.y);
          y[2] = fma2(pair(z[4], z[5]), c2, m1.x);
          y[3] = fma2(pair(z[6], z[7]), c2, m1.y);
        };
        bool raise = i == 0;  // the first tile's maxima
        if (!raise) {
          float top = -INFINITY;
          each([&](int b) {
            uint64_t e[4];
            exponent(b, e);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float y0, y1;
              unpair(e[k], y0, y1);
              top = fmaxf(top, fmaxf(y0, y1));
            }
          });
          raise = bar_any(bar, 128, top > highest || failed);
        }
        if (raise) {
          each([&](int b) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)  // NaN takes no part
              v[k] = x[8 * b + k] == x[8 * b + k] ? x[8 * b + k] : -INFINITY;
            const float m = over_four<true>(fold_columns<true>(v, lane));
            if ((lane & 3) == 0) ctl.red[quarter][c0 + 8 * b + (lane >> 2)] = m;
          });
          if (bar_any(bar, 128, failed || *abort_flag != 0)) {
            leave = true;
            break;
          }
          for (int j = c0 + gt; j < c0 + my_rows; j += 128) {
            float top = -INFINITY, low = INFINITY;  // of the quarters that hold a token
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float v = ctl.red[w][j];
              top = fmaxf(top, v);
              if (v > -INFINITY) low = fminf(low, v);
            }
            const float m = a.c * top, down = a.c * (top - low) > kPeak ? peak_base : base;
            const float ref = fabsf(m) < kNoShift ? m - down : m, old = -nref[j];
            ctl.fac[j] = ref > old ? ex2_approx(old - ref) : 1.f;
            if (ref > old) nref[j] = -ref;
          }
          bar_sync(bar, 128);
          if (i > 0) {
            const uint32_t before = tiles - 1u;
            failed |= !mbar_wait(&ctl.pv_done[before % S::PBUFS], (before / S::PBUFS) & 1u);
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
              if (b < nb) {
                const float* f = &ctl.fac[c0 + 8 * b];
                float o[8];
                tmem_ld8(tmem + lanes + S::kColO + c0 + 8 * b, o);
                tmem_wait_ld();
                tmem_arrived(o);
#pragma unroll
                for (int k = 0; k < 8; ++k) o[k] *= f[k];
                if constexpr (kPairs) {
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    l[4 * b + k] = mul2(l[4 * b + k], pair(f[2 * k], f[2 * k + 1]));
                } else {
                  lf[b] *= f[lane >> 2];
                }
                tmem_st8(tmem + lanes + S::kColO + c0 + 8 * b, o);
              }
            tmem_wait_st();
          }
        }
        // this buffer of weights is free once its last tile has been multiplied
        const uint32_t pb = tiles % S::PBUFS, use = tiles / S::PBUFS;
        if (use >= 1) failed |= !mbar_wait(&ctl.pv_done[pb], (use - 1u) & 1u);
        each([&](int b) {
          uint64_t e[4];
          float y[8];
          exponent(b, e);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            unpair(e[k], y[2 * k], y[2 * k + 1]);
            y[2 * k] = ex2_approx(y[2 * k]);
            y[2 * k + 1] = ex2_approx(y[2 * k + 1]);
            if constexpr (kPairs) l[4 * b + k] = add2(l[4 * b + k], pair(y[2 * k], y[2 * k + 1]));
          }
          // The weights enter the second product in the inputs' type (half a
          // step of it each, no more than the output's own rounding); their sum
          // l is of the unrounded ones, whose errors would not average out
          // where a few tokens have all the weight.
          const uint32_t chunk = static_cast<uint32_t>((c0 >> 3) + b);
          const uint32_t swap = static_cast<uint32_t>(gt >> 2) & 1u;  // 32-byte swizzle
          sts_u4(s_p + pb * a.p_bytes + (chunk >> 1) * 4096u + gt * 32u +
                     (((chunk & 1u) ^ swap) << 4),
                 pack2<F16>(y[0], y[1]), pack2<F16>(y[2], y[3]), pack2<F16>(y[4], y[5]),
                 pack2<F16>(y[6], y[7]));
          if constexpr (!kPairs) lf[b] += fold_columns<false>(y, lane);
        });
        if (!whole && group == 0) {
          // Zero weights do not silence values that are not finite, and the
          // tile's rest may hold anything: what no row sees is zeroed, and of
          // what only some rows see the non-finite values are taken out here
          // and added to those rows at the end.
          const bool some = tok >= it.begin && tok < it.end;
          const bool all = tok < it.lim0 && tok >= lo_last;
          // in a step of 16 tokens that is multiplied at all
          const bool used = (tok | 15) >= it.begin && (tok & ~15) < it.end;
          if (used && !all) failed |= !mbar_wait(&ctl.full[v_s], v_phase);
          const uint32_t v_row = s_ring + v_s * S::kStage + gt * 128;
          if (!used) {
          } else if (!some) {
#pragma unroll
            for (int q = 0; q < S::HALVES; ++q)
#pragma unroll
              for (int k = 0; k < 8; ++k) sts_u4(v_row + q * S::kSlab + k * 16, 0, 0, 0, 0);
          } else if (!all) {
            bool odd = false;
            constexpr uint32_t kExp = F16 ? 0x7C00u : 0x7F80u;
#pragma unroll 4
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
            if (odd) ctl.odd[list][atomicAdd(&ctl.odd_n[list], 1)] = tok;
          }
        }
        if (++v_s == v_end) v_s = a.k_stages, v_phase ^= 1u;
        fence_proxy_async();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl.p_full[pb]);
      }
      if (leave) {
        *abort_flag = 1;
        break;
      }

      // ---- the item's rows ----------------------------------------------
      const bool alone = it.starts && it.ends;
      const int64_t part_row = static_cast<int64_t>(2 * id + (it.starts ? 1 : 0)) * a.n_cols;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        if (b < nb) {
          float sum;
          if constexpr (kPairs) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) unpair(l[4 * b + k], v[2 * k], v[2 * k + 1]);
            sum = over_four<false>(fold_columns<false>(v, lane));
          } else {
            sum = over_four<false>(lf[b]);
          }
          if ((lane & 3) == 0) ctl.red[quarter][c0 + 8 * b + (lane >> 2)] = sum;
        }
      if (bar_any(bar, 128, failed || *abort_flag != 0)) {
        *abort_flag = 1;
        break;
      }
      // every warp for itself: the factor of column j in lane j % 32
      constexpr int kPer = (S::NC + 31) / 32;
      float fac[kPer];
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        const int j = c0 + 32 * q + lane;
        fac[q] = 1.f;
        if (32 * q + lane < my_rows) {
          const float sum = (ctl.red[0][j] + ctl.red[1][j]) + (ctl.red[2][j] + ctl.red[3][j]);
          const bool seen = lims[j] > 0;
          if (alone) fac[q] = seen ? 1.f / sum : 0.f;  // no token: O is zero
          if (quarter == 0) {
            const float m = -nref[j];
            if (!alone)
              reinterpret_cast<float2*>(a.part_ml)[part_row + j] = make_float2(m, sum);
            else if (a.lse)
              a.lse[it.row0 * a.Hq + it.head0 + ctl.at[j] / S::D] =
                  seen ? plus_log2(m, sum) * 0.69314718055994531f : -INFINITY;
          }
        }
      }
      if (it.tiles > 0) {
        const uint32_t last = tiles - 1u;
        failed |= !mbar_wait(&ctl.odd_full, lists & 1u);
        failed |= !mbar_wait(&ctl.pv_done[last % S::PBUFS], (last / S::PBUFS) & 1u);
        tc_fence_after();
        ++lists;
      }
      if (failed) *abort_flag = 1;  // seen by all at the next item
      const int odd_n = it.tiles > 0 ? ctl.odd_n[list] : 0;
      const bool writer = S::D == 128 || lane < 16;  // M = 64 fills 16 lanes of each warp's 32
      const int d = S::D == 128 ? gt : quarter * 16 + lane;
      uint16_t* const out =
          static_cast<uint16_t*>(a.out) + (it.row0 * a.Hq + it.head0) * S::D + d;
      float* const part = a.part_o + (part_row + c0) * S::D + d;
#pragma unroll 1
      for (int b = 0; b < nb; ++b) {
        float o[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) o[k] = 0.f;
        if (it.tiles > 0) {
          tmem_ld8(tmem + lanes + S::kColO + c0 + 8 * b, o);
          tmem_wait_ld();
          tmem_arrived(o);
        }
        for (int q = 0; q < odd_n; ++q) {
          const int u = ctl.odd[list][q];
          const int32_t page = a.table[it.r * a.stride + (u >> a.shift)];
          if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.num_pages) || !writer) continue;
          const uint32_t bits = static_cast<const uint16_t*>(a.v_cache)[
              page * a.page_stride + (u & ((1 << a.shift) - 1)) * a.token_stride +
              it.kv_head * a.head_stride + d];
          constexpr uint32_t kExp = F16 ? 0x7C00u : 0x7F80u;
          if ((bits & kExp) != kExp) continue;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (static_cast<uint32_t>(lims[c0 + 8 * b + k] - 1 - u) < window)
              o[k] += half_to_float<F16>(bits);
        }
        const int4* at4 = reinterpret_cast<const int4*>(&ctl.at[c0 + 8 * b]);
        const int4 a0 = at4[0], a1 = at4[1];
        const int to[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
        const float mine = kPer > 1 && b >= 4 ? fac[kPer - 1] : fac[0];
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __shfl_sync(0xFFFFFFFFu, mine, (8 * b + k) & 31);
        const int live = writer ? my_rows - 8 * b : 0;  // columns of the block to write
        if (alone) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < live) out[to[k]] = static_cast<uint16_t>(pack2<F16>(o[k] * f[k], 0.f));
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k < live) part[(8 * b + k) * S::D] = o[k];
        }
      }
      if (it.ends && !it.starts) {
        recorded = true;
        if (tid == 128) {
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
    if (!recorded && tid == 128) a.records[id].valid = 0;
    if (*abort_flag != 0 && tid == 128) set_status(&ctl.status, DSPARK_ERR_TIMEOUT);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) tmem_dealloc(tmem, S::kTmem);
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
  constexpr int kWords = (DSPARK_PAGED_MAX_CTAS + 31) / 32;
  constexpr int kEach = (kWords + kJoinWarps - 1) / kJoinWarps;  // records per thread
  constexpr int V = D / 32;                                      // floats per lane
  constexpr int kBatch = 8;                                      // pieces in flight per warp
  __shared__ uint32_t s_valid[kWords], s_bad[kWords];
  __shared__ AttnRecord s_rec;
  __shared__ float s_acc[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  // All records at once (one trip to the cache), then the one that is asked for.
  const int words = (a.n + 31) / 32;
  int4 rec[kEach][2];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = (warp + k * kJoinWarps) * 32 + lane;
    rec[k][0] = rec[k][1] = make_int4(0, 0, 0, 0);
    if (i < a.n) {
      rec[k][0] = reinterpret_cast<const int4*>(a.records + i)[0];
      rec[k][1] = reinterpret_cast<const int4*>(a.records + i)[1];
    }
  }
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const uint32_t v = __ballot_sync(0xFFFFFFFFu, rec[k][0].x != 0);
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, rec[k][0].z != DSPARK_OK);
    if (lane == 0 && warp + k * kJoinWarps < words)
      s_valid[warp + k * kJoinWarps] = v, s_bad[warp + k * kJoinWarps] = b;
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
#pragma unroll
  for (int k = 0; k < kEach; ++k)
    if ((warp + k * kJoinWarps) * 32 + lane == id) {
      reinterpret_cast<int4*>(&s_rec)[0] = rec[k][0];
      reinterpret_cast<int4*>(&s_rec)[1] = rec[k][1];
    }
  __syncthreads();
  const AttnRecord r = s_rec;
  const int chunk0 = id / a.ctas * a.ctas, pieces = id - chunk0 - r.first + 1;
  const int row = blockIdx.y * (kJoinWarps / a.per_row) + warp / a.per_row;
  const int sub = warp % a.per_row;
  // Sums of 2^(m - top) l and O over the warp's pieces, a batch at a time: its
  // maxima and rows are fetched together, and the sums so far are scaled.
  float acc[V] = {}, sum = 0.f, top = -INFINITY;
  if (row < r.rows) {
    const float2* ml = reinterpret_cast<const float2*>(a.part_ml);
    for (int k0 = sub; k0 < pieces; k0 += kBatch * a.per_row) {
      float2 p[kBatch];
      float o[kBatch][V];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int k = k0 + q * a.per_row;
        p[q] = make_float2(-INFINITY, 0.f);
        if (k < pieces) {
          const int64_t s =
              (2 * static_cast<int64_t>(chunk0 + r.first + k) + (k == 0 ? 1 : 0)) * a.n_cols + row;
          p[q] = ml[s];
          const float* from = a.part_o + s * D + lane * V;
          if constexpr (V == 4)
            *reinterpret_cast<float4*>(o[q]) = *reinterpret_cast<const float4*>(from);
          else
            *reinterpret_cast<float2*>(o[q]) = *reinterpret_cast<const float2*>(from);
        }
      }
      float now = top;
#pragma unroll
      for (int q = 0; q < kBatch; ++q) now = fmaxf(now, p[q].x);
      const float f = top == -INFINITY ? 0.f : ex2_approx(top - now);
      sum *= f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] *= f;
      top = now;
#pragma unroll
      for (int q = 0; q < kBatch; ++q)
        if (k0 + q * a.per_row < pieces) {
          const float w = ex2_approx(p[q].x - top);
          sum = fmaf(w, p[q].y, sum);
#pragma unroll
          for (int v = 0; v < V; ++v) acc[v] = fmaf(w, o[q][v], acc[v]);
        }
    }
  }
  if (a.per_row > 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) s_acc[warp][lane * V + v] = acc[v];
    if (lane == 0) s_ml[warp] = make_float2(top, sum);
    __syncthreads();
    if (sub == 0) {
      for (int w = 1; w < a.per_row; ++w) top = fmaxf(top, s_ml[warp + w].x);
      sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] = 0.f;
      for (int w = 0; w < a.per_row; ++w) {
        const float2 p = s_ml[warp + w];
        if (p.x == -INFINITY) continue;  // a warp without pieces
        const float f = ex2_approx(p.x - top);
        sum = fmaf(f, p.y, sum);
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = fmaf(f, s_acc[warp + w][lane * V + v], acc[v]);
      }
    }
  }
  if (row < r.rows && sub == 0) {
    const bool seen = r.lim0 + row / a.Gs > 0;
    const int64_t at = (r.row0 + row / a.Gs) * a.Hq + r.head0 + row % a.Gs;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + at * D + lane * V);
    const float inv = 1.f / sum;
#pragma unroll
    for (int v = 0; v < V; v += 2)
      out[v / 2] = seen ? pack2<F16>(acc[v] * inv, acc[v + 1] * inv) : 0u;
    if (a.lse && lane == 0) a.lse[at] = seen ? plus_log2(top, sum) * 0.69314718055994531f : -INFINITY;
  }
}

}  // namespace dspark
