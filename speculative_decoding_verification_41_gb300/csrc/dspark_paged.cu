// dspark_paged.cu -- bookkeeping of the paged key-value cache (sm_103a):
// dspark_pages_reserve, dspark_pages_release and dspark_kv_append
// (include/dspark_paged.h).
//
// Reserve and release are prefix sums over the requests (tokens, pages) and a
// scatter of their pages and slots. A sum over a thousand requests takes one
// CTA about a microsecond, a second launch about as long, so every CTA forms
// the sums for itself from the lengths (8 bytes per request, in L2 after the
// first) and then writes its own share of the outputs: no CTA waits for
// another, and nothing needs zeroed memory. CTA 0 writes what there is one of
// per request and judges the data.
#include <algorithm>
#include <climits>

#include "../../include/dspark_paged.h"
#include "dspark_common.cuh"

namespace dspark {
namespace {

constexpr int kPagedThreads = 1024;         // requests per step of the sums
constexpr int kPagedWarps = kPagedThreads / 32;
// Sums saturate here, above every limit they meet (max_tokens may be 2^30); two of
// them still add within 32 bits.
constexpr uint32_t kCap = (1u << 30) + 1u;
constexpr int kTokensPerCta = 1024;          // slot-map rows per filling CTA, at least

struct Sum3 {
  uint32_t tok, page, draft;
};
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kCap); }
__device__ __forceinline__ Sum3 add(Sum3 a, Sum3 b) {
  return Sum3{sat_add(a.tok, b.tok), sat_add(a.page, b.page), sat_add(a.draft, b.draft)};
}

// Inclusive saturating sums over the CTA's threads; `total` receives the sum of
// all of them. (Saturating addition of non-negative numbers is associative.)
__device__ __forceinline__ Sum3 block_scan(Sum3 v, Sum3* warp_sums, Sum3& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sum3 u{__shfl_up_sync(0xFFFFFFFFu, v.tok, o), __shfl_up_sync(0xFFFFFFFFu, v.page, o),
           __shfl_up_sync(0xFFFFFFFFu, v.draft, o)};
    if (lane >= o) v = add(v, u);
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  Sum3 w = warp_sums[lane];  // every warp sums the warps' totals for itself
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sum3 u{__shfl_up_sync(0xFFFFFFFFu, w.tok, o), __shfl_up_sync(0xFFFFFFFFu, w.page, o),
           __shfl_up_sync(0xFFFFFFFFu, w.draft, o)};
    if (lane >= o) w = add(w, u);
  }
  const int prev = max(warp - 1, 0);
  Sum3 before{__shfl_sync(0xFFFFFFFFu, w.tok, prev), __shfl_sync(0xFFFFFFFFu, w.page, prev),
              __shfl_sync(0xFFFFFFFFu, w.draft, prev)};
  total = Sum3{__shfl_sync(0xFFFFFFFFu, w.tok, 31), __shfl_sync(0xFFFFFFFFu, w.page, 31),
               __shfl_sync(0xFFFFFFFFu, w.draft, 31)};
  return warp > 0 ? add(before, v) : v;
}
static_assert(kPagedWarps == 32, "block_scan sums 32 warps in one");

// the first index of [0, n) whose inclusive sum exceeds x (n if there is none)
__device__ __forceinline__ int first_above(const uint32_t* incl, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (incl[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

struct ReserveArgs {
  const int32_t *ctx, *new_len;
  int32_t* table;
  const int32_t *stack, *stack_count;
  int32_t* ctx_out;
  int64_t *row_off, *draft_off;
  int32_t *slots, *pos, *count_out, *status;
  int64_t stride;
  int32_t extra, B, shift, num_pages, max_pages, max_tokens, per_cta;
  bool vec;      // slot_map and positions take 16-byte stores
  bool lengths;  // write ctx_out and count_out
};

// CTA 0: per-request outputs, status. CTA i > 0: slot-map rows [(i-1)*per_cta,
// i*per_cta). New pages are dealt out to all.
__global__ void __launch_bounds__(kPagedThreads, 1) k_pages_reserve(const ReserveArgs a) {
  __shared__ Sum3 warp_sums[kPagedWarps];
  __shared__ uint32_t s_tok[kPagedThreads], s_page[kPagedThreads];  // inclusive, in this step
  __shared__ int32_t s_ctx[kPagedThreads];
  __shared__ uint32_t s_first, s_why;
  const int tid = threadIdx.x;
  if (tid == 0) s_why = 0;
  pdl_wait();  // predecessor grid complete, its writes visible
  pdl_trigger();
  const bool books = blockIdx.x == 0;
  const int32_t count = *a.stack_count;
  const uint32_t avail = count < 0 || count > a.num_pages ? 0u : static_cast<uint32_t>(count);
  bool bad = avail != static_cast<uint32_t>(count), many = false, dry = false;
  const int64_t room = static_cast<int64_t>(a.max_pages) << a.shift;
  const uint32_t mask = (1u << a.shift) - 1u;
  const int32_t none = a.num_pages << a.shift;  // slot of a page outside the pool
  const uint32_t t0 = books ? 0u : (blockIdx.x - 1u) * static_cast<uint32_t>(a.per_cta);
  const uint32_t t1 =
      books ? 0u : min(t0 + static_cast<uint32_t>(a.per_cta), static_cast<uint32_t>(a.max_tokens));
  Sum3 carry{0, 0, 0};  // given to the requests of earlier steps
  bool closed = false;  // a request did not fit: all after it get nothing

  for (int base = 0; base < a.B; base += kPagedThreads) {
    const int r = base + tid;
    Sum3 own{0, 0, 0};
    int32_t ctx = 0;
    if (r < a.B) {
      ctx = a.ctx[r];
      const int32_t d = a.new_len[r];
      const int64_t end = static_cast<int64_t>(ctx) + d + a.extra;
      if (ctx < 0 || d < 0 || end > room) {
        bad = true;
      } else {
        own.tok = min(static_cast<uint32_t>(end - ctx), kCap);
        own.draft = min(static_cast<uint32_t>(d), kCap);
        own.page = static_cast<uint32_t>(((end + mask) >> a.shift) -
                                         ((static_cast<int64_t>(ctx) + mask) >> a.shift));
      }
    }
    Sum3 all;
    Sum3 in = block_scan(own, warp_sums, all);
    const Sum3 reach = add(carry, in);
    const bool no_row = reach.tok > static_cast<uint32_t>(a.max_tokens);
    const bool no_page = reach.page > avail;
    const bool refused = own.tok > 0 && (closed || no_row || no_page);
    // What does not fit is a suffix of the requests with new tokens: the sums
    // up to the last one served are those of the whole step where all fit.
    s_tok[tid] = in.tok;
    s_page[tid] = in.page;
    s_ctx[tid] = ctx;
    uint32_t served = kPagedThreads;
    if (__syncthreads_or(refused)) {
      if (tid == 0) s_first = kPagedThreads;
      __syncthreads();
      if (refused) atomicMin(&s_first, static_cast<uint32_t>(tid));
      __syncthreads();
      served = s_first;
      if (static_cast<uint32_t>(tid) == served && !closed) {  // the status is this request's
        many = no_row;
        dry = no_page;
      }
      if (static_cast<uint32_t>(tid) + 1u == served) warp_sums[0] = in;
      __syncthreads();
      all = served > 0 ? warp_sums[0] : Sum3{0, 0, 0};
      if (static_cast<uint32_t>(tid) >= served) own = Sum3{0, 0, 0}, in = all;
      closed = true;
    }
    const int n_req = static_cast<int>(min(served, static_cast<uint32_t>(a.B - base)));

    if (books) {
      if (r < a.B) {
        const int64_t tok = static_cast<int64_t>(carry.tok) + in.tok;
        a.row_off[r + 1] = tok;
        if (a.draft_off) a.draft_off[r + 1] = static_cast<int64_t>(carry.draft) + in.draft;
        if (a.lengths) a.ctx_out[r] = ctx + static_cast<int32_t>(own.tok);
        if (own.tok > 0 && (static_cast<uint32_t>(ctx) & mask) != 0u) {
          // the page that already holds the request's last tokens takes some
          const int32_t p = a.table[static_cast<int64_t>(r) * a.stride + (ctx >> a.shift)];
          bad |= static_cast<uint32_t>(p) >= static_cast<uint32_t>(a.num_pages);
        }
      }
#pragma unroll 8
      for (uint32_t i = tid; i < all.page; i += kPagedThreads) {
        const int32_t p = a.stack[avail - 1u - (carry.page + i)];
        bad |= static_cast<uint32_t>(p) >= static_cast<uint32_t>(a.num_pages);
      }
    }
    // new pages, a block of them per CTA in turn (a small call's all in CTA 0)
    for (uint32_t i = blockIdx.x * kPagedThreads + tid; i < all.page;
         i += gridDim.x * kPagedThreads) {
      const int q = first_above(s_page, n_req, i);
      const uint32_t before = q > 0 ? s_page[q - 1] : 0u;
      const uint32_t have = (static_cast<uint32_t>(s_ctx[q]) + mask) >> a.shift;
      a.table[static_cast<int64_t>(base + q) * a.stride + have + (i - before)] =
          a.stack[avail - 1u - (carry.page + i)];
    }
    // Rows of this step's requests in the CTA's range: one per thread where that
    // does for all (a decoding step: one chain of search, page id, store), else
    // four in a row, which share a search and are stored together (2 M rows: 12.9 us
    // one by one; a step of 64 requests: 3.1 us one by one, 4.2 in fours).
    const uint32_t lo = max(t0, carry.tok), hi = min(t1, carry.tok + all.tok);
    // where the page id of row x of this step is, x in request q, and its position
    auto page_of = [&](uint32_t x, int q, uint32_t& p) -> const int32_t* {
      const uint32_t c = static_cast<uint32_t>(s_ctx[q]);
      p = c + (x - (q > 0 ? s_tok[q - 1] : 0u));
      const uint32_t have = (c + mask) >> a.shift, blk = p >> a.shift;
      return blk < have ? a.table + static_cast<int64_t>(base + q) * a.stride + blk
                        : a.stack + (avail - 1u - (carry.page + (q > 0 ? s_page[q - 1] : 0u) +
                                                   (blk - have)));
    };
    auto slot_of = [&](int32_t page, uint32_t p) {
      return static_cast<uint32_t>(page) < static_cast<uint32_t>(a.num_pages)
                 ? (page << a.shift) + static_cast<int32_t>(p & mask)
                 : none;
    };
    if (a.per_cta <= kPagedThreads) {
      const uint32_t t = t0 + tid;
      if (t >= lo && t < hi) {
        uint32_t p;
        const int32_t page = *page_of(t - carry.tok, first_above(s_tok, n_req, t - carry.tok), p);
        a.slots[t] = slot_of(page, p);
        if (a.pos) a.pos[t] = static_cast<int32_t>(p);
      }
    } else {
      for (uint32_t g = (lo & ~3u) + 4u * tid; g < hi; g += 4u * kPagedThreads) {
        int32_t slot[4], page[4];
        uint32_t pos[4];
        const int32_t* from[4];
        int q = -1;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t t = min(max(g + k, lo), hi - 1u), x = t - carry.tok;
          if (q < 0)
            q = first_above(s_tok, n_req, x);
          else
            while (s_tok[q] <= x) ++q;
          from[k] = page_of(x, q, pos[k]);
        }
        // mostly one page, and one trip to the cache
#pragma unroll
        for (int k = 0; k < 4; ++k) page[k] = *from[k];
#pragma unroll
        for (int k = 0; k < 4; ++k) slot[k] = slot_of(page[k], pos[k]);
        if (a.vec && g >= lo && g + 4u <= hi) {
          *reinterpret_cast<int4*>(a.slots + g) = make_int4(slot[0], slot[1], slot[2], slot[3]);
          if (a.pos)
            *reinterpret_cast<uint4*>(a.pos + g) = make_uint4(pos[0], pos[1], pos[2], pos[3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (g + k >= lo && g + k < hi) {
              a.slots[g + k] = slot[k];
              if (a.pos) a.pos[g + k] = static_cast<int32_t>(pos[k]);
            }
        }
      }
    }
    carry = add(carry, all);
    if (base + kPagedThreads < a.B) __syncthreads();  // the step's sums are read no more
  }
  // rows past the last token
  const uint32_t pad = max(t0, carry.tok);
  for (uint32_t g = (pad & ~3u) + 4u * tid; g < t1; g += 4u * kPagedThreads) {
    if (a.vec && g >= pad && g + 4u <= t1) {
      *reinterpret_cast<int4*>(a.slots + g) = make_int4(-1, -1, -1, -1);
      if (a.pos) *reinterpret_cast<int4*>(a.pos + g) = make_int4(-1, -1, -1, -1);
    } else {
      for (uint32_t t = max(g, pad); t < min(g + 4u, t1); ++t) {
        a.slots[t] = -1;
        if (a.pos) a.pos[t] = -1;
      }
    }
  }
  if (books) {
    if (bad || many || dry) atomicOr(&s_why, (bad ? 1u : 0u) | (many ? 2u : 0u) | (dry ? 4u : 0u));
    __syncthreads();
    const uint32_t any_bad = s_why & 1u, any_many = s_why & 2u, any_dry = s_why & 4u;
    if (tid == 0) {
      a.row_off[0] = 0;
      if (a.draft_off) a.draft_off[0] = 0;
      if (a.lengths) *a.count_out = count - static_cast<int32_t>(carry.page);
      *a.status = any_bad    ? DSPARK_ERR_BAD_DATA
                  : any_many ? DSPARK_ERR_TOO_LARGE
                  : any_dry  ? DSPARK_ERR_NO_PAGES
                             : DSPARK_OK;
    }
  }
}

struct ReleaseArgs {
  const int32_t *ctx, *reserved, *kept, *table;
  int32_t *stack;
  const int32_t *stack_count;
  int32_t *ctx_out, *count_out, *status;
  int64_t stride;
  int32_t extra, B, shift, num_pages, max_pages;
  bool push, lengths;  // push the pages; write ctx_out and count_out
};

// CTA 0: per-request outputs, status. The pages are dealt out in blocks to all.
__global__ void __launch_bounds__(kPagedThreads, 1) k_pages_release(const ReleaseArgs a) {
  __shared__ Sum3 warp_sums[kPagedWarps];
  __shared__ uint32_t s_page[kPagedThreads];
  __shared__ uint32_t s_stay[kPagedThreads];
  const int tid = threadIdx.x;
  pdl_wait();
  pdl_trigger();
  const bool books = blockIdx.x == 0;
  const int32_t count = *a.stack_count;
  const bool bad_count = count < 0 || count > a.num_pages;
  const uint32_t first = bad_count ? static_cast<uint32_t>(a.num_pages)  // every push is dropped
                                   : static_cast<uint32_t>(count);
  bool bad = bad_count;
  const int64_t room = static_cast<int64_t>(a.max_pages) << a.shift;
  const uint32_t mask = (1u << a.shift) - 1u;
  uint32_t carry = 0;
  for (int base = 0; base < a.B; base += kPagedThreads) {
    const int r = base + tid;
    Sum3 own{0, 0, 0};
    uint32_t stay = 0;
    int32_t keep = 0;
    if (r < a.B) {
      const int32_t ctx = a.ctx[r], end = a.reserved[r], kept = a.kept[r];
      keep = end;
      if (ctx < 0 || end < ctx || end > room || kept < -1 ||
          (kept >= 0 && end > ctx &&
           static_cast<int64_t>(kept) + a.extra > static_cast<int64_t>(end) - ctx)) {
        bad = true;
      } else {
        if (kept < 0)
          keep = 0;
        else if (end > ctx)
          keep = ctx + kept + a.extra;
        stay = (static_cast<uint32_t>(keep) + mask) >> a.shift;
        own.page = ((static_cast<uint32_t>(end) + mask) >> a.shift) - stay;
      }
    }
    Sum3 all;
    const Sum3 in = block_scan(own, warp_sums, all);
    s_page[tid] = in.page;
    s_stay[tid] = stay;
    __syncthreads();
    if (books && a.lengths && r < a.B) a.ctx_out[r] = keep;
    const int n_req = min(kPagedThreads, a.B - base);
    for (uint32_t i = blockIdx.x * kPagedThreads + tid; a.push && i < all.page;
         i += gridDim.x * kPagedThreads) {
      const uint32_t to = first + carry + i;
      if (to >= static_cast<uint32_t>(a.num_pages)) break;
      const int q = first_above(s_page, n_req, i);
      const uint32_t before = q > 0 ? s_page[q - 1] : 0u;
      a.stack[to] = a.table[static_cast<int64_t>(base + q) * a.stride + s_stay[q] + (i - before)];
    }
    carry = sat_add(carry, all.page);
    __syncthreads();
  }
  if (books) {
    const int any_bad = __syncthreads_or(bad);
    if (tid == 0) {
      const uint32_t now = first + carry;
      const bool over = now > static_cast<uint32_t>(a.num_pages);
      if (a.lengths) *a.count_out = bad_count ? count : over ? a.num_pages : static_cast<int32_t>(now);
      *a.status = any_bad || over ? DSPARK_ERR_BAD_DATA : DSPARK_OK;
    }
  }
}

// A CTA takes a group of whole rows of about 1,024 16-byte pieces: four loads of
// keys and four of values in flight per thread before the first store. CTAs that
// end and begin keep the memory busier than CTAs that loop: 100,000 rows of 8 x
// 128 in 114 us (6.7 TB/s) against 133 us with eight looping CTAs per SM. CTA 0
// only judges the slots, so that one CTA writes the status.
constexpr int kAppendThreads = 256;
constexpr int kAppendPieces = 4;

struct AppendArgs {
  const uint4 *k, *v;
  uint4 *kc, *vc;
  const int32_t* slots;
  int32_t* status;
  int64_t row, head, page, token, chead;  // strides in 16-byte pieces
  int32_t n, pieces, d_shift, shift, n_slots, rows;  // pieces per row; rows per group
};

__global__ void __launch_bounds__(kAppendThreads) k_kv_append(const AppendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) {
    bool bad = false;
#pragma unroll 4
    for (int i = tid; i < a.n; i += kAppendThreads) bad |= a.slots[i] >= a.n_slots;
    const int any = __syncthreads_or(bad);
    if (tid == 0) *a.status = any ? DSPARK_ERR_BAD_DATA : DSPARK_OK;
    return;
  }
  const uint32_t mask = (1u << a.shift) - 1u, dmask = (1u << a.d_shift) - 1u;
  for (int64_t r0 = (blockIdx.x - 1) * static_cast<int64_t>(a.rows); r0 < a.n;
       r0 += (gridDim.x - 1) * static_cast<int64_t>(a.rows)) {
    const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), a.n - r0));
    const int total = rows * a.pieces;
    for (int i0 = tid; i0 < total; i0 += kAppendPieces * kAppendThreads) {
      uint4 k[kAppendPieces], v[kAppendPieces];
      int64_t to[kAppendPieces];
#pragma unroll
      for (int j = 0; j < kAppendPieces; ++j) {
        const int i = i0 + j * kAppendThreads;
        to[j] = -1;
        if (i >= total) continue;
        const int q = i / a.pieces, w = i - q * a.pieces;
        const int64_t head = w >> a.d_shift;
        const int d = static_cast<int>(w & dmask);
        const int32_t s = a.slots[r0 + q];
        if (s < 0 || s >= a.n_slots) continue;
        to[j] = (s >> a.shift) * a.page + static_cast<int64_t>(s & mask) * a.token +
                head * a.chead + d;
        const int64_t from = (r0 + q) * a.row + head * a.head + d;
        k[j] = __ldg(a.k + from);
        v[j] = __ldg(a.v + from);
      }
#pragma unroll
      for (int j = 0; j < kAppendPieces; ++j)
        if (to[j] >= 0) {
          a.kc[to[j]] = k[j];
          a.vc[to[j]] = v[j];
        }
    }
  }
}

int page_shift(int32_t page_size) {
  for (int s = 3; s <= 10; ++s)
    if (page_size == 1 << s) return s;
  return -1;
}

bool pool_ok(int32_t B, int32_t page_size, int32_t num_pages, int64_t table_stride,
             int32_t max_pages) {
  return B >= 0 && page_shift(page_size) >= 0 && num_pages >= 1 &&
         static_cast<int64_t>(num_pages) * page_size <= INT32_MAX && max_pages >= 1 &&
         static_cast<int64_t>(max_pages) * page_size <= INT32_MAX && table_stride >= max_pages;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" int dspark_pages_reserve(
    const int32_t* context_len, const int32_t* new_len, int32_t extra, int32_t B,
    int32_t page_size, int32_t num_pages, int32_t* block_table, int64_t table_stride,
    int32_t max_pages, const int32_t* free_pages, const int32_t* free_count, int32_t max_tokens,
    int32_t* context_out, int64_t* row_off, int64_t* draft_off, int32_t* slot_map,
    int32_t* positions, int32_t* free_count_out, int32_t* device_status,
    struct CUstream_st* stream) {
  if (!pool_ok(B, page_size, num_pages, table_stride, max_pages) || extra < 0 || max_tokens < 0 ||
      max_tokens > (1 << 30) || !free_pages || !free_count || !row_off || !free_count_out ||
      !device_status || (max_tokens > 0 && !slot_map) ||
      (B > 0 && (!context_len || !new_len || !block_table || !context_out)))
    return DSPARK_ERR_INVALID_ARG;
  const int fill = static_cast<int>(
      std::min<int64_t>(DSPARK_CEILDIV(max_tokens, kTokensPerCta), 147));
  ReserveArgs a{};
  a.ctx = context_len, a.new_len = new_len, a.table = block_table, a.stack = free_pages;
  a.stack_count = free_count, a.ctx_out = context_out, a.row_off = row_off;
  a.draft_off = draft_off, a.slots = slot_map, a.pos = positions, a.count_out = free_count_out;
  a.status = device_status, a.stride = table_stride, a.extra = extra, a.B = B;
  a.shift = page_shift(page_size), a.num_pages = num_pages, a.max_pages = max_pages;
  a.max_tokens = max_tokens;
  a.per_cta = fill > 0 ? static_cast<int32_t>(4 * DSPARK_CEILDIV(max_tokens, 4 * fill)) : 0;
  a.vec = aligned16(slot_map) && aligned16(positions);
  // Lengths written over the ones that other CTAs still read: in a launch of
  // its own, after this one.
  const bool over = context_out == context_len || context_out == new_len ||
                    free_count_out == free_count;
  a.lengths = !over;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (launch_pdl(k_pages_reserve, 1 + std::max(fill, 1), kPagedThreads, 0, st, a) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  a.lengths = true;
  if (over && launch_pdl(k_pages_reserve, 1, kPagedThreads, 0, st, a) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  if (cudaGetLastError() != cudaSuccess) return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

extern "C" int dspark_pages_release(const int32_t* context_len, const int32_t* reserved_len,
                                    const int32_t* kept_len, int32_t extra, int32_t B,
                                    int32_t page_size, int32_t num_pages,
                                    const int32_t* block_table, int64_t table_stride,
                                    int32_t max_pages, int32_t* free_pages,
                                    const int32_t* free_count, int32_t* context_out,
                                    int32_t* free_count_out, int32_t* device_status,
                                    struct CUstream_st* stream) {
  if (!pool_ok(B, page_size, num_pages, table_stride, max_pages) || extra < 0 || !free_pages ||
      !free_count || !free_count_out || !device_status ||
      (B > 0 && (!context_len || !reserved_len || !kept_len || !block_table || !context_out)))
    return DSPARK_ERR_INVALID_ARG;
  ReleaseArgs a{};
  a.ctx = context_len, a.reserved = reserved_len, a.kept = kept_len, a.table = block_table;
  a.stack = free_pages, a.stack_count = free_count, a.ctx_out = context_out;
  a.count_out = free_count_out, a.status = device_status, a.stride = table_stride;
  a.extra = extra, a.B = B, a.shift = page_shift(page_size), a.num_pages = num_pages;
  a.max_pages = max_pages;
  const bool over = context_out == context_len || context_out == reserved_len ||
                    context_out == kept_len || free_count_out == free_count;
  a.push = true;
  a.lengths = !over;
  const int64_t most = std::min<int64_t>(num_pages, static_cast<int64_t>(B) * max_pages);
  const int grid = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(DSPARK_CEILDIV(most, 8 * kPagedThreads), 148)));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (launch_pdl(k_pages_release, grid, kPagedThreads, 0, st, a) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  a.push = false;
  a.lengths = true;
  if (over && launch_pdl(k_pages_release, 1, kPagedThreads, 0, st, a) != cudaSuccess)
    return DSPARK_ERR_CUDA;
  if (cudaGetLastError() != cudaSuccess) return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}

extern "C" int dspark_kv_append(const void* k, const void* v, int64_t row_stride,
                                int64_t in_head_stride, const int32_t* slot_map, int32_t n,
                                int32_t Hkv, int32_t D, int32_t dtype, void* k_cache,
                                void* v_cache, int64_t page_stride, int64_t token_stride,
                                int64_t head_stride, int32_t page_size, int32_t num_pages,
                                int32_t* device_status, struct CUstream_st* stream) {
  if (n < 0 || Hkv < 1 || Hkv > 65536 || (D != 64 && D != 128) ||
      (dtype != DSPARK_BF16 && dtype != DSPARK_F16) || !pool_ok(0, page_size, num_pages, 1, 1) ||
      !device_status || !aligned16(k) || !aligned16(v) || !aligned16(k_cache) ||
      !aligned16(v_cache) || (n > 0 && (!k || !v || !slot_map || !k_cache || !v_cache)) ||
      row_stride < 0 || in_head_stride < 0 || page_stride < 0 || token_stride < 0 ||
      head_stride < 0 ||
      ((row_stride | in_head_stride | page_stride | token_stride | head_stride) & 7) != 0)
    return DSPARK_ERR_INVALID_ARG;
  AppendArgs a{};
  a.k = static_cast<const uint4*>(k), a.v = static_cast<const uint4*>(v);
  a.kc = static_cast<uint4*>(k_cache), a.vc = static_cast<uint4*>(v_cache);
  a.slots = slot_map, a.status = device_status;
  a.row = row_stride / 8, a.head = in_head_stride / 8, a.page = page_stride / 8;
  a.token = token_stride / 8, a.chead = head_stride / 8;
  a.n = n, a.pieces = Hkv * (D / 8), a.d_shift = D == 64 ? 3 : 4;
  a.shift = page_shift(page_size), a.n_slots = num_pages * page_size;
  a.rows = std::max(1, kAppendPieces * kAppendThreads / a.pieces);
  const int64_t groups = static_cast<int64_t>(DSPARK_CEILDIV(n, a.rows));
  const int grid = 1 + static_cast<int>(std::min<int64_t>(groups, 1 << 20));
  if (launch_pdl(k_kv_append, grid, kAppendThreads, 0, reinterpret_cast<cudaStream_t>(stream),
                 a) != cudaSuccess ||
      cudaGetLastError() != cudaSuccess)
    return DSPARK_ERR_CUDA;
  return DSPARK_OK;
}
