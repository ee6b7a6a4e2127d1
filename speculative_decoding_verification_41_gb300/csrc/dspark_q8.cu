// dspark_q8.cu -- rotary positions, and the write of the 8-bit paged cache and its
// reading back (sm_103a): dspark_rotary, dspark_kv_append_q8, dspark_kv_gather_q8
// (include/dspark_q8.h). All three are bound by the bytes they move.
#include <algorithm>
#include <climits>
#include <cmath>

#include "dspark_q8.cuh"

namespace dspark {
namespace {

constexpr int kMaxPairs = 64;  // of a head

struct Turns {
  const uint64_t* turns;
  const int32_t* positions;
  float gain;
  int32_t rot;    // elements of a head that turn
  bool inter;     // pairs are neighbours
};

// Cosine and sine of pair j at a position, times the gain. The angle in turns is
// position * turns[j] mod 1 in 64-bit fixed point, which loses nothing for far
// positions; its upper half, as binary32, is right to 2^-25 of a half turn.
__device__ __forceinline__ float2 turn_of(const Turns& t, int32_t position, int j) {
  const uint64_t a = t.turns[j] * static_cast<uint64_t>(static_cast<uint32_t>(position));
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(a >> 32)) * 0x1p-31f, &s, &c);
  return make_float2(c * t.gain, s * t.gain);
}

// ---------------------------------------------------------------------------
// dspark_rotary
// ---------------------------------------------------------------------------
// A thread turns `unit` u of a head: the 8 elements 8u .. 8u+7 and, with halves, their
// 8 partners; units past the turned part are copied. Its unit is the same for all the
// heads and rows it takes, so cosines and sines, made once per row and pair, are read
// from shared memory.
constexpr int kRotThreads = 256;
constexpr int kRotRows = 16;  // rows of a CTA, at most
constexpr int kRotDeep = 2;   // units in flight per thread

struct RotaryArgs {
  const uint16_t* x;
  uint16_t* out;
  int64_t row, head, orow, ohead;
  Turns t;
  int32_t n, heads, units, pair_units, rows, sign;
};

template <bool F16>
__global__ void __launch_bounds__(kRotThreads) k_rotary(const RotaryArgs a) {
  __shared__ float s_cos[kRotRows * kMaxPairs], s_sin[kRotRows * kMaxPairs];
  __shared__ int32_t s_pos[kRotRows];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, pairs = a.t.rot / 2;
  const int r0 = blockIdx.x * a.rows, rows = min(a.rows, a.n - r0);
  const int u = tid % a.units, lane = tid / a.units, lanes = kRotThreads / a.units;
  const bool turns = u < a.pair_units, halves = !a.t.inter;
  const int d0 = halves && !turns ? a.t.rot + 8 * (u - a.pair_units) : 8 * u;
  const int items = lane < lanes ? rows * a.heads : 0;
  bool ready = false;
  for (int i0 = lane;; i0 += kRotDeep * lanes) {
    uint4 x[kRotDeep], y[kRotDeep];
    int row[kRotDeep];
#pragma unroll
    for (int k = 0; k < kRotDeep; ++k) {
      const int i = i0 + k * lanes;
      row[k] = -1;
      if (i >= items) continue;
      row[k] = i / a.heads;
      const uint16_t* from = a.x + (r0 + row[k]) * a.row + (i - row[k] * a.heads) * a.head + d0;
      x[k] = *reinterpret_cast<const uint4*>(from);
      if (halves && turns) y[k] = *reinterpret_cast<const uint4*>(from + pairs);
    }
    if (!ready) {
      for (int i = tid; i < rows * pairs; i += kRotThreads) {
        const int r = i / pairs, j = i - r * pairs;
        const float2 cs = turn_of(a.t, a.t.positions[r0 + r], j);
        s_cos[r * kMaxPairs + j] = cs.x;
        s_sin[r * kMaxPairs + j] = a.sign * cs.y;
      }
      if (tid < rows) s_pos[tid] = a.t.positions[r0 + tid];
      __syncthreads();
      ready = true;
    }
    if (i0 >= items) break;
#pragma unroll
    for (int k = 0; k < kRotDeep; ++k) {
      if (row[k] < 0 || s_pos[row[k]] < 0) continue;
      const int i = i0 + k * lanes;
      uint16_t* to = a.out + (r0 + row[k]) * a.orow + (i - row[k] * a.heads) * a.ohead + d0;
      uint32_t v[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
      if (turns && halves) {
        uint32_t w[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
        const float* c = s_cos + row[k] * kMaxPairs + d0;
        const float* s = s_sin + row[k] * kMaxPairs + d0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 p = word_to_f32<F16>(v[q]), r = word_to_f32<F16>(w[q]);
          const float2 cc = *reinterpret_cast<const float2*>(c + 2 * q);
          const float2 ss = *reinterpret_cast<const float2*>(s + 2 * q);
          v[q] = f32_to_word<F16>(p.x * cc.x - r.x * ss.x, p.y * cc.y - r.y * ss.y);
          w[q] = f32_to_word<F16>(r.x * cc.x + p.x * ss.x, r.y * cc.y + p.y * ss.y);
        }
        *reinterpret_cast<uint4*>(to + pairs) = make_uint4(w[0], w[1], w[2], w[3]);
      } else if (turns) {
        const float4 c = *reinterpret_cast<const float4*>(s_cos + row[k] * kMaxPairs + 4 * u);
        const float4 s = *reinterpret_cast<const float4*>(s_sin + row[k] * kMaxPairs + 4 * u);
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 p = word_to_f32<F16>(v[q]);
          v[q] = f32_to_word<F16>(p.x * cc[q] - p.y * ss[q], p.y * cc[q] + p.x * ss[q]);
        }
      }
      *reinterpret_cast<uint4*>(to) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// dspark_kv_append_q8
// ---------------------------------------------------------------------------
// A run is the neighbouring rows of slot_map that one block takes. A CTA takes the
// runs that begin among its kChunk rows, in batches of whole runs of kBatch rows at
// most (a longer run by itself, in pieces, twice: its size first). A group of D / 8
// lanes has a batch's rows of one head of K or V in registers, 8 elements a lane, finds
// the size of every run, then the scales, and writes the codes.
// CTA 0 only judges the slots, so that one CTA writes the status.
constexpr int kQ8Threads = 256;
constexpr int kChunk = 16, kBatch = 16;

struct AppendQ8Args {
  const uint16_t *k, *v;
  uint8_t *kc, *vc;
  float *ks, *vs;
  const int32_t* slots;
  int32_t* status;
  int64_t row, head;                  // of k and v, elements
  int64_t page, token, chead;         // of the codes, bytes
  int64_t spage, sblock, shead;       // of the scales, elements
  Turns t;
  int32_t n, heads, n_slots, p_shift, b_shift;
};

// the smallest e >= -126 with a <= 448 * 2^e, as the bits of 2^e; a: bits of a finite
// magnitude
__device__ __forceinline__ float scale_for(uint32_t a) {
  const int e = static_cast<int>(a >> 23) - 127 - 8 + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}
// Quantised with 1 / s where that is exact.
__device__ __forceinline__ bool power_of_two(float s) {
  return (__float_as_uint(s) & 0x7FFFFFu) == 0;
}

template <int D, bool F16, int ROT>  // ROT: 0 none, 1 halves, 2 neighbours
__global__ void __launch_bounds__(kQ8Threads) k_kv_append_q8(const AppendQ8Args a) {
  constexpr int LPR = D / 8;                   // lanes of a group
  constexpr int kGroups = kQ8Threads / LPR;
  constexpr int kTrig = ROT ? kBatch * kMaxPairs : 1;
  __shared__ alignas(16) float s_cos[kTrig], s_sin[kTrig];
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, wl = tid & 31, lane = tid % LPR, group = tid / LPR;
  if (blockIdx.x == 0) {
    bool bad = false;
#pragma unroll 8
    for (int i = tid; i < a.n; i += kQ8Threads) bad |= a.slots[i] >= a.n_slots;
    const int any = __syncthreads_or(bad);
    if (tid == 0) *a.status = any ? DSPARK_ERR_BAD_DATA : DSPARK_OK;
    return;
  }
  const int bmask = (1 << a.b_shift) - 1, pmask = (1 << a.p_shift) - 1;
  auto slot_of = [&](int i) {  // -1: nothing to write
    if (i < 0 || i >= a.n) return -1;
    int32_t s = a.slots[i];
    if (s >= a.n_slots) s = -1;
    if (ROT && a.t.positions[i] < 0) s = -1;
    return s;
  };
  const int r0 = (blockIdx.x - 1) * kChunk;
  // rows r0 - 1 + wl in the lanes: which begin a run, which count
  const int my_slot = slot_of(r0 - 1 + wl);
  const int my_block = my_slot < 0 ? -1 : my_slot >> a.b_shift;
  const int before = __shfl_up_sync(0xFFFFFFFFu, my_block, 1);
  const uint32_t begins = __ballot_sync(0xFFFFFFFFu, wl > 0 && my_block >= 0 && my_block != before) >> 1;
  const uint32_t counts = __ballot_sync(0xFFFFFFFFu, my_block >= 0) >> 1;  // bit j: row r0 + j
  auto run_end = [&](int j) -> int {  // of the run that begins at row r0 + j, relative
    const uint32_t past = ~((2u << j) - 1u);
    const uint32_t stop = (begins | ~counts) & past & 0x7FFFFFFFu;
    if (stop) return __ffs(stop) - 1;
    const int block = __shfl_sync(0xFFFFFFFFu, my_block, j + 1);
    for (int i = r0 + 31;; i += 32) {
      const int s = slot_of(i + wl);
      const uint32_t other = __ballot_sync(0xFFFFFFFFu, s < 0 || (s >> a.b_shift) != block);
      if (other) return i - r0 + __ffs(other) - 1;
    }
  };
  uint32_t todo = begins & ((1u << kChunk) - 1u);
  const int rounds = (2 * a.heads + kGroups - 1) / kGroups;

  while (todo) {
    const int j0 = __ffs(todo) - 1;
    int end = run_end(j0);
    todo &= todo - 1;
    while (todo) {  // runs that fit in the batch
      const int e = run_end(__ffs(todo) - 1);
      if (e - j0 > kBatch) break;
      end = e;
      todo &= todo - 1;
    }
    const int s0 = r0 + j0, rows = end - j0;
    const bool one = rows <= kBatch;
    // rows s0 + wl in the lanes
    auto trig = [&](int from, int n) {  // of rows from .. from + n - 1
      if constexpr (ROT != 0) {
        const int pairs = a.t.rot / 2;
        __syncthreads();
        for (int i = tid; i < n * pairs; i += kQ8Threads) {
          const int r = i / pairs, j = i - r * pairs;
          const float2 cs = turn_of(a.t, a.t.positions[from + r], j);
          s_cos[r * kMaxPairs + j] = cs.x;
          s_sin[r * kMaxPairs + j] = cs.y;
        }
        __syncthreads();
      }
    };
    if (one) trig(s0, rows);
    for (int round = 0; round < rounds; ++round) {
      const int task = round * kGroups + group;
      const bool active = task < 2 * a.heads;
      const bool value = task >= a.heads;
      const int head = active ? (value ? task - a.heads : task) : 0;
      const uint16_t* const in = (value ? a.v : a.k) + head * a.head + 8 * lane;
      uint8_t* const codes = (value ? a.vc : a.kc) + head * a.chead + 8 * lane;
      float* const scales = (value ? a.vs : a.ks) + head * a.shead;
      // 8 elements of a row in binary32, turned if they are of a key; r: row of the trig
      auto elements = [&](const uint4& w, int r, float (&y)[8]) {
        const uint32_t own[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 p = word_to_f32<F16>(own[q]);
          y[2 * q] = p.x, y[2 * q + 1] = p.y;
        }
        if constexpr (ROT == 1) {
          const int half = a.t.rot / 16;  // lanes of a half
          const int other = lane < half ? lane + half : lane < 2 * half ? lane - half : lane;
          uint32_t got[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) got[q] = __shfl_sync(0xFFFFFFFFu, own[q], other, LPR);
          if (!value && lane < 2 * half) {
            const int j = 8 * (lane < half ? lane : lane - half);
            const float sign = lane < half ? -1.f : 1.f;
            const float* c = s_cos + r * kMaxPairs + j;
            const float* s = s_sin + r * kMaxPairs + j;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 p = word_to_f32<F16>(got[q]);
              y[2 * q] = fmaf(y[2 * q], c[2 * q], sign * p.x * s[2 * q]);
              y[2 * q + 1] = fmaf(y[2 * q + 1], c[2 * q + 1], sign * p.y * s[2 * q + 1]);
            }
          }
        }
        if constexpr (ROT == 2) {
          if (!value && 8 * lane < a.t.rot) {
            const float* c = s_cos + r * kMaxPairs + 4 * lane;
            const float* s = s_sin + r * kMaxPairs + 4 * lane;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float p = y[2 * q], o = y[2 * q + 1];
              y[2 * q] = fmaf(p, c[q], -o * s[q]);
              y[2 * q + 1] = fmaf(o, c[q], p * s[q]);
            }
          }
        }
      };
      auto size_of = [&](const float (&y)[8]) {  // bits of the largest finite magnitude
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t b = __float_as_uint(y[q]) & 0x7FFFFFFFu;
          m = max(m, b < 0x7F800000u ? b : 0u);
        }
        return m;
      };
      auto over_group = [&](uint32_t m) {
#pragma unroll
        for (int o = LPR / 2; o >= 1; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        return m;
      };
      auto put = [&](int slot, const float (&y)[8], float s) {
        uint32_t lo, hi;
        float z[8];
        if (power_of_two(s)) {
          const float inv = 1.f / s;
#pragma unroll
          for (int q = 0; q < 8; ++q) z[q] = y[q] * inv;
        } else {
#pragma unroll
          for (int q = 0; q < 8; ++q) z[q] = __fdiv_rn(y[q], s);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (fabsf(y[q]) == INFINITY) z[q] = NAN;
        lo = e4m3x4(z[0], z[1], z[2], z[3]);
        hi = e4m3x4(z[4], z[5], z[6], z[7]);
        *reinterpret_cast<uint2*>(codes + (slot >> a.p_shift) * a.page +
                                  (slot & pmask) * a.token) = make_uint2(lo, hi);
      };
      // The scale of the run whose rows have this size, with its block's other tokens
      // rounded again where it rises.
      auto settle = [&](int slot, bool fresh, uint32_t size) {
        float* const at = scales + (slot >> a.p_shift) * a.spage +
                          ((slot & pmask) >> a.b_shift) * a.sblock;
        float s = scale_for(size);
        const float old = fresh ? 0.f : *at;
        if (is_scale(old)) {
          if (__uint_as_float(size) <= 448.f * old) {
            s = old;
          } else {
            const float f = old / s;  // 2^e > old
            uint8_t* const first = codes + (slot >> a.p_shift) * a.page +
                                   ((slot & pmask) & ~bmask) * a.token;
            for (int t = 0; t <= bmask; ++t) {
              uint2* const p = reinterpret_cast<uint2*>(first + t * a.token);
              const uint2 c = *p;
              const float2 c0 = e4m3x2_to_f32(c.x), c1 = e4m3x2_to_f32(c.x >> 16);
              const float2 c2 = e4m3x2_to_f32(c.y), c3 = e4m3x2_to_f32(c.y >> 16);
              *p = make_uint2(e4m3x4(c0.x * f, c0.y * f, c1.x * f, c1.y * f),
                              e4m3x4(c2.x * f, c2.y * f, c3.x * f, c3.y * f));
            }
          }
        }
        __syncwarp(LPR == 32 ? 0xFFFFFFFFu : ((1u << LPR) - 1u) << (wl & ~(LPR - 1)));
        if (lane == 0) *at = s;  // every lane has read it
        return s;
      };
      if (one) {
        const int slot_l = wl < rows ? slot_of(s0 + wl) : -1;
        const uint32_t live = __ballot_sync(0xFFFFFFFFu, slot_l >= 0);
        const uint32_t starts = (begins >> j0) & ((1u << rows) - 1u);
        // which of the lanes' rows are in a run that has its block's first token
        const uint32_t zero = __ballot_sync(0xFFFFFFFFu, slot_l >= 0 && (slot_l & bmask) == 0);
        const uint32_t upto = (2u << wl) - 1u;  // (lane 31: all)
        const int from = 31 - __clz(starts & upto);
        const uint32_t later = starts & ~upto;
        const uint32_t mine = (later ? (1u << (__ffs(later) - 1)) - 1u : 0xFFFFFFFFu) &
                              ~((1u << from) - 1u);
        const uint32_t fresh = __ballot_sync(0xFFFFFFFFu, (zero & mine) != 0);
        uint4 x[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          x[j] = make_uint4(0, 0, 0, 0);
          if (active && (live >> j) & 1u)
            x[j] = *reinterpret_cast<const uint4*>(in + (s0 + j) * a.row);
        }
        uint32_t size[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          size[j] = 0;
          if (j < rows) {
            float y[8];
            elements(x[j], j, y);
            size[j] = over_group(size_of(y));
          }
        }
        // of a run: in its first row
#pragma unroll
        for (int j = kBatch - 2; j >= 0; --j)
          if (!((starts >> (j + 1)) & 1u)) size[j] = max(size[j], size[j + 1]);
        float s = 1.f;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (j >= rows) break;
          const int slot = __shfl_sync(0xFFFFFFFFu, slot_l, j);
          if (active && (starts >> j) & 1u) s = settle(slot, (fresh >> j) & 1u, size[j]);
          __syncwarp();
          float y[8];
          elements(x[j], j, y);
          if (active && slot >= 0) put(slot, y, s);
        }
      } else {
        // a run of more rows than the registers hold
        uint32_t size = 0;
        bool fresh = false;
        for (int b = 0; b < rows; b += kBatch) {
          const int m = min(kBatch, rows - b);
          trig(s0 + b, m);
#pragma unroll 4
          for (int j = 0; j < m; ++j) {
            const int slot = slot_of(s0 + b + j);
            fresh |= slot >= 0 && (slot & bmask) == 0;
            const uint4 x = *reinterpret_cast<const uint4*>(in + (s0 + b + j) * a.row);
            float y[8];
            elements(x, j, y);
            size = max(size, size_of(y));
          }
        }
        size = over_group(size);
        float s = 1.f;
        if (active) s = settle(slot_of(s0), fresh, size);
        __syncwarp();
        for (int b = 0; b < rows; b += kBatch) {
          const int m = min(kBatch, rows - b);
          trig(s0 + b, m);
#pragma unroll 4
          for (int j = 0; j < m; ++j) {
            const uint4 x = *reinterpret_cast<const uint4*>(in + (s0 + b + j) * a.row);
            float y[8];
            elements(x, j, y);
            if (active) put(slot_of(s0 + b + j), y, s);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// dspark_kv_gather_q8
// ---------------------------------------------------------------------------
constexpr int kGatherPieces = 4;

struct GatherQ8Args {
  const uint8_t *kc, *vc;
  const float *ks, *vs;
  uint16_t *k, *v;
  const int32_t* slots;
  int32_t* status;
  int64_t row, head, page, token, chead, spage, sblock, shead;
  int32_t n, pieces, d_shift, n_slots, p_shift, b_shift, rows;  // pieces of 8 per row
};

template <bool F16>
__global__ void __launch_bounds__(kQ8Threads) k_kv_gather_q8(const GatherQ8Args a) {
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) {
    bool bad = false;
#pragma unroll 8
    for (int i = tid; i < a.n; i += kQ8Threads) bad |= a.slots[i] >= a.n_slots;
    const int any = __syncthreads_or(bad);
    if (tid == 0) *a.status = any ? DSPARK_ERR_BAD_DATA : DSPARK_OK;
    return;
  }
  const int pmask = (1 << a.p_shift) - 1, dmask = (1 << a.d_shift) - 1;
  for (int64_t r0 = (blockIdx.x - 1) * static_cast<int64_t>(a.rows); r0 < a.n;
       r0 += (gridDim.x - 1) * static_cast<int64_t>(a.rows)) {
    const int rows = static_cast<int>(min(static_cast<int64_t>(a.rows), a.n - r0));
    const int total = rows * a.pieces;
    for (int i0 = tid; i0 < total; i0 += kGatherPieces * kQ8Threads) {
      uint2 k[kGatherPieces], v[kGatherPieces];
      float ks[kGatherPieces], vs[kGatherPieces];
      int64_t to[kGatherPieces];
#pragma unroll
      for (int j = 0; j < kGatherPieces; ++j) {
        const int i = i0 + j * kQ8Threads;
        to[j] = -1;
        if (i >= total) continue;
        const int q = i / a.pieces, w = i - q * a.pieces;
        const int64_t head = w >> a.d_shift;
        const int d = 8 * (w & dmask);
        const int32_t s = a.slots[r0 + q];
        if (s < 0 || s >= a.n_slots) continue;
        to[j] = (r0 + q) * a.row + head * a.head + d;
        const int64_t page = s >> a.p_shift, t = s & pmask;
        const int64_t from = page * a.page + t * a.token + head * a.chead + d;
        const int64_t sf = page * a.spage + (t >> a.b_shift) * a.sblock + head * a.shead;
        k[j] = *reinterpret_cast<const uint2*>(a.kc + from);
        v[j] = *reinterpret_cast<const uint2*>(a.vc + from);
        ks[j] = a.ks[sf];
        vs[j] = a.vs[sf];
      }
      auto wide = [](const uint2& c, float s) {
        const float2 c0 = e4m3x2_to_f32(c.x), c1 = e4m3x2_to_f32(c.x >> 16);
        const float2 c2 = e4m3x2_to_f32(c.y), c3 = e4m3x2_to_f32(c.y >> 16);
        return make_uint4(f32_to_word<F16>(c0.x * s, c0.y * s), f32_to_word<F16>(c1.x * s, c1.y * s),
                          f32_to_word<F16>(c2.x * s, c2.y * s), f32_to_word<F16>(c3.x * s, c3.y * s));
      };
#pragma unroll
      for (int j = 0; j < kGatherPieces; ++j)
        if (to[j] >= 0) {
          *reinterpret_cast<uint4*>(a.k + to[j]) = wide(k[j], ks[j]);
          *reinterpret_cast<uint4*>(a.v + to[j]) = wide(v[j], vs[j]);
        }
    }
  }
}

// ---------------------------------------------------------------------------
// host checks
// ---------------------------------------------------------------------------
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int shift_of(int32_t v, int lo, int hi) {  // of a power of two in [2^lo, 2^hi]
  for (int s = lo; s <= hi; ++s)
    if (v == 1 << s) return s;
  return -1;
}

bool turns_ok(const dspark_rotation* r, int32_t D) {
  return r->turns && r->rot_dim >= 16 && r->rot_dim <= D && r->rot_dim % 16 == 0 &&
         (r->pairs == DSPARK_ROTARY_HALF || r->pairs == DSPARK_ROTARY_INTERLEAVED) &&
         std::isfinite(r->gain);
}

// what the append and the gather have in common
bool cache_ok(int32_t n, int32_t Hkv, int32_t D, int32_t dtype, int64_t page_stride,
              int64_t token_stride, int64_t head_stride, int64_t spage, int64_t sblock,
              int64_t shead, int32_t block, int32_t page_size, int32_t num_pages) {
  return n >= 0 && Hkv >= 1 && Hkv <= 65536 && (D == 64 || D == 128) &&
         (dtype == DSPARK_BF16 || dtype == DSPARK_F16) && shift_of(page_size, 3, 10) >= 0 &&
         shift_of(block, 0, 10) >= 0 && block <= page_size && num_pages >= 1 &&
         static_cast<int64_t>(num_pages) * page_size <= INT32_MAX && page_stride >= 0 &&
         token_stride >= 0 && head_stride >= 0 && spage >= 0 && sblock >= 0 && shead >= 0 &&
         ((page_stride | token_stride | head_stride) & 15) == 0;
}

template <int D, bool F16>
cudaError_t append_launch(const AppendQ8Args& a, int rot, int grid, cudaStream_t st) {
  if (rot == 0) return launch_pdl(k_kv_append_q8<D, F16, 0>, grid, kQ8Threads, 0, st, a);
  if (rot == 1) return launch_pdl(k_kv_append_q8<D, F16, 1>, grid, kQ8Threads, 0, st, a);
  return launch_pdl(k_kv_append_q8<D, F16, 2>, grid, kQ8Threads, 0, st, a);
}

}  // namespace
}  // namespace dspark

using namespace dspark;

extern "C" int dspark_rotary(const void* x, int64_t row_stride, int64_t head_stride,
                             const int32_t* positions, const dspark_rotation* rotation,
                             int32_t inverse, int32_t n, int32_t heads, int32_t D, int32_t dtype,
                             void* out, int64_t out_row_stride, int64_t out_head_stride,
                             struct CUstream_st* stream) {
  if (!rotation || n < 0 || heads < 1 || heads > 65536 || (D != 64 && D != 128) ||
      (dtype != DSPARK_BF16 && dtype != DSPARK_F16) || (inverse != 0 && inverse != 1) ||
      !turns_ok(rotation, D) || row_stride < 0 || head_stride < 0 || out_row_stride < 0 ||
      out_head_stride < 0 ||
      ((row_stride | head_stride | out_row_stride | out_head_stride) & 7) != 0 ||
      !aligned16(x) || !aligned16(out) || (n > 0 && (!x || !out || !positions)) ||
      (x == out && n > 0 && (row_stride != out_row_stride || head_stride != out_head_stride)))
    return DSPARK_ERR_INVALID_ARG;
  if (n == 0) return DSPARK_OK;
  RotaryArgs a{};
  a.x = static_cast<const uint16_t*>(x), a.out = static_cast<uint16_t*>(out);
  a.row = row_stride, a.head = head_stride, a.orow = out_row_stride, a.ohead = out_head_stride;
  a.t = Turns{rotation->turns, positions, rotation->gain, rotation->rot_dim,
              rotation->pairs == DSPARK_ROTARY_INTERLEAVED};
  a.n = n, a.heads = heads;
  a.pair_units = rotation->rot_dim / (a.t.inter ? 8 : 16);
  a.units = a.pair_units + (D - rotation->rot_dim) / 8;
  a.sign = inverse ? -1 : 1;
  a.rows = std::clamp(kRotDeep * (kRotThreads / a.units) / heads, 1, kRotRows);
  const int grid = static_cast<int>(DSPARK_CEILDIV(n, a.rows));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t rc = dtype == DSPARK_F16
                             ? launch_pdl(k_rotary<true>, grid, kRotThreads, 0, st, a)
                             : launch_pdl(k_rotary<false>, grid, kRotThreads, 0, st, a);
  return rc == cudaSuccess && cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

extern "C" int dspark_kv_append_q8(
    const void* k, const void* v, int64_t row_stride, int64_t in_head_stride,
    const dspark_rotation* rotation, const int32_t* positions, const int32_t* slot_map, int32_t n,
    int32_t Hkv, int32_t D, int32_t dtype, void* k_cache, void* v_cache, int64_t page_stride,
    int64_t token_stride, int64_t head_stride, float* k_scale, float* v_scale,
    int64_t scale_page_stride, int64_t scale_block_stride, int64_t scale_head_stride,
    int32_t block, int32_t page_size, int32_t num_pages, int32_t* device_status,
    struct CUstream_st* stream) {
  if (!cache_ok(n, Hkv, D, dtype, page_stride, token_stride, head_stride, scale_page_stride,
                scale_block_stride, scale_head_stride, block, page_size, num_pages) ||
      !device_status || row_stride < 0 || in_head_stride < 0 ||
      ((row_stride | in_head_stride) & 7) != 0 || !aligned16(k) || !aligned16(v) ||
      !aligned16(k_cache) || !aligned16(v_cache) ||
      (n > 0 && (!k || !v || !slot_map || !k_cache || !v_cache || !k_scale || !v_scale)) ||
      (rotation && (!turns_ok(rotation, D) || (n > 0 && !positions))))
    return DSPARK_ERR_INVALID_ARG;
  AppendQ8Args a{};
  a.k = static_cast<const uint16_t*>(k), a.v = static_cast<const uint16_t*>(v);
  a.kc = static_cast<uint8_t*>(k_cache), a.vc = static_cast<uint8_t*>(v_cache);
  a.ks = k_scale, a.vs = v_scale, a.slots = slot_map, a.status = device_status;
  a.row = row_stride, a.head = in_head_stride, a.page = page_stride, a.token = token_stride;
  a.chead = head_stride, a.spage = scale_page_stride, a.sblock = scale_block_stride;
  a.shead = scale_head_stride, a.n = n, a.heads = Hkv, a.n_slots = num_pages * page_size;
  a.p_shift = shift_of(page_size, 3, 10), a.b_shift = shift_of(block, 0, 10);
  int rot = 0;
  if (rotation) {
    a.t = Turns{rotation->turns, positions, rotation->gain, rotation->rot_dim,
                rotation->pairs == DSPARK_ROTARY_INTERLEAVED};
    rot = a.t.inter ? 2 : 1;
  }
  const int grid = 1 + static_cast<int>(DSPARK_CEILDIV(n, kChunk));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool f16 = dtype == DSPARK_F16;
  const cudaError_t rc = D == 64 ? (f16 ? append_launch<64, true>(a, rot, grid, st)
                                        : append_launch<64, false>(a, rot, grid, st))
                                 : (f16 ? append_launch<128, true>(a, rot, grid, st)
                                        : append_launch<128, false>(a, rot, grid, st));
  return rc == cudaSuccess && cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

extern "C" int dspark_kv_gather_q8(
    const void* k_cache, const void* v_cache, int64_t page_stride, int64_t token_stride,
    int64_t head_stride, const float* k_scale, const float* v_scale, int64_t scale_page_stride,
    int64_t scale_block_stride, int64_t scale_head_stride, int32_t block, int32_t page_size,
    int32_t num_pages, const int32_t* slot_map, int32_t n, int32_t Hkv, int32_t D, int32_t dtype,
    void* k, void* v, int64_t row_stride, int64_t out_head_stride, int32_t* device_status,
    struct CUstream_st* stream) {
  if (!cache_ok(n, Hkv, D, dtype, page_stride, token_stride, head_stride, scale_page_stride,
                scale_block_stride, scale_head_stride, block, page_size, num_pages) ||
      !device_status || row_stride < 0 || out_head_stride < 0 ||
      ((row_stride | out_head_stride) & 7) != 0 || !aligned16(k) || !aligned16(v) ||
      !aligned16(k_cache) || !aligned16(v_cache) ||
      (n > 0 && (!k || !v || !slot_map || !k_cache || !v_cache || !k_scale || !v_scale)))
    return DSPARK_ERR_INVALID_ARG;
  GatherQ8Args a{};
  a.kc = static_cast<const uint8_t*>(k_cache), a.vc = static_cast<const uint8_t*>(v_cache);
  a.ks = k_scale, a.vs = v_scale, a.k = static_cast<uint16_t*>(k);
  a.v = static_cast<uint16_t*>(v), a.slots = slot_map, a.status = device_status;
  a.row = row_stride, a.head = out_head_stride, a.page = page_stride, a.token = token_stride;
  a.chead = head_stride, a.spage = scale_page_stride, a.sblock = scale_block_stride;
  a.shead = scale_head_stride, a.n = n, a.pieces = Hkv * (D / 8), a.d_shift = D == 64 ? 3 : 4;
  a.n_slots = num_pages * page_size, a.p_shift = shift_of(page_size, 3, 10);
  a.b_shift = shift_of(block, 0, 10);
  a.rows = std::max(1, kGatherPieces * kQ8Threads / a.pieces);
  const int64_t groups = static_cast<int64_t>(DSPARK_CEILDIV(n, a.rows));
  const int grid = 1 + static_cast<int>(std::min<int64_t>(groups, 1 << 20));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t rc = dtype == DSPARK_F16
                             ? launch_pdl(k_kv_gather_q8<true>, grid, kQ8Threads, 0, st, a)
                             : launch_pdl(k_kv_gather_q8<false>, grid, kQ8Threads, 0, st, a);
  return rc == cudaSuccess && cudaGetLastError() == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
