// beam_attention: the beam rows of a step over their request's prompt cache and
// their own ancestors.
//
// OneLA (paper summary), section 3.3: a child refers to its parent's records.
// The tree of a request's beams is the back-pointer history that beam_step
// writes; nothing is copied per beam.
//
//   out[row][h] = sum_j softmax_j(scale * <q, k_j>) v_j
//
// over the cache_len[r] tokens of the prompt and the row's `level` ancestors,
// with the running maximum m and sum l of the softmax:
//   m' = max(m, x),  l' = l 2^(m - m') + 2^(x - m'),  o' = o 2^(m - m') + 2^(x - m') v.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "internal.h"
#include "tcgen05.cuh"

namespace sidbeam {
namespace {

using namespace dev;

struct AttnArgs {
  const __nv_bfloat16* q;
  int64_t q_stride;
  const __nv_bfloat16 *k, *v;
  int64_t page_stride, token_stride;
  int n_pages, page_size;
  const int32_t* table;
  int table_stride;
  const int32_t* len;
  int level;
  const int32_t* bp;
  const __nv_bfloat16 *kb, *vb;
  int R, B, H, Hkv;
  float scale_log2;  // |scale| log2(e), never 0
  uint32_t q_flip;   // sign bits of a bf16 pair: a negative scale negates q
  __nv_bfloat16* out;
  int64_t out_stride;
  uint32_t* status;
  int G;              // H / Hkv
  uint32_t g_magic;   // ceil(2^32 / G)
  int pairs, units;
  int split, split_log2;
  int page_log2;      // of page_size (with a page table)
  uint32_t level16;   // 16-byte words of a level of k_beam, v_beam
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -INFINITY;

// ------------------------------------------------------------ shape of the work
// The rows of a request's beams and of the G = H / Hkv heads that share a key head
// are one M axis, row i = b * G + head, in tiles of 128; keys come in tiles of 128.
// A CTA runs two streams, each a chain S = Q K^T, softmax, O += P V with its own
// S, P (in S's place) and O in TMEM, so that one stream's softmax runs under the
// other's MMAs.
//  kDual: a unit is two row tiles of a (request, key head); the streams take one
//         each and share every key tile, which is loaded once for both.
//  else:  a unit is one row tile; the streams take every other key tile, and the
//         two (m, l, O) are joined at its end.
// CTAs are persistent over units, with a warp group per row tile for the rows' work:
// while the streams run a unit, it scores the rows' ancestors and loads the next
// unit's Q; while they run the next one, it joins, normalises and writes. Few
// units are split over the keys among the CTAs of a cluster instead, and joined
// through distributed shared memory in rank order.
//
// What bounds it, measured with 16 query and 8 key heads of 128. Two figures: at the
// full clock of 1,965 MHz (some ms of calls after a pause), and in seconds of calls, where
// the 1,000 W power cap lowers the clock (MHz in brackets):
//  - Many rows, long prompts: the softmax, whose exponentials and conversions share
//    their issue slots with the TMEM reads. 16 requests x 512 beams: 540 us and 615 (1,732)
//    over 8192 tokens (1,018 and 894 TFLOP/s), 148 and 166 (1,750) over 2048, 83 and 91
//    (1,762) over 1024, 26 and 26 over 128.
//  - Ancestors: 1024 tokens and 1, 2 or 4 levels take 101 and 111, 107 and 117, 137 and 142
//    against 83 and 91: each row gathers its own levels' keys and values, and the rows'
//    warp groups take longer over them than the streams over the prompt.
//  - One row a head (32 requests x 5000 tokens): the cache's bytes, 6.1 TB/s and 5.4
//    (1,600) from pages of 64 (94% and 83% of the copy bandwidth).
//  - One request, one row: latency. 128 tokens take 6.0 us, 1000 tokens 8.9 (full clock).
constexpr int kRows = 128;
constexpr int kKeys = 128;
constexpr int kMaxSplitLog2 = 3;

template <int D, bool kDual>
struct Plan {
  // Warp groups: softmax 0, softmax 1, rows of tile 0, (MMA, TMA, tails, -), and
  // with two tiles the rows of tile 1.
  static constexpr int kThreads = kDual ? 640 : 512;
  static constexpr int kTiles = kDual ? 2 : 1;             // row tiles of a unit
  static constexpr int kTile = kKeys * D * 2;              // bytes of a K, V or Q tile
  static constexpr int kHalf = kKeys * 128;                // bytes of 64 of its columns
  static constexpr int kSlots = D == 128 ? (kDual ? 4 : 5) : 8;  // ring of K and V tiles
  static constexpr int kAhead = kDual ? 1 : 2;             // K tiles loaded before a V tile
  static constexpr int kLevels = kDual ? 8 : SIDBEAM_MAX_DEPTH;
  static constexpr int kScores = kTiles * kRows * kLevels * 4;
  static constexpr int kSlotTab = kTiles * kRows * kLevels * 2;
  static constexpr int kMl = 2 * kRows * 8;
  static constexpr int kRing = kTiles * kTile;             // offset of the ring (Q is first)
  static constexpr int kAfter = kRing + kSlots * kTile;
  static constexpr int kSmem = kAfter + kScores + kSlotTab + kMl + 1024;
  static constexpr int kPart = D + 4;                      // floats of a partial row: o, m, l
  static_assert(kTiles * kRows * kPart * 4 <= kAfter, "partial rows fit Q and the ring");
};

// Instruction descriptors (kind::f16, fp32 accumulator, bf16 operands, M = 128):
// S = Q K^T, both K-major, N = 128; O += P V, V with its D axis contiguous
// ("MN-major", bit 16), N = D.
constexpr uint32_t kIdescQK = (1u << 4) | (1u << 7) | (1u << 10) | ((128u >> 3) << 17) |
                              ((128u >> 4) << 24);
constexpr uint32_t idesc_pv(int d) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 16) | (static_cast<uint32_t>(d >> 3) << 17) |
         ((128u >> 4) << 24);
}

// Descriptor of a V tile as the MN-major operand: 64 columns of D (128 bytes,
// swizzled) per row of keys, 8-row atoms 1024 bytes apart (stride offset), the
// next 64 columns one half further (leading offset).
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t half_bytes) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>(half_bytes >> 4) << 16) |
         (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
         (static_cast<uint64_t>(2) << 61);
}

struct Bars {
  uint64_t full[8], empty[8];        // ring slots: loaded / multiplied
  uint64_t landed[8];                // a ragged V tile is in its slot, its tail not yet zero
  uint64_t q_full[2], q_empty[2];    // a Q tile is in place / multiplied
  uint64_t s_full[2], p_ready[2];    // a step's scores / weights in TMEM
  uint64_t ml_full[2], o_full[2];    // a unit's row maxima and sums / O complete
  uint64_t o_empty[2];               // both have been read
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

// 8 bf16 of a 16-byte word.
__device__ __forceinline__ void bf16x4(const uint2& u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x << 16);
  f[1] = __uint_as_float(u.x & 0xFFFF0000u);
  f[2] = __uint_as_float(u.y << 16);
  f[3] = __uint_as_float(u.y & 0xFFFF0000u);
}

// Byte offset of 16-byte unit c (0 .. D/8 - 1) of row `row` in a swizzled tile.
__device__ __forceinline__ uint32_t unit_at(int row, int c) {
  return static_cast<uint32_t>((c >> 3) * (kKeys * 128) + row * 128 + (((c ^ row) & 7) << 4));
}

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One unit as every role sees it.
struct Unit {
  int r, g, row0, rows;  // request, key head, first row, valid rows (of all its tiles)
  int t0, n, len;        // first key tile, key tiles, tokens of the request
  int ragged;            // keys in the last tile if it is this CTA's and not full, else 0
};

template <bool kDual>
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, int w, int rank) {
  Unit u;
  const unsigned rg = static_cast<unsigned>(w) / static_cast<unsigned>(a.pairs);
  const int pair = w - static_cast<int>(rg) * a.pairs;
  u.r = static_cast<int>(rg / static_cast<unsigned>(a.Hkv));
  u.g = static_cast<int>(rg) - u.r * a.Hkv;
  constexpr int kUnitRows = kDual ? 2 * kRows : kRows;
  u.row0 = pair * kUnitRows;
  u.rows = min(kUnitRows, a.B * a.G - u.row0);
  const int cap = a.table ? a.table_stride << a.page_log2 : a.page_size;
  u.len = max(0, min(a.len[u.r], cap));
  const int tiles = (u.len + kKeys - 1) / kKeys;  // < 2^24
  u.t0 = (tiles * rank) >> a.split_log2;
  const int t1 = (tiles * (rank + 1)) >> a.split_log2;
  u.n = t1 - u.t0;
  u.ragged = u.n > 0 && t1 == tiles ? u.len & (kKeys - 1) : 0;
  return u;
}

// Steps of stream s (key tiles it works on) and the key tile of its step j.
template <bool kDual>
__device__ __forceinline__ int steps_of(const Unit& u, int s) {
  return kDual ? (s == 0 || u.rows > kRows ? u.n : 0) : (u.n + 1 - s) >> 1;
}
template <bool kDual>
__device__ __forceinline__ int tile_of(int s, int j) {
  return kDual ? j : 2 * j + s;
}

// Positions in the load order of the T-th key tile's K and V, counted over all of
// a CTA's units: K_0 .. K_{ahead-1}, then V_T, K_{T+ahead} in turn. (The positions
// of K tiles past the last one stay unused; nothing follows in their slots.)
__device__ __forceinline__ int pos_k(int t, int ahead) { return t < ahead ? t : 2 * t - ahead + 1; }
__device__ __forceinline__ int pos_v(int t, int ahead) { return 2 * t + ahead; }

// kPath: the rows have ancestors; kSplit: units are split over clusters. (Flags of
// the instance, since every part that a kernel does not have is room in the
// instruction cache: 128 KB of code measured 15-20% slower than 96 KB.)
template <int D, bool kDual, bool kPath, bool kSplit>
__global__ void __launch_bounds__(kDual ? 640 : 512, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ AttnArgs a) {
  using P = Plan<D, kDual>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem + P::kRing;
  float* scores = reinterpret_cast<float*>(smem + P::kAfter);  // [tiles][128][kLevels]
  uint16_t* slots = reinterpret_cast<uint16_t*>(scores + P::kScores / 4);
  float2* ml = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(slots) + P::kSlotTab);
  __shared__ Bars bar;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = kSplit ? static_cast<int>(cluster_rank()) : 0;
  const int first_unit = static_cast<int>(blockIdx.x) >> a.split_log2;
  const int stride = kSplit ? a.units : static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.empty[s], 1);
      mbar_init(&bar.landed[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar.q_full[s], 4);
      mbar_init(&bar.q_empty[s], 1);
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.p_ready[s], 4);
      mbar_init(&bar.ml_full[s], 4);
      mbar_init(&bar.o_full[s], 1);
      mbar_init(&bar.o_empty[s], 4);
    }
    mbar_init(&bar.drain, 1);
    bar.abort = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(&bar.tmem, 512);
  wait_prior();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  release_next();
  // All 512 columns are this CTA's, so they begin at column 0.
  constexpr uint32_t tmem = 0u;
  const int quarter = warp & 3;
  const uint32_t quad = static_cast<uint32_t>(quarter * 32) << 16;  // a warp's TMEM lanes

  // Registers: 640 threads start with 96 each: 96 + 96 + 120 + 120 + 48 = 5 * 96;
  // 512 start with 128 each: 160 + 160 + 136 + 56 = 4 * 128.
  if (warp >= 12 && warp < 16) {
    if constexpr (kDual)
      asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    if (warp == 12) {
      // -------------------------------------------------------- MMA issue
      // One thread for both streams, in the order of the loads. (A thread per
      // stream keeps the two in step, so that they want the exponentials, and then
      // the tensor core, at the same time: measured 13% slower. And where it saw
      // only its stream's slots it could take an older phase of a slot for the one
      // it waits for: a wait tells phases apart by parity alone.)
      // What stands between a step's weights and the next scores is on the path
      // of every step, so a step's other waits (its V, the next K) come first, and
      // its two products are issued back to back.
      if (elect_one()) {
        bool ok = true;
        auto wait = [&](uint64_t* b, int phase) {
          ok = ok && lane_wait(b, static_cast<uint32_t>(phase), &bar.abort, a.status);
        };
        auto wait_load = [&](int pos) { wait(&bar.full[pos % P::kSlots], pos / P::kSlots); };
        const uint32_t ring_at = smem_addr(ring);
        const uint64_t q0 = smem_desc(smem_addr(smem));
        // S of stream s from the K tile at a position of the ring.
        auto qk = [&](int s, int pos) {
          const uint64_t k = smem_desc(ring_at + (pos % P::kSlots) * P::kTile);
          const uint64_t q = q0 + (kDual && s ? P::kTile >> 4 : 0);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * P::kHalf + (kk & 3) * 32) >> 4;
            umma_f16(tmem + s * kKeys, q + off, k + off, kIdescQK, kk > 0 ? 1u : 0u);
          }
          umma_commit(&bar.s_full[s]);
        };
        // O of stream s += P V with the V tile at a position of the ring.
        auto pv = [&](int s, int pos, bool first) {
          const uint64_t v = smem_desc_mn(ring_at + (pos % P::kSlots) * P::kTile, P::kHalf);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
            umma_f16_ts(tmem + 256 + s * 128, tmem + s * kKeys + kk * 8, v + kk * (2048 >> 4),
                        idesc_pv(D), kk > 0 || !first ? 1u : 0u);
        };
        auto free_slot = [&](int pos) { umma_commit(&bar.empty[pos % P::kSlots]); };
        int base = 0, units = 0, units1 = 0;  // tiles and units behind (of stream 1)
        int count0 = 0, count1 = 0;           // steps behind, of each stream
        if constexpr (kDual) {
          auto next = [&](int& w, Unit& u) {  // the next unit with key tiles
            for (; w < a.units; w += stride) {
              u = unit_of<kDual>(a, w, rank);
              if (u.n > 0) {
                w += stride;
                return true;
              }
            }
            return false;
          };
          int w = first_unit;
          Unit u;
          bool have = next(w, u);
          bool out0 = false, out1 = false;  // the unit's first products are out
          while (ok && have) {
            const bool two = u.rows > kRows;
            const int n = u.n;
            const bool more = next(w, u);
            const bool two_next = more && u.rows > kRows;
            const bool begun0 = out0, begun1 = out1;
            out0 = out1 = false;
            // Step j of stream s, then the stream's next product: of this unit, or
            // the first of the next one (before step 0: this unit's first, where
            // the unit before did not leave it behind).
#pragma unroll 1
            for (int e = -2; ok && e < 2 * n; ++e) {
              const int j = e >> 1, s = e & 1;
              if (s && !two) continue;
              if (j < 0 && (s ? begun1 : begun0)) continue;
              const int behind = s ? units1 : units;
              const bool last = j + 1 == n, closing = s || !two;
              const int vp = pos_v(base + j, 1), kp = pos_k(base + j + 1, 1);
              // (Stream 1 finds the loads that stream 0 has waited for.)
              if (!last) {
                if (j < 0) wait(&bar.q_full[s], behind);
                if (s == 0) wait_load(kp);
              }
              if (j >= 0) {
                if (s == 0) wait_load(vp);
                if (j == 0 && behind > 0) wait(&bar.o_empty[s], behind - 1);
                wait(&bar.p_ready[s], s ? count1++ : count0++);
                if (!ok) break;
                tc_fence_after();
                pv(s, vp, j == 0);
              }
              if (last) {
                umma_commit(&bar.o_full[s]);
                if (closing) free_slot(vp);
                if (!(s ? two_next : more)) continue;
                wait(&bar.q_full[s], behind + 1);
                if (s == 0) wait_load(kp);
                if (s) out1 = true; else out0 = true;
              }
              if (!ok) break;
              tc_fence_after();
              qk(s, kp);
              if (last ? s || !two_next : closing) free_slot(kp);
              if (last ? u.n == 1 : j + 2 == n) umma_commit(&bar.q_empty[s]);
              if (j >= 0 && !last && closing) free_slot(vp);
            }
            ++units;
            if (two) ++units1;
            base += n;
            have = more;
          }
        } else {
#pragma unroll 1
          for (int w = first_unit; ok && w < a.units; w += stride) {
            const Unit u = unit_of<kDual>(a, w, rank);
            if (u.n == 0) continue;
            wait(&bar.q_full[0], units);
            // Two products ahead of the first weights, then in turn.
#pragma unroll 1
            for (int i = -2; ok && i < u.n; ++i) {
              const int s = i & 1;
              const int vp = pos_v(base + i, 2), kp = pos_k(base + i + 2, 2);
              if (i >= 0) wait_load(vp);
              if (i + 2 < u.n) wait_load(kp);
              if (i >= 0) {
                const int behind = s ? units1 : units;
                if (i < 2 && behind > 0) wait(&bar.o_empty[s], behind - 1);
                wait(&bar.p_ready[s], s ? count1++ : count0++);
              }
              if (!ok) break;
              tc_fence_after();
              if (i >= 0) pv(s, vp, i < 2);
              if (i + 2 < u.n) {
                qk(s, kp);
                free_slot(kp);
                if (i + 3 == u.n) umma_commit(&bar.q_empty[0]);
              } else if (i >= 0) {
                umma_commit(&bar.o_full[s]);
              }
              if (i >= 0) free_slot(vp);
            }
            ++units;
            if (u.n > 1) ++units1;
            base += u.n;
          }
        }
        umma_commit(&bar.drain);
        drain_wait(&bar.drain, 0u);
      }
      __syncwarp();
    } else if (warp == 13) {
      // -------------------------------------------------------- loads
      const int box = a.table ? min(a.page_size, kKeys) : kKeys;  // tokens of one copy
      const int boxes = kKeys / box;
      const int my_box = lane & (boxes - 1), my_half = lane / boxes;
      const bool mine = my_half < D / 64;
      if (lane == 0) {
        prefetch_map(&map_k);
        prefetch_map(&map_v);
      }
      // Two cursors over the same sequence of (unit, key tile).
      struct Cursor {
        int w, i, t;  // next unit index, tile of the unit, tiles loaded
        Unit u;
      };
      auto advance = [&](Cursor& c) {  // to the next tile; false past the last
        ++c.i;
        while (c.i >= c.u.n) {
          c.w += stride;
          if (c.w >= a.units) return false;
          c.u = unit_of<kDual>(a, c.w, rank);
          if (lane == 0 && c.u.len != a.len[c.u.r]) atomicOr(a.status, kStatusBadCache);
          c.i = 0;
        }
        return true;
      };
      Cursor ck{first_unit - stride, 0, 0, {}}, cv;
      ck.u.n = 0;
      bool more_k = advance(ck);
      cv = ck;
      bool more_v = more_k;
      int top = 0;  // positions issued
      bool ok = true;
#pragma unroll 1
      while (ok && (more_k || more_v)) {
        const bool is_k = more_k && ck.t < cv.t + P::kAhead;
        const Cursor& c = is_k ? ck : cv;
        const int pos = is_k ? pos_k(ck.t, P::kAhead) : pos_v(cv.t, P::kAhead);
        const int tile = c.u.t0 + c.i;
        const int token = tile * kKeys + my_box * box;
        const bool issue = mine && token < c.u.len;
        int page = c.u.r, at = token;
        if (a.table) {
          at = token & (a.page_size - 1);
          if (issue) {
            page = a.table[static_cast<int64_t>(c.u.r) * a.table_stride + (token >> a.page_log2)];
            if (page < 0 || page >= a.n_pages) {
              atomicOr(a.status, kStatusBadCache);
              page = a.n_pages;  // outside the tensor: the copy writes zeros
            }
          }
        }
        const int s = pos % P::kSlots;
        if (pos >= P::kSlots &&
            !warp_wait(&bar.empty[s], (pos / P::kSlots) - 1, &bar.abort, a.status)) {
          ok = false;
          break;
        }
        const int count = min(boxes, (c.u.len - tile * kKeys + box - 1) / box);
        // (A ragged V tile is handed on by the warp that clears its tail.)
        uint64_t* to = !is_k && c.u.ragged && c.i == c.u.n - 1 ? &bar.landed[s] : &bar.full[s];
        if (lane == 0) mbar_arrive_expect_tx(to, count * (D / 64) * box * 128);
        __syncwarp();
        if (issue)
          tma_load_4d(smem_addr(ring + s * P::kTile + my_half * P::kHalf + my_box * box * 128),
                      is_k ? &map_k : &map_v, my_half * 64, c.u.g, at, page, to);
        __syncwarp();
        top = pos + 1;
        if (is_k) {
          ++ck.t;
          more_k = advance(ck);
        } else {
          ++cv.t;
          more_v = advance(cv);
        }
      }
      // Copies in flight land before the CTA goes away (normally all have).
#pragma unroll 1
      for (int p = max(0, top - P::kSlots); p < top; ++p) {
        // Position p was issued unless it is that of a K tile past the last one.
        const bool v_pos = p >= P::kAhead && ((p - P::kAhead) & 1) == 0;
        const int t = v_pos ? (p - P::kAhead) / 2
                            : (p < P::kAhead ? p : (p + P::kAhead - 1) / 2);
        if (v_pos ? t < cv.t : t < ck.t)
          drain_wait(&bar.full[p % P::kSlots], (p / P::kSlots) & 1u);
      }
      __syncwarp();
    } else if (warp == 14) {
      // -------------------------------------------------------- tails of V
      // Rows of V past a request's end may hold anything, and 0 * NaN is not 0:
      // they are cleared between the copy and the products.
      int tiles = 0;
      uint32_t phases = 0u;  // of each slot's `landed`
      for (int w = first_unit; w < a.units; w += stride) {
        const Unit u = unit_of<kDual>(a, w, rank);
        tiles += u.n;
        if (!u.ragged) continue;
        const int vs = pos_v(tiles - 1, P::kAhead) % P::kSlots;
        if (!warp_wait(&bar.landed[vs], phases >> vs & 1u, &bar.abort, a.status)) break;
        phases ^= 1u << vs;
        constexpr int kUnits = D / 8;
#pragma unroll 4
        for (int e = u.ragged * kUnits + lane; e < kKeys * kUnits; e += 32)
          *reinterpret_cast<uint4*>(ring + vs * P::kTile + unit_at(e / kUnits, e % kUnits)) =
              make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.full[vs]);
      }
    }
  } else if (warp < 8) {
    if constexpr (kDual)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 96;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    // ---------------------------------------------------------- softmax
    const int s = warp >> 2;
    const uint32_t t_s = tmem + s * kKeys + quad, t_o = tmem + 256 + s * 128 + quad;
    const float sc = a.scale_log2;
    int count = 0, done = 0;
    bool ok = true;
    for (int w = first_unit; ok && w < a.units; w += stride) {
      const Unit u = unit_of<kDual>(a, w, rank);
      const int steps = steps_of<kDual>(u, s);
      if (steps == 0) continue;
      const int tile_rows = kDual && s == 1 ? u.rows - kRows : min(u.rows, kRows);
      const bool active = quarter * 32 < tile_rows;
      // A row's weights are 2^(x - m) for a reference m that follows the row's
      // maximum. A tile is weighed in two halves, so that only a half's maximum
      // stands before its weights; m moves (with O and l) before the first half
      // once it is behind by 2^kNear, before the second only if it is behind by
      // 2^kFar (the first half's weights then move too), far below any overflow.
      constexpr float kNear = 8.f, kFar = 60.f;
      float m = kNegInf, l = 0.f, seen = kNegInf;  // seen: the maximum so far
      for (int j = 0; j < steps; ++j, ++count) {
        if (!warp_wait(&bar.s_full[s], count, &bar.abort, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (active) {
          const int last = u.ragged && tile_of<kDual>(s, j) == u.n - 1 ? u.ragged : kKeys;
#pragma unroll 1
          for (int h = 0; h < kKeys; h += 64) {
            float x[64];
            uint32_t* xr = reinterpret_cast<uint32_t*>(x);
            tmem_ld32_async(t_s + h, xr);
            tmem_ld32_async(t_s + h + 32, xr + 32);
            tmem_wait_ld32(xr);
            tmem_wait_ld32(xr + 32);
            if (h + 64 > last) {
#pragma unroll
              for (int e = 0; e < 64; ++e)
                if (h + e >= last) x[e] = kNegInf;
            }
            float t4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) t4[e] = fmaxf(x[e], x[e + 4]);
#pragma unroll
            for (int e = 8; e < 64; e += 8)
#pragma unroll
              for (int k = 0; k < 4; ++k) t4[k] = fmaxf(fmaxf(t4[k], x[e + k]), x[e + 4 + k]);
            seen = fmaxf(seen, fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * sc);
            if (j == 0 && h == 0) {
              m = seen;
            } else if (const bool moves = seen > m + (h == 0 ? kNear : kFar);
                       __any_sync(0xFFFFFFFFu, moves)) {
              // (A row that need not move keeps its reference, so that no row's
              // result depends on its neighbours.)
              const float f = moves ? ex2_approx(m - seen) : 1.f;
              l *= f;
              m = moves ? seen : m;
              if (j > 0) {
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  uint32_t o[16];
                  tmem_ld16(t_o + c, o);
#pragma unroll
                  for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tmem_st16(t_o + c, o);
                }
              }
              if (h > 0) {  // the first half's weights
                tmem_wait_st();
#pragma unroll 1
                for (int c = 0; c < 32; c += 16) {
                  uint32_t p[16];
                  tmem_ld16(t_s + c, p);
#pragma unroll
                  for (int e = 0; e < 16; ++e)
                    p[e] = bf16x2(__uint_as_float(p[e] << 16) * f,
                                  __uint_as_float(p[e] & 0xFFFF0000u) * f);
                  tmem_st16(t_s + c, p);
                }
              }
            }
            const float mref = m > kNegInf ? m : 0.f;
            const uint64_t sc2 = pack_f32x2(sc, sc), m2 = pack_f32x2(-mref, -mref);
            uint64_t l2[2] = {pack_f32x2(l, 0.f), pack_f32x2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
              uint32_t p[16];
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                float p0, p1;
                unpack_f32x2(fma_f32x2(pack_f32x2(x[c + e], x[c + e + 1]), sc2, m2), p0, p1);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                l2[(e >> 1) & 1] = add_f32x2(l2[(e >> 1) & 1], pack_f32x2(p0, p1));
                p[e >> 1] = bf16x2(p0, p1);
              }
              tmem_st16(t_s + ((h + c) >> 1), p);
            }
            float la, lb;
            unpack_f32x2(add_f32x2(l2[0], l2[1]), la, lb);
            l = la + lb;
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_ready[s]);
      }
      if (!ok) break;
      if (done > 0 && !warp_wait(&bar.o_empty[s], done - 1, &bar.abort, a.status)) break;
      ml[s * kRows + quarter * 32 + lane] = make_float2(m, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.ml_full[s]);
      ++done;
    }
  } else {
    if constexpr (kDual)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    else
      asm volatile("setmaxnreg.inc.sync.aligned.u32 136;");
    // ---------------------------------------------------------- rows
    // A warp group per row tile. A warp keeps to the 32 rows of its TMEM lanes
    // throughout, so its pieces of Q and the tables need no barrier beyond the warp.
    const int tile = kDual && warp >= 16 ? 1 : 0;
    const int first_s = tile, end_s = kDual ? tile + 1 : 2;  // the tile's streams
    const int my0 = quarter * 32;  // first of the warp's rows in a tile
    int done0 = 0, done1 = 0;      // units behind, of the tile's streams
    bool ok = true;
    // (2^32 / 1 does not fit the magic factor.)
    auto beam_of = [&](int i) {
      return a.G == 1 ? i : static_cast<int>(__umulhi(static_cast<uint32_t>(i), a.g_magic));
    };
    // The warp's valid rows of a tile.
    auto rows_in = [&](const Unit& u) {
      return min(32, u.rows - tile * kRows - my0);
    };
    // Elements from the row of the unit's first beam to this lane's row of a tile
    // (strides are below 2^24, a unit has at most 256 beams).
    auto row_off = [&](const Unit& u, int64_t row_stride) {
      const int i = u.row0 + tile * kRows + my0 + lane, b = beam_of(i);
      return static_cast<uint32_t>(b - beam_of(u.row0)) * static_cast<uint32_t>(row_stride) +
             static_cast<uint32_t>((i - b * a.G) * D);
    };
    auto row_base = [&](const Unit& u, int64_t row_stride) {
      return (static_cast<int64_t>(u.r) * a.B + beam_of(u.row0)) * row_stride + u.g * a.G * D;
    };
    // 16-byte word of [level][R * B][Hkv][D] where slot 0 of the unit's request and
    // key head begins at level 0, and words from a slot to the next.
    auto beam_base = [&](const Unit& u) {
      return static_cast<uint32_t>((static_cast<int64_t>(u.r) * a.B * a.Hkv + u.g) * (D / 8));
    };
    const uint32_t slot16 = static_cast<uint32_t>(a.Hkv * (D / 8));

    // Q of unit u into the tile, behind the last product with the one before.
    // (`more`: the unit before, not yet counted, used it.)
    auto load_q = [&](const Unit& u, int more) {
      constexpr int kUnits = D / 8, kPer = 32 / kUnits;
      const int c = lane % kUnits;
      const int users = done0 + more;
      if (users > 0 && !warp_wait(&bar.q_empty[tile], users - 1, &bar.abort, a.status)) ok = false;
      if (!ok) return;
      uint8_t* qt = smem + tile * P::kTile;
      const int valid = rows_in(u);
      const uint32_t off = row_off(u, a.q_stride);
      const __nv_bfloat16* src = a.q + row_base(u, a.q_stride) + c * 8;
#pragma unroll 2
      for (int lr = lane / kUnits; lr < 32; lr += kPer) {
        const uint32_t at = __shfl_sync(0xFFFFFFFFu, off, lr);
        if (lr < valid) cp_async16(qt + unit_at(my0 + lr, c), src + at);
      }
      cp_async_wait();
      __syncwarp();
      if (a.q_flip) {
#pragma unroll 1
        for (int e = lane; e < 32 * kUnits; e += 32) {
          uint4* q = reinterpret_cast<uint4*>(qt + unit_at(my0 + e / kUnits, e % kUnits));
          *q = make_uint4(q->x ^ a.q_flip, q->y ^ a.q_flip, q->z ^ a.q_flip, q->w ^ a.q_flip);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (steps_of<kDual>(u, tile) > 0 && lane == 0) mbar_arrive(&bar.q_full[tile]);
    };

    // The slots of the rows' ancestors at every level. Returns whether this lane's
    // row is dead.
    auto walk_path = [&](const Unit& u) {
      uint16_t* tab = slots + (tile * kRows + my0) * P::kLevels;
      int at = lane < rows_in(u) ? beam_of(u.row0 + tile * kRows + my0 + lane) : -1;
#pragma unroll 1
      for (int v = a.level - 1; v >= 0; --v) {
        tab[lane * P::kLevels + v] = static_cast<uint16_t>(at);
        const int p = at < 0 ? -1 : a.bp[(static_cast<int64_t>(v) * a.R + u.r) * a.B + at];
        at = p < 0 || (v > 0 && p >= a.B) ? -1 : p;
      }
      __syncwarp();
      // Dead rows (and those past the last) take a live row's slots, so that what
      // is loaded for them is a live beam's; their weights are zero.
      const uint32_t live = __ballot_sync(0xFFFFFFFFu, at >= 0);
      if (at < 0) {
#pragma unroll 1
        for (int v = 0; v < a.level; ++v)
          tab[lane * P::kLevels + v] = live ? tab[(__ffs(live) - 1) * P::kLevels + v] : 0;
      }
      __syncwarp();
      return at < 0;
    };

    // The rows' own softmax over their ancestors, for the warp's rows of a tile,
    // on the small tensor-core product: 16 rows by the (at most 16) beams that
    // they belong to, of whose block only a row's own beam counts. The orders of D
    // inside the products are free as long as both sides share them, so that each
    // lane reads whole 16-byte words. (One row per lane instead measured 4 times
    // the time: a lane's loads then touch 32 lines at once.) The weighted values,
    // summed in fp32 against the path's maximum, wait in the rows' places of the output,
    // rounded to bf16 once: two row tiles of D = 128 would take 128 KB in fp32, and 20 KB
    // of shared memory are left. Maximum and sum stay, in fp32, in the row's first two
    // table entries. (Error against 64 bits with 4 levels and with none: 0.0023.)
    auto attend_path = [&](const Unit& u, bool dead) {
      const int valid = rows_in(u);
      if (valid <= 0) return;
      const uint16_t* tab = slots + (tile * kRows + my0) * P::kLevels;
      float* xs = scores + (tile * kRows + my0) * P::kLevels;
      const int i0 = u.row0 + tile * kRows + my0;
      const int c = lane & 3, n8 = lane >> 2;
      const uint8_t* qt = smem + tile * P::kTile;
      const uint4* kb16 = reinterpret_cast<const uint4*>(a.kb);
      const uint4* vb16 = reinterpret_cast<const uint4*>(a.vb);
      const uint32_t base16 = beam_base(u);
      // ---- scores: rounds of 16 rows x 8 beams x a level, a round's loads in
      // flight under the round before
      {
        constexpr int kWords = D / 32;  // 16-byte words of a lane's quarter of D
        uint4 kw[kWords];
        // This lane's key: beam b0 + n0 + n8 (or the last one, again), through its
        // first row in the group.
        auto load = [&](int rg, int n0, int v0) {
          const int b0 = beam_of(i0 + rg), b_end = beam_of(i0 + min(rg + 15, valid - 1));
          const uint16_t* of =
              tab + max(rg, min(b0 + n0 + n8, b_end) * a.G - i0) * P::kLevels;
          const uint4* src =
              kb16 + (base16 + v0 * a.level16 + of[v0] * slot16 + c * static_cast<uint32_t>(kWords));
#pragma unroll
          for (int k = 0; k < kWords; ++k) kw[k] = src[k];
        };
        load(0, 0, 0);
        int rg = 0, n0 = 0, v0 = 0;
#pragma unroll 1
        while (rg < valid) {
          const int b0 = beam_of(i0 + rg), b_end = beam_of(i0 + min(rg + 15, valid - 1));
          const int lo = beam_of(i0 + rg + n8) - b0 - n0, hi = beam_of(i0 + rg + n8 + 8) - b0 - n0;
          float z[2][4] = {};  // two chains, added below
#pragma unroll
          for (int k = 0; k < kWords; ++k) {
            const uint4 qa =
                *reinterpret_cast<const uint4*>(qt + unit_at(my0 + rg + n8, c * kWords + k));
            const uint4 qb =
                *reinterpret_cast<const uint4*>(qt + unit_at(my0 + rg + n8 + 8, c * kWords + k));
            mma_16816(z[0], qa.x, qb.x, qa.y, qb.y, kw[k].x, kw[k].y);
            mma_16816(z[1], qa.z, qb.z, qa.w, qb.w, kw[k].z, kw[k].w);
          }
          const int rg_now = rg, v_now = v0;
          if (++v0 == a.level) {
            v0 = 0;
            n0 += 8;
            if (n0 > b_end - b0) {
              n0 = 0;
              rg += 16;
            }
          }
          if (rg < valid) load(rg, n0, v0);
          if ((lo >> 1) == c)
            xs[(rg_now + n8) * P::kLevels + v_now] =
                (lo & 1 ? z[0][1] + z[1][1] : z[0][0] + z[1][0]) * a.scale_log2;
          if ((hi >> 1) == c)
            xs[(rg_now + n8 + 8) * P::kLevels + v_now] =
                (hi & 1 ? z[0][3] + z[1][3] : z[0][2] + z[1][2]) * a.scale_log2;
        }
      }
      __syncwarp();
      // ---- softmax, a row per lane
      float mp = kNegInf, lp = 0.f;
      {
        float* x = xs + lane * P::kLevels;
        if (!dead)
          for (int v = 0; v < a.level; ++v) mp = fmaxf(mp, x[v]);
#pragma unroll 1
        for (int v = 0; v < a.level; ++v) {
          x[v] = dead ? 0.f : ex2_approx(x[v] - mp);
          lp += x[v];
        }
        // (A NaN goes on in lp; as a weight it would make its neighbours' part a
        // slow one below.)
        if (!(lp >= 0.f))
#pragma unroll 1
          for (int v = 0; v < a.level; ++v) x[v] = 0.f;
      }
      __syncwarp();
      // ---- values: parts of 16 rows by 32 columns, in rounds of 8 beams x 2 levels,
      // a round's loads in flight under the round before
      const uint32_t off = row_off(u, a.out_stride);
      __nv_bfloat16* out = a.out + row_base(u, a.out_stride);
      uint2 vw[4];
      // Keys of this lane: beams b0 + n0 + 2c, + 1 (or the last one, again) at two
      // levels; columns d0 + 4 n8 .. + 3 of each.
      auto load = [&](int rg, int d0, int n0, int v0) {
        const int b0 = beam_of(i0 + rg), b_end = beam_of(i0 + min(rg + 15, valid - 1));
        const int kb = b0 + n0 + 2 * c;
        const uint16_t* of0 = tab + max(rg, min(kb, b_end) * a.G - i0) * P::kLevels;
        const uint16_t* of1 = tab + max(rg, min(kb + 1, b_end) * a.G - i0) * P::kLevels;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int v = min(v0 + (e >> 1), a.level - 1);
          vw[e] = reinterpret_cast<const uint2*>(
              vb16 + (base16 + v * a.level16 + (e & 1 ? of1 : of0)[v] * slot16))[d0 / 4 + n8];
        }
      };
      load(0, 0, 0, 0);
      float y[4][4];
      int rg = 0, d0 = 0, n0 = 0, v0 = 0;
#pragma unroll 1
      while (rg < valid) {
        const int b0 = beam_of(i0 + rg), b_end = beam_of(i0 + min(rg + 15, valid - 1));
        const int lo = beam_of(i0 + rg + n8) - b0 - n0, hi = beam_of(i0 + rg + n8 + 8) - b0 - n0;
        if (n0 == 0 && v0 == 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[k][e] = 0.f;
        }
        // Weights: a row's in the place of its own beam, as the sum of two bf16
        // (its values are rounded once on their way through the output, which
        // takes what rounding the weights is allowed).
        uint32_t aw[4], ar[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int at = e & 1 ? hi : lo, v = v0 + (e >> 1);
          const float wt = (at >> 1) == c && v < a.level
                               ? xs[(rg + n8 + (e & 1) * 8) * P::kLevels + v]
                               : 0.f;
          const float head = __uint_as_float(__float_as_uint(wt) & 0xFFFF0000u);
          aw[e] = at & 1 ? bf16x2(0.f, head) : bf16x2(head, 0.f);
          ar[e] = at & 1 ? bf16x2(0.f, wt - head) : bf16x2(wt - head, 0.f);
        }
        const uint32_t w[4][2] = {
            {vw[0].x, vw[0].y}, {vw[1].x, vw[1].y}, {vw[2].x, vw[2].y}, {vw[3].x, vw[3].y}};
        const int rg_now = rg, d_now = d0;
        v0 += 2;
        bool part_done = false;
        if (v0 >= a.level) {
          v0 = 0;
          n0 += 8;
          if (n0 > b_end - b0) {
            n0 = 0;
            part_done = true;
            d0 += 32;
            if (d0 == D) {
              d0 = 0;
              rg += 16;
            }
          }
        }
        if (rg < valid) load(rg, d0, n0, v0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t e0 = __byte_perm(w[0][k], w[1][k], 0x5410);
          const uint32_t e1 = __byte_perm(w[2][k], w[3][k], 0x5410);
          const uint32_t o0 = __byte_perm(w[0][k], w[1][k], 0x7632);
          const uint32_t o1 = __byte_perm(w[2][k], w[3][k], 0x7632);
          mma_16816(y[2 * k], aw[0], aw[1], aw[2], aw[3], e0, e1);
          mma_16816(y[2 * k + 1], aw[0], aw[1], aw[2], aw[3], o0, o1);
          mma_16816(y[2 * k], ar[0], ar[1], ar[2], ar[3], e0, e1);
          mma_16816(y[2 * k + 1], ar[0], ar[1], ar[2], ar[3], o0, o1);
        }
        if (!part_done) continue;
        // An infinity or NaN in one beam's values would reach its neighbours
        // through their zero weights: such a part is added up row by row.
        float all = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) all += (y[k][0] + y[k][1]) + (y[k][2] + y[k][3]);
        if (__any_sync(0xFFFFFFFFu, !(fabsf(all) < 3.0e38f))) {
#pragma unroll 1
          for (int lr = rg_now; lr < min(rg_now + 16, valid); ++lr) {
            const uint32_t at = __shfl_sync(0xFFFFFFFFu, off, lr);
#pragma unroll 1
            for (int d = d_now + lane; d < d_now + 32; d += 32) {
              float z = 0.f;
#pragma unroll 1
              for (int v = 0; v < a.level; ++v) {
                const int64_t at16 = base16 + v * a.level16 + tab[lr * P::kLevels + v] * slot16;
                const float wt = xs[lr * P::kLevels + v];
                if (wt > 0.f) z = fmaf(wt, __bfloat162float(a.vb[at16 * 8 + d]), z);
              }
              out[at + d] = __float2bfloat16(z);
            }
          }
        } else {
          // This lane: columns 8 c .. + 7 of the part's rows n8 and n8 + 8.
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int lr = rg_now + n8 + half * 8, e = half * 2;
            const uint32_t at = __shfl_sync(0xFFFFFFFFu, off, lr);
            if (lr < valid)
              *reinterpret_cast<uint4*>(out + at + d_now + c * 8) =
                  make_uint4(bf16x2(y[0][e], y[1][e]), bf16x2(y[2][e], y[3][e]),
                             bf16x2(y[0][e + 1], y[1][e + 1]), bf16x2(y[2][e + 1], y[3][e + 1]));
          }
        }
      }
      __syncwarp();
      xs[lane * P::kLevels] = mp;
      xs[lane * P::kLevels + 1] = lp;
    };

    // Joins the streams and the path of the warp's rows of a tile, a row per lane,
    // and writes them: bf16 rows, or (split keys) partial rows in fp32.
    auto finish = [&](const Unit& u, bool dead) {
      const int valid = rows_in(u);
      const bool path = kPath && rank == 0;
      const uint32_t off = row_off(u, a.out_stride);
      __nv_bfloat16* out = a.out + row_base(u, a.out_stride);
      float mp = kNegInf, lp = 0.f;
      if (path && lane < valid) {
        const float* x = scores + (tile * kRows + my0 + lane) * P::kLevels;
        mp = x[0];
        lp = x[1];
        for (int c = 0; c < D; c += 64)
          asm volatile("prefetch.global.L1 [%0];" ::"l"(out + off + c));
      }
      float2 st_a = make_float2(kNegInf, 0.f), st_b = st_a;
#pragma unroll 1
      for (int s = first_s; s < end_s; ++s) {
        if (steps_of<kDual>(u, s) == 0) continue;
        const int done = !kDual && s ? done1 : done0;
        if (!warp_wait(&bar.ml_full[s], done, &bar.abort, a.status) ||
            !warp_wait(&bar.o_full[s], done, &bar.abort, a.status)) {
          ok = false;
          return;
        }
        const float2 got = ml[s * kRows + my0 + lane];
        if (kDual || s == 0) st_a = got; else st_b = got;
      }
      tc_fence_after();
      // One reference for all sources of the row that have keys (l is 0 without,
      // and NaN where the row's scores are: that reaches the output, except for
      // the q of a dead row).
      const bool has_a = !(st_a.y <= 0.f) && !dead, has_b = !(st_b.y <= 0.f) && !dead;
      const bool has_p = !(lp <= 0.f) && !dead;
      const float top = fmaxf(fmaxf(has_a ? st_a.x : kNegInf, has_b ? st_b.x : kNegInf),
                              has_p ? mp : kNegInf);
      const float ref = top > kNegInf ? top : 0.f;
      float f0 = has_a ? ex2_approx(st_a.x - ref) : 0.f;
      float f1 = has_b ? ex2_approx(st_b.x - ref) : 0.f;
      float fp = has_p ? ex2_approx(mp - ref) : 0.f;
      const float sum = f0 * st_a.y + f1 * st_b.y + fp * lp;
      const float total = has_a || has_b || has_p ? sum : 0.f;
      if constexpr (!kSplit) {
        const float inv = total == 0.f ? 0.f : 1.f / total;
        f0 *= inv;
        f1 *= inv;
        fp *= inv;
      }
      float* part = reinterpret_cast<float*>(smem) + (tile * kRows + my0 + lane) * P::kPart;
      if (kSplit && valid > 0) {
        part[D] = top;
        part[D + 1] = total;
      }
      const int sa = kDual ? tile : 0;
      const bool read_a = valid > 0 && steps_of<kDual>(u, sa) > 0;
      const bool read_b = !kDual && valid > 0 && steps_of<kDual>(u, 1) > 0;
      const bool with_path = kPath && has_p && lane < valid;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint4 pw[4];
        if (with_path) {
#pragma unroll
          for (int e = 0; e < 4; ++e) pw[e] = *reinterpret_cast<const uint4*>(out + off + c + e * 8);
        }
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0.f;
        if (read_a) {
          uint32_t v[32];
          tmem_ld32(tmem + 256 + sa * 128 + quad + c, v);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = has_a ? __uint_as_float(v[e]) * f0 : 0.f;
        }
        if (read_b) {
          uint32_t v[32];
          tmem_ld32(tmem + 256 + 128 + quad + c, v);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (has_b) o[e] = fmaf(__uint_as_float(v[e]), f1, o[e]);
        }
        if (c + 32 == D) {  // O has been read
          tc_fence_before();
          __syncwarp();
#pragma unroll 1
          for (int s = first_s; s < end_s; ++s)
            if (steps_of<kDual>(u, s) > 0) {
              if (lane == 0) mbar_arrive(&bar.o_empty[s]);
              if (!kDual && s) ++done1; else ++done0;
            }
        }
        if (with_path) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            const uint4 w = pw[e / 8];
            float f[4];
            bf16x4(make_uint2(w.x, w.y), f);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[e + k] = fmaf(fp, f[k], o[e + k]);
            bf16x4(make_uint2(w.z, w.w), f);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[e + 4 + k] = fmaf(fp, f[k], o[e + 4 + k]);
          }
        }
        if constexpr (kSplit) {
          if (valid > 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(part + c + e) =
                  make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        } else {
        if (lane < valid) {
#pragma unroll
          for (int e = 0; e < 32; e += 8)
            *reinterpret_cast<uint4*>(out + off + c + e) =
                make_uint4(bf16x2(o[e], o[e + 1]), bf16x2(o[e + 2], o[e + 3]),
                           bf16x2(o[e + 4], o[e + 5]), bf16x2(o[e + 6], o[e + 7]));
        }
        }
      }
    };

    Unit u;
    if (first_unit < a.units) {
      u = unit_of<kDual>(a, first_unit, rank);
      load_q(u, 0);
    }
    for (int w = first_unit; ok && w < a.units; w += stride) {
      const bool have_next = w + stride < a.units;
      if (have_next) {
        // The next unit's q on its way to L2.
        const Unit nx = unit_of<kDual>(a, w + stride, rank);
        if (lane < rows_in(nx))
          for (int c = 0; c < D; c += 64)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(a.q + row_base(nx, a.q_stride) +
                                                          row_off(nx, a.q_stride) + c));
      }
      bool dead = false;
      if constexpr (kPath) {
        dead = walk_path(u);
        if (rank == 0) attend_path(u, dead);
      }
      // The next unit's Q comes in once this one's last products are done.
      Unit nx = u;
      if (have_next) {
        nx = unit_of<kDual>(a, w + stride, rank);
        load_q(nx, steps_of<kDual>(u, tile) > 0);
      }
      if constexpr (kSplit) {
        // Partial rows go where Q and the ring are: both streams end first, and
        // every warp has read Q. (One unit only: all of these warps come here.)
        for (int s = 0; s < 2; ++s)
          if (steps_of<kDual>(u, s) > 0 && !warp_wait(&bar.o_full[s], 0, &bar.abort, a.status))
            ok = false;
        named_sync(1, kDual ? 256 : 128);
      }
      if (ok) finish(u, dead);
      u = nx;
    }
  }
  __syncwarp();
  if constexpr (kSplit) {
    // ---------------------------------------------------------- joined output
    cluster_sync();
    const Unit u = unit_of<kDual>(a, first_unit, rank);
    const float* part = reinterpret_cast<const float*>(smem);
    constexpr int kWarps = P::kThreads / 32;
    for (int i = rank * kWarps + warp; i < u.rows; i += kWarps * a.split) {
      const float* mine = part + i * P::kPart;
      float mp = kNegInf, lp = 0.f;
      if (lane < a.split) {
        const uint32_t at = peer_addr(mine, lane);
        mp = ld_peer(at + D * 4);
        lp = ld_peer(at + D * 4 + 4);
      }
      const float top = warp_max(mp);
      const float wt = mp > kNegInf ? ex2_approx(mp - top) : 0.f;
      const float sum = warp_sum(wt * lp);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int p = 0; p < a.split; ++p) {
        const float wp = __shfl_sync(0xFFFFFFFFu, wt, p);
        if (wp > 0.f && lane < D / 4) {
          const float4 v = ld_peer4(peer_addr(mine, p) + lane * 16);
          o.x = fmaf(wp, v.x, o.x);
          o.y = fmaf(wp, v.y, o.y);
          o.z = fmaf(wp, v.z, o.z);
          o.w = fmaf(wp, v.w, o.w);
        }
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const int ii = u.row0 + i, b = ii / a.G, h = u.g * a.G + (ii - b * a.G);
      if (lane < D / 4)
        *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(u.r) * a.B + b) * a.out_stride +
                                  h * D + lane * 4) =
            make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while its rows are read
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_free(tmem, 512);
}

// 4-D map of a cache [n_pages][page_size][Hkv][D], box [1][box][1][64].
bool make_map(CUtensorMap* map, const void* base, const AttnArgs& a, int D, int box) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(a.Hkv),
                              static_cast<cuuint64_t>(a.page_size),
                              static_cast<cuuint64_t>(a.n_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(D) * 2,
                                 static_cast<cuuint64_t>(a.token_stride) * 2,
                                 static_cast<cuuint64_t>(a.page_stride) * 2};
  const cuuint32_t boxes[4] = {64, 1, static_cast<cuuint32_t>(box), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
            boxes, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kDual, bool kPath, bool kSplit>
int launch_kernel(const AttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, int sms,
                  cudaStream_t stream) {
  using P = Plan<D, kDual>;
  constexpr auto kernel = attention_kernel<D, kDual, kPath, kSplit>;
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_error(e, "beam_attention: cudaGetDevice");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P::kSmem);
      if (e != cudaSuccess) return cuda_error(e, "beam_attention: cudaFuncSetAttribute");
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  // As few CTAs as end in the same number of rounds: the SMs left over would only
  // compete for the cache's bytes early on. Against a CTA per SM, at full clock and in
  // seconds of calls under the power cap: 32 rows of 2500-5000 tokens (256 units, 128 CTAs)
  // 87 us and 94, against 98 and 102; all of 5000 107 and 121, against 109 and 122; 64 x 128
  // beams over 1000-2000 tokens (512 units) 153 and 179, against 161 and 183; all of 2000
  // 179 and 215 both ways.
  const int rounds = (a.units + sms - 1) / sms;
  const unsigned grid =
      static_cast<unsigned>(kSplit ? a.units * a.split : (a.units + rounds - 1) / rounds);
  e = launch_dependent(kernel, dim3(grid), P::kThreads, P::kSmem, kSplit ? a.split : 1, stream, mk,
                       mv, a);
  return e == cudaSuccess ? SIDBEAM_OK : cuda_error(e, "beam_attention: launch");
}

template <int D, bool kDual>
int launch_attention(AttnArgs& a, cudaStream_t stream) {
  using P = Plan<D, kDual>;
  CUtensorMap mk, mv;
  const int box = a.table ? std::min(a.page_size, kKeys) : kKeys;
  if (!make_map(&mk, a.k, a, D, box) || !make_map(&mv, a.v, a, D, box))
    return set_error(SIDBEAM_ERR_CUDA, "beam_attention: tensor map encoding failed");
  const int sms = device_sm_count();
  const int unit_rows = P::kTiles * kRows;
  a.pairs = (a.B * a.G + unit_rows - 1) / unit_rows;
  const int64_t units = static_cast<int64_t>(a.pairs) * a.Hkv * a.R;
  if (units > 0x7FFFFFFFll - sms)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: too many rows and heads");
  a.units = static_cast<int>(units);
  const int64_t cap = a.table ? static_cast<int64_t>(a.table_stride) * a.page_size : a.page_size;
  const int64_t max_tiles = (cap + kKeys - 1) / kKeys;
  // CTAs per unit: doubled while all clusters run at once and at most one CTA of a unit
  // has no key tile (3 tiles on 4 CTAs, 7 on 8), by the capacity: the lengths are not
  // known here. One row, 16 / 8 heads of 128, us at full clock on 1, 2, 4, 8 CTAs a unit
  // (measured together; those chosen take 0.2 us less by now):
  //   384 tokens    9.4   9.5   8.5   8.9        1024   15.2  12.9   9.7   9.1
  //   512          10.2   9.6   8.6   9.1        2048   25.4  18.3  13.1  10.3
  // (256 tokens: 7.3, split 8.4.) Two rows of 2048: 25.4, 18.3, 13.4, and 19.8 on 8,
  // since 16 clusters of 8 do not run at once.
  a.split_log2 = 0;
  while (a.split_log2 < kMaxSplitLog2 && max_tiles > 2 && (2 << a.split_log2) <= max_tiles + 1 &&
         units << (a.split_log2 + 1) <= sms) {
    static std::mutex mu;
    static int cache[64][4] = {};
    int room = 0;
    const cudaError_t e = clusters_at_once(attention_kernel<D, kDual, true, true>, P::kThreads,
                                           P::kSmem, a.split_log2 + 1, mu, cache, &room);
    if (e != cudaSuccess) return cuda_error(e, "beam_attention: cudaOccupancyMaxActiveClusters");
    if (units > room) break;
    ++a.split_log2;
  }
  a.split = 1 << a.split_log2;
  if (a.level > 0)
    return a.split > 1 ? launch_kernel<D, kDual, true, true>(a, mk, mv, sms, stream)
                       : launch_kernel<D, kDual, true, false>(a, mk, mv, sms, stream);
  return a.split > 1 ? launch_kernel<D, kDual, false, true>(a, mk, mv, sms, stream)
                     : launch_kernel<D, kDual, false, false>(a, mk, mv, sms, stream);
}

bool misaligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

}  // namespace
}  // namespace sidbeam

using namespace sidbeam;

extern "C" int beam_attention(const sidbeam_attention* args, void* stream) {
  if (!args) return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: NULL arguments");
  const auto [q, q_row_stride, k_cache, v_cache, page_stride, token_stride, n_pages, page_size,
              page_table, cache_len, bp_parent, k_beam, v_beam, pages_per_request, level, R, B, H,
              Hkv, D, scale, out, out_row_stride, workspace, workspace_bytes] = *args;
  if (!q || !k_cache || !v_cache || !cache_len || !out)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: NULL pointer argument");
  if (R < 1 || B < 1 || B > SIDBEAM_MAX_BEAM || static_cast<int64_t>(R) * B > 0x7FFFFFFFll)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: R=%d, B=%d (at most %d)", R, B,
                     SIDBEAM_MAX_BEAM);
  if (D != 64 && D != 128)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: head size D=%d must be 64 or 128", D);
  if (H < 1 || Hkv < 1 || H % Hkv != 0 || H / Hkv > 128 || Hkv > 65535 || H > 65536)
    return set_error(SIDBEAM_ERR_INVALID_ARG,
                     "beam_attention: H=%d must be a multiple of Hkv=%d, at most 128 times it", H,
                     Hkv);
  if (level < 0 || level > SIDBEAM_MAX_DEPTH)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: level=%d outside [0, %d]", level,
                     SIDBEAM_MAX_DEPTH);
  if (level > 0 && (!bp_parent || !k_beam || !v_beam))
    return set_error(SIDBEAM_ERR_INVALID_ARG,
                     "beam_attention: bp_parent, k_beam or v_beam is NULL at level %d", level);
  if (!(scale > -3.0e38f && scale < 3.0e38f))
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: scale must be finite");
  if (n_pages < 1 || page_size < 1)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: n_pages=%d page_size=%d", n_pages,
                     page_size);
  if (page_table) {
    if (page_size < 16 || page_size > 65536 || (page_size & (page_size - 1)) != 0)
      return set_error(SIDBEAM_ERR_INVALID_ARG,
                       "beam_attention: page_size=%d must be a power of two in [16, 65536]",
                       page_size);
    if (pages_per_request < 1 ||
        static_cast<int64_t>(pages_per_request) * page_size > 0x7FFFFFFFll - 256)
      return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: pages_per_request=%d",
                       pages_per_request);
  } else if (n_pages != R || page_size > 0x7FFFFFFF - 256) {
    return set_error(SIDBEAM_ERR_INVALID_ARG,
                     "beam_attention: without a page table n_pages=%d must be R=%d", n_pages, R);
  }
  const int64_t row = static_cast<int64_t>(H) * D;
  if (q_row_stride < row || out_row_stride < row ||
      token_stride < static_cast<int64_t>(Hkv) * D || page_stride < token_stride)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: a stride is smaller than its row");
  if (q_row_stride >= 1 << 24 || out_row_stride >= 1 << 24)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: a row stride is 2^24 or more");
  if (static_cast<int64_t>(R) * B * Hkv * (D / 8) * std::max(level, 1) > 0xFFFFFFFFll)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: k_beam of 64 GiB or more");
  if (page_stride > (1ll << 38))
    return set_error(SIDBEAM_ERR_INVALID_ARG, "beam_attention: page_stride too large");
  if (misaligned(q, 16) || misaligned(k_cache, 16) || misaligned(v_cache, 16) ||
      misaligned(out, 16) || ((q_row_stride | out_row_stride | token_stride | page_stride) & 7) ||
      (level > 0 && (misaligned(k_beam, 16) || misaligned(v_beam, 16))))
    return set_error(SIDBEAM_ERR_ALIGNMENT,
                     "beam_attention: pointers must be 16-byte aligned, strides multiples of 8");
  if (!workspace || workspace_bytes < 256 || misaligned(workspace, 256))
    return set_error(SIDBEAM_ERR_WORKSPACE,
                     "beam_attention: workspace of >= 256 bytes, 256-byte aligned");
  AttnArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_row_stride;
  a.k = static_cast<const __nv_bfloat16*>(k_cache);
  a.v = static_cast<const __nv_bfloat16*>(v_cache);
  a.page_stride = page_stride;
  a.token_stride = token_stride;
  a.n_pages = n_pages;
  a.page_size = page_size;
  a.table = page_table;
  a.table_stride = pages_per_request;
  a.len = cache_len;
  a.level = level;
  a.bp = bp_parent;
  a.kb = static_cast<const __nv_bfloat16*>(k_beam);
  a.vb = static_cast<const __nv_bfloat16*>(v_beam);
  a.R = R;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  // A zero scale keeps a factor (it leaves every finite score 0 to within 2^-60):
  // masked scores are -inf, and -inf * 0 is not.
  a.scale_log2 = std::max(fabsf(scale) * kLog2e, 1e-30f);
  a.q_flip = scale < 0.f ? 0x80008000u : 0u;
  a.G = H / Hkv;
  a.level16 = static_cast<uint32_t>(static_cast<int64_t>(R) * B * Hkv * (D / 8));
  a.page_log2 = 0;
  while (page_table && (1 << a.page_log2) < page_size) ++a.page_log2;
  a.g_magic = a.G > 1 ? static_cast<uint32_t>((0x100000000ull + a.G - 1) / a.G) : 0u;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.out_stride = out_row_stride;
  a.status = static_cast<uint32_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Two row tiles a unit where there are two: each key tile is read, and each page
  // of it asked for, once for 256 rows, and two warp groups see to the ancestors. For
  // 16 x 512 beams at full clock, 1024 tokens (one tile a unit in brackets): 82 us (81),
  // at 4 levels 137 (206), from pages of 16 88 (135); over 128 tokens 26 (31), over 8192
  // 543 (519).
  // More than 8 levels need the table space that one tile leaves.
  const bool dual = static_cast<int64_t>(B) * a.G > kRows && level <= 8;
  if (D == 64)
    return dual ? launch_attention<64, true>(a, s) : launch_attention<64, false>(a, s);
  return dual ? launch_attention<128, true>(a, s) : launch_attention<128, false>(a, s);
}
