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
  float scale_log2;
  __nv_bfloat16* out;
  int64_t out_stride;
  uint32_t* status;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -INFINITY;

// ------------------------------------------------------------ shape of the work
// A work item is (request, key/value head, two tiles of 128 rows): the rows of
// the beams and of the H / Hkv heads that share the keys are one M axis, row
// i = b * (H / Hkv) + head. Keys come in tiles of 128.
//
// One CTA runs two streams, each a chain S = Q K^T, softmax, O += P V with its
// own S, P (in S's place) and O in TMEM, so that one stream's softmax runs under
// the other's MMAs. With two row tiles the streams take one each and share every
// key tile (loaded once). With one row tile both streams work on it, on every
// other key tile, and their sums are joined at the end. Few items are split once
// more along the keys over the CTAs of a cluster and joined through distributed
// shared memory, always in the same order.
constexpr int kRows = 128;
constexpr int kKeys = 128;
constexpr int kThreads = 320;  // two softmax groups of 4 warps, TMA warp, MMA warp
constexpr int kMaxSplit = 8;

template <int D>
struct Plan {
  static constexpr int kHalves = D / 64;             // 128-byte columns of a row
  static constexpr int kTile = kKeys * D * 2;        // bytes of a K, V or Q tile
  static constexpr int kHalf = kKeys * 128;          // bytes of one 64-column half
  static constexpr int kSlots = D == 128 ? 5 : 8;    // ring of K and V tiles
  static constexpr int kSmem = 2 * kTile + kSlots * kTile + 1024;
  static constexpr int kPitch = D + 4;               // floats of a partial row: o, m, l
  static_assert(2 * kRows * kPitch * 4 <= kSlots * kTile, "partials fit the ring");
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

// The whole warp waits; one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* abort,
                                          uint32_t* status) {
  const bool ok = bounded_wait(bar, parity, abort, status, kStatusTimeout);
  return __all_sync(0xFFFFFFFFu, ok);
}

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t q_ready[2], s_full[2], p_ready[2], o_full[2];
  uint64_t v_clean, drain;
  uint32_t tmem;
  int abort;
};

// Position in the load order of key tile i's K and V (n tiles, K tiles loaded
// `ahead` of the V tiles): K_0 .. K_{ahead-1}, then V_i, K_{i+ahead} in turn.
__device__ __forceinline__ int pos_k(int i, int ahead) { return i + max(0, i - ahead + 1); }
__device__ __forceinline__ int pos_v(int i, int ahead, int n) { return i + min(n, i + ahead); }

// Element range 8 bf16 of a 16-byte unit.
__device__ __forceinline__ void bf16x8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// Byte offset of 16-byte unit c (0 .. D/8 - 1) of row `row` in a swizzled tile.
template <int D>
__device__ __forceinline__ uint32_t unit_at(int row, int c) {
  return static_cast<uint32_t>((c >> 3) * Plan<D>::kHalf + row * 128 + (((c ^ row) & 7) << 4));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v, const AttnArgs a, int pairs,
                     int split) {
  using P = Plan<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem + 2 * P::kTile;
  __shared__ Bars bar;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int r = static_cast<int>(blockIdx.x) / (pairs * split), g = blockIdx.y;
  const int G = a.H / a.Hkv;
  const int row0 = (static_cast<int>(blockIdx.x) / split - r * pairs) * 2 * kRows;
  const int rows = min(2 * kRows, a.B * G - row0);  // valid rows of both tiles
  const bool dual = rows > kRows;

  int64_t cap = a.table ? static_cast<int64_t>(a.table_stride) * a.page_size : a.page_size;
  const int len_in = a.len[r];
  const int len = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(len_in), cap)));
  const int tiles = (len + kKeys - 1) / kKeys;
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * rank / split);
  const int n = static_cast<int>(static_cast<int64_t>(tiles) * (rank + 1) / split) - t0;
  const int ahead = dual ? 1 : 2;
  // Keys of the request's last tile if it is ragged and this CTA's, else 0.
  const int ragged = (t0 + n == tiles) && n > 0 ? len & (kKeys - 1) : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      mbar_init(&bar.full[s], 1);
      mbar_init(&bar.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      const int tile_rows = dual && s ? rows - kRows : min(rows, kRows);
      const int active = (tile_rows + 31) / 32;
      mbar_init(&bar.q_ready[s], active);
      mbar_init(&bar.s_full[s], 1);
      mbar_init(&bar.p_ready[s], active);
      mbar_init(&bar.o_full[s], 1);
    }
    mbar_init(&bar.v_clean, 1);
    mbar_init(&bar.drain, 1);
    bar.abort = 0;
    if (len != len_in) atomicOr(a.status, kStatusBadCache);
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(&bar.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;

  if (warp == 8) {
    // ---------------------------------------------------------- loads
    const int box = a.table ? min(a.page_size, kKeys) : kKeys;  // tokens of one copy
    const int boxes = kKeys / box;
    const int my_box = lane & (boxes - 1), my_half = lane / boxes;
    const bool mine = my_half < P::kHalves;
    if (lane == 0) {
      prefetch_map(&map_k);
      prefetch_map(&map_v);
    }
    const int loads = 2 * n;
    int page_of = -1, page = 0;  // this lane's page number in tile `page_of`
    int pos = 0, ki = 0, vi = 0;
    for (; pos < loads; ++pos) {
      const bool is_k = ki < n && ki < vi + ahead;
      const int tile = t0 + (is_k ? ki : vi);
      const int token = tile * kKeys + my_box * box;
      const bool issue = mine && token < len;
      if (a.table && issue && page_of != tile) {
        page = a.table[static_cast<int64_t>(r) * a.table_stride + token / a.page_size];
        if (page < 0 || page >= a.n_pages) {
          atomicOr(a.status, kStatusBadCache);
          page = a.n_pages;  // outside the tensor: the copy writes zeros
        }
        page_of = tile;
      }
      const int s = pos % P::kSlots;
      if (pos >= P::kSlots &&
          !warp_wait(&bar.empty[s], ((pos / P::kSlots) - 1) & 1u, &bar.abort, a.status))
        break;
      const int count = min(boxes, (len - tile * kKeys + box - 1) / box);
      if (lane == 0) mbar_arrive_expect_tx(&bar.full[s], count * P::kHalves * box * 128);
      __syncwarp();
      if (issue)
        tma_load_4d(smem_addr(ring + s * P::kTile + my_half * P::kHalf + my_box * box * 128),
                    is_k ? &map_k : &map_v, my_half * 64, g, a.table ? token & (a.page_size - 1) : token,
                    a.table ? page : r, &bar.full[s]);
      __syncwarp();
      if (is_k) ++ki; else ++vi;
    }
    if (ragged && pos == loads) {
      // The last V tile: rows past the end may hold anything, and 0 * NaN is
      // not 0, so they are cleared once the copy has landed.
      const int p = pos_v(n - 1, ahead, n), s = p % P::kSlots;
      warp_wait(&bar.full[s], (p / P::kSlots) & 1u, &bar.abort, a.status);
      constexpr int kUnits = D / 8;
      for (int e = ragged * kUnits + lane; e < kKeys * kUnits; e += 32)
        *reinterpret_cast<uint4*>(ring + s * P::kTile + unit_at<D>(e / kUnits, e % kUnits)) =
            make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.v_clean);
    }
    if (lane == 0)
      for (int j = max(0, pos - P::kSlots); j < pos; ++j)
        drain_wait(&bar.full[j % P::kSlots], (j / P::kSlots) & 1u);
    __syncwarp();
  } else if (warp == 9) {
    // ---------------------------------------------------------- MMA issue
    if (lane == 0 && n > 0) {
      auto wait = [&](uint64_t* b, uint32_t parity) {
        const bool ok = bounded_wait(b, parity, &bar.abort, a.status, kStatusTimeout);
        tc_fence_after();
        return ok;
      };
      auto wait_load = [&](int pos) {
        return wait(&bar.full[pos % P::kSlots], (pos / P::kSlots) & 1u);
      };
      auto free_load = [&](int pos) { umma_commit(&bar.empty[pos % P::kSlots]); };
      auto qk = [&](int s, int i) {
        const uint32_t qa = smem_addr(smem + (dual ? s : 0) * P::kTile);
        const uint32_t ka = smem_addr(ring + (pos_k(i, ahead) % P::kSlots) * P::kTile);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * P::kHalf + (kk & 3) * 32;
          umma_f16(tmem + s * kKeys, smem_desc(qa + off), smem_desc(ka + off), kIdescQK,
                   kk > 0 ? 1u : 0u);
        }
        umma_commit(&bar.s_full[s]);
      };
      auto pv = [&](int s, int i, bool accumulate) {
        const uint32_t va = smem_addr(ring + (pos_v(i, ahead, n) % P::kSlots) * P::kTile);
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          umma_f16_ts(tmem + 256 + s * 128, tmem + s * kKeys + kk * 8,
                      smem_desc_mn(va + kk * 2048, P::kHalf), idesc_pv(D),
                      kk > 0 || accumulate ? 1u : 0u);
      };
      const bool path = a.level > 0 && rank == 0;
      bool ok = wait(&bar.q_ready[0], 0u) && (!dual || wait(&bar.q_ready[1], 0u));
      if (dual) {
        ok = ok && wait_load(pos_k(0, ahead));
        if (ok) {
          qk(0, 0);
          qk(1, 0);
          free_load(pos_k(0, ahead));
        }
        for (int i = 0; ok && i < n; ++i) {
          for (int s = 0; ok && s < 2; ++s) {
            ok = wait(&bar.p_ready[s], i & 1u);
            if (ok && s == 0) ok = wait_load(pos_v(i, ahead, n));
            if (ok && s == 0 && i == n - 1 && ragged) ok = wait(&bar.v_clean, 0u);
            if (!ok) break;
            pv(s, i, path || i > 0);
            if (i + 1 < n) {
              if (s == 0) ok = wait_load(pos_k(i + 1, ahead));
              if (ok) qk(s, i + 1);
            } else {
              umma_commit(&bar.o_full[s]);
            }
          }
          if (!ok) break;
          free_load(pos_v(i, ahead, n));
          if (i + 1 < n) free_load(pos_k(i + 1, ahead));
        }
      } else {
        for (int s = 0; ok && s < min(2, n); ++s) {
          ok = wait_load(pos_k(s, ahead));
          if (!ok) break;
          qk(s, s);
          free_load(pos_k(s, ahead));
        }
        for (int i = 0; ok && i < n; ++i) {
          const int s = i & 1;
          ok = wait(&bar.p_ready[s], (i >> 1) & 1u) && wait_load(pos_v(i, ahead, n)) &&
               (!(ragged && i == n - 1) || wait(&bar.v_clean, 0u));
          if (!ok) break;
          pv(s, i, (path && s == 0) || i > 1);
          free_load(pos_v(i, ahead, n));
          if (i + 2 < n) {
            ok = wait_load(pos_k(i + 2, ahead));
            if (!ok) break;
            qk(s, i + 2);
            free_load(pos_k(i + 2, ahead));
          } else {
            umma_commit(&bar.o_full[s]);
          }
        }
      }
      umma_commit(&bar.drain);
      drain_wait(&bar.drain, 0u);
    }
    __syncwarp();
  }
  // The softmax warps' state lives past this point: their rows' o, m and l.
  const int s = warp >> 2;                         // stream of a softmax warp
  const int quarter = warp & 3;                    // its TMEM lanes
  const int tile_row = quarter * 32;               // first of its 32 rows in the tile
  const int first = row0 + (dual && s == 1 ? kRows : 0);
  const int tile_rows = dual && s == 1 ? rows - kRows : min(rows, kRows);
  const bool active = warp < 8 && tile_row < tile_rows;
  const int n_s = dual ? n : (n + 1 - s) / 2;      // key tiles of this stream
  const bool init = a.level > 0 && rank == 0 && (dual || s == 0);
  const uint32_t quad = static_cast<uint32_t>(tile_row) << 16;
  const uint32_t t_s = tmem + s * kKeys + quad, t_o = tmem + 256 + s * 128 + quad;
  float m = kNegInf, l = 0.f;
  bool dead = false;
  if (active) {
    // ---------------------------------------------------------- Q, path
    const int lrow = tile_row + lane;              // row of the tile
    const int i_row = first + lrow;
    const bool valid = lrow < tile_rows;
    uint8_t* qt = smem + (dual ? s : 0) * P::kTile;
    if (dual || s == 0) {
      // Coalesced: D / 8 lanes read a row. A negative scale flips q's signs (the
      // maximum below needs a factor >= 0).
      constexpr int kUnits = D / 8, kPer = 32 / kUnits;
      const uint32_t flip = a.scale_log2 < 0.f ? 0x80008000u : 0u;
      const int c = lane % kUnits;
#pragma unroll 8
      for (int j = 0; j < kUnits; ++j) {
        const int lr = tile_row + j * kPer + lane / kUnits;
        if (lr < tile_rows) {
          const int i = first + lr, b = i / G, h = g * G + (i - b * G);
          uint4 u = *reinterpret_cast<const uint4*>(
              a.q + (static_cast<int64_t>(r) * a.B + b) * a.q_stride + h * D + c * 8);
          u.x ^= flip;
          u.y ^= flip;
          u.z ^= flip;
          u.w ^= flip;
          *reinterpret_cast<uint4*>(qt + unit_at<D>(lr, c)) = u;
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_ready[s]);
    }
    const float sc = fabsf(a.scale_log2);
    if (a.level > 0) {
      int slot[SIDBEAM_MAX_DEPTH];
      float x[SIDBEAM_MAX_DEPTH];
      int at = valid ? i_row / G : -1;
      for (int u = a.level - 1; u >= 0; --u) {
        slot[u] = at;
        if (at >= 0) {
          const int p = a.bp[(static_cast<int64_t>(u) * a.R + r) * a.B + at];
          at = p < 0 ? -1 : (u > 0 && p >= a.B ? -1 : p);
        }
      }
      dead = at < 0;
      if (init) {
        const int64_t hd = static_cast<int64_t>(a.Hkv) * D;
        if (!dead) {
          for (int u = 0; u < a.level; ++u) {
            const uint4* k = reinterpret_cast<const uint4*>(
                a.kb + ((static_cast<int64_t>(u) * a.R + r) * a.B + slot[u]) * hd + g * D);
            float z = 0.f;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
              float kf[8], qf[8];
              bf16x8(k[c], kf);
              bf16x8(*reinterpret_cast<const uint4*>(qt + unit_at<D>(lrow, c)), qf);
#pragma unroll
              for (int e = 0; e < 8; ++e) z = fmaf(kf[e], qf[e], z);
            }
            x[u] = z * sc;
            m = fmaxf(m, x[u]);
          }
          for (int u = 0; u < a.level; ++u) {
            x[u] = ex2_approx(x[u] - m);
            l += x[u];
          }
        }
        for (int c0 = 0; c0 < D; c0 += 32) {
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.f;
          if (!dead) {
            for (int u = 0; u < a.level; ++u) {
              const uint4* v = reinterpret_cast<const uint4*>(
                  a.vb + ((static_cast<int64_t>(u) * a.R + r) * a.B + slot[u]) * hd + g * D + c0);
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                float vf[8];
                bf16x8(v[c], vf);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[c * 8 + e] = fmaf(x[u], vf[e], o[c * 8 + e]);
              }
            }
          }
          __syncwarp();
          tmem_st32(t_o + c0, reinterpret_cast<const uint32_t*>(o));
        }
        tmem_wait_st();
        tc_fence_before();
      }
    }
    // ---------------------------------------------------------- softmax
    bool started = init;
    for (int j = 0; j < n_s; ++j) {
      if (!warp_wait(&bar.s_full[s], j & 1u, &bar.abort, a.status)) break;
      tc_fence_after();
      float x[kKeys];
#pragma unroll
      for (int c = 0; c < kKeys; c += 32)
        tmem_ld32_async(t_s + c, reinterpret_cast<uint32_t*>(x) + c);
      tmem_wait_ld();
      const bool cut = ragged && j == n_s - 1 && (dual || ((n - 1) & 1) == s);
      if (cut) {
#pragma unroll
        for (int e = 0; e < kKeys; ++e)
          if (e >= ragged) x[e] = kNegInf;
      }
      float t = x[0];
#pragma unroll
      for (int e = 1; e < kKeys; ++e) t = fmaxf(t, x[e]);
      t *= sc;
      // The reference m moves only when a row's maximum passes it by 2^8: smaller
      // growth keeps the weights below 2^8 and spares the pass over O.
      const bool grow = !started || t > m + 8.f;
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float mn = fmaxf(m, t);
        if (started) {
          const float f = m > kNegInf ? ex2_approx(m - mn) : 0.f;
          l *= f;
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(t_o + c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(t_o + c, o);
          }
        }
        m = mn;
        started = true;
      }
      uint32_t p[kKeys / 2];
      float l0 = 0.f, l1 = 0.f;
      const float mref = m > kNegInf ? m : 0.f;
#pragma unroll
      for (int e = 0; e < kKeys; e += 2) {
        float p0 = ex2_approx(fmaf(x[e], sc, -mref)), p1 = ex2_approx(fmaf(x[e + 1], sc, -mref));
        if (cut) {
          p0 = e < ragged ? p0 : 0.f;
          p1 = e + 1 < ragged ? p1 : 0.f;
        }
        l0 += p0;
        l1 += p1;
        p[e / 2] = bf16x2(p0, p1);
      }
      l += l0 + l1;
      tmem_st32(t_s, p);
      tmem_st32(t_s + 32, p + 32);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.p_ready[s]);
    }
    if (n_s > 0) {
      warp_wait(&bar.o_full[s], 0u, &bar.abort, a.status);
      tc_fence_after();
    }
    if (dead) l = 0.f;
  }
  const bool has_o = n_s > 0 || init;
  if (dual && split == 1) {
    // ---------------------------------------------------------- direct output
    if (active) {
      // The warp's own rows of the Q tile (its MMAs are done) take the rows'
      // bf16 results and give them back in whole 128-byte lines.
      uint8_t* qt = smem + s * P::kTile;
      const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (has_o) {
          tmem_ld32(t_o + c, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        float f[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = l > 0.f ? __uint_as_float(o[e]) * inv : 0.f;
#pragma unroll
        for (int e = 0; e < 32; e += 8)
          *reinterpret_cast<uint4*>(qt + unit_at<D>(tile_row + lane, (c + e) / 8)) =
              make_uint4(bf16x2(f[e], f[e + 1]), bf16x2(f[e + 2], f[e + 3]),
                         bf16x2(f[e + 4], f[e + 5]), bf16x2(f[e + 6], f[e + 7]));
      }
      __syncwarp();
      constexpr int kUnits = D / 8, kPer = 32 / kUnits;
      const int c = lane % kUnits;
#pragma unroll
      for (int j = 0; j < kUnits; ++j) {
        const int lr = tile_row + j * kPer + lane / kUnits;
        if (lr < tile_rows) {
          const int i = first + lr, b = i / G, h = g * G + (i - b * G);
          *reinterpret_cast<uint4*>(a.out + (static_cast<int64_t>(r) * a.B + b) * a.out_stride +
                                    h * D + c * 8) =
              *reinterpret_cast<const uint4*>(qt + unit_at<D>(lr, c));
        }
      }
    }
  } else {
    // ---------------------------------------------------------- joined output
    // Partial rows [stream][row] of (o, m, l) in fp32 where the ring was.
    float* part = reinterpret_cast<float*>(ring);
    __syncthreads();  // every MMA and copy of this CTA has finished
    if (active) {
      float* o_row = part + (s * kRows + tile_row + lane) * P::kPitch;
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (has_o) {
          tmem_ld32(t_o + c, o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          *reinterpret_cast<uint4*>(o_row + c + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
      }
      o_row[D] = l > 0.f ? m : kNegInf;
      o_row[D + 1] = l;
    }
    if (split > 1)
      cluster_sync();
    else
      __syncthreads();
    if (warp < 8) {
      const int sources = dual ? split : 2 * split;
      for (int i = rank * 8 + warp; i < rows; i += 8 * split) {
        // Source p: rank p (two row tiles), or rank p / 2's stream p & 1.
        auto at = [&](int p) {
          const int st = dual ? i / kRows : p & 1;
          return peer_addr(part + (st * kRows + i % kRows) * P::kPitch, dual ? p : p >> 1);
        };
        float mp = kNegInf, lp = 0.f;
        if (lane < sources) {
          mp = ld_peer(at(lane) + D * 4);
          lp = ld_peer(at(lane) + D * 4 + 4);
        }
        const float top = warp_max(mp);
        const float w = mp > kNegInf ? ex2_approx(mp - top) : 0.f;
        const float sum = warp_sum(w * lp);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < sources; ++p) {
          const float wp = __shfl_sync(0xFFFFFFFFu, w, p);
          if (wp > 0.f && lane < D / 4) {
            const float4 v = ld_peer4(at(p) + lane * 16);
            o.x = fmaf(wp, v.x, o.x);
            o.y = fmaf(wp, v.y, o.y);
            o.z = fmaf(wp, v.z, o.z);
            o.w = fmaf(wp, v.w, o.w);
          }
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const int ii = row0 + i, b = ii / G, h = g * G + (ii - b * G);
        if (lane < D / 4)
          *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(r) * a.B + b) * a.out_stride +
                                    h * D + lane * 4) =
              make_uint2(bf16x2(o.x * inv, o.y * inv), bf16x2(o.z * inv, o.w * inv));
      }
    }
    if (split > 1) cluster_sync();  // no CTA leaves while its rows are read
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free(tmem, 512);
}

// 4-D map of a cache [n_pages][page_size][Hkv][D], box [1][box][1][64].
template <int D>
bool make_map(CUtensorMap* map, const void* base, const AttnArgs& a, int box) {
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

template <int D>
int launch_attention(const AttnArgs& a, cudaStream_t stream) {
  using P = Plan<D>;
  CUtensorMap mk, mv;
  const int box = a.table ? std::min(a.page_size, kKeys) : kKeys;
  if (!make_map<D>(&mk, a.k, a, box) || !make_map<D>(&mv, a.v, a, box))
    return set_error(SIDBEAM_ERR_CUDA, "beam_attention: tensor map encoding failed");
  static std::mutex mu;
  static bool done[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_error(e, "beam_attention: cudaGetDevice");
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev < 0 || dev >= 64 || !done[dev]) {
      e = cudaFuncSetAttribute(attention_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               P::kSmem);
      if (e != cudaSuccess) return cuda_error(e, "beam_attention: cudaFuncSetAttribute");
      if (dev >= 0 && dev < 64) done[dev] = true;
    }
  }
  const int all = a.B * (a.H / a.Hkv);
  const int pairs = (all + 2 * kRows - 1) / (2 * kRows);
  const int64_t items = static_cast<int64_t>(pairs) * a.Hkv * a.R;
  const int64_t cap = a.table ? static_cast<int64_t>(a.table_stride) * a.page_size : a.page_size;
  const int64_t max_tiles = (cap + kKeys - 1) / kKeys;
  // CTAs per item: while they fit the SMs and each has two key tiles.
  int split = 1;
  while (split < kMaxSplit && items * split * 2 <= device_sm_count() && split * 4 <= max_tiles)
    split *= 2;
  cudaLaunchConfig_t lc{};
  lc.gridDim = dim3(static_cast<unsigned>(pairs * split * a.R), static_cast<unsigned>(a.Hkv));
  lc.blockDim = dim3(kThreads);
  lc.dynamicSmemBytes = P::kSmem;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  e = cudaLaunchKernelEx(&lc, attention_kernel<D>, mk, mv, a, pairs, split);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? SIDBEAM_OK : cuda_error(e, "beam_attention: launch");
}

bool misaligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

}  // namespace
}  // namespace sidbeam

using namespace sidbeam;

extern "C" int beam_attention(const void* q, int64_t q_row_stride, const void* k_cache,
                              const void* v_cache, int64_t page_stride, int64_t token_stride,
                              int n_pages, int page_size, const int32_t* page_table,
                              int pages_per_request, const int32_t* cache_len, int level,
                              const int32_t* bp_parent, const void* k_beam, const void* v_beam,
                              int R, int B, int H, int Hkv, int D, float scale, void* out,
                              int64_t out_row_stride, void* workspace, size_t workspace_bytes,
                              void* stream) {
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
  a.scale_log2 = scale * kLog2e;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.out_stride = out_row_stride;
  a.status = static_cast<uint32_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return D == 64 ? launch_attention<64>(a, s) : launch_attention<128>(a, s);
}
