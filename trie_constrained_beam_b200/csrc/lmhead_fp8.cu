// SID-range lm_head with both operands in e4m3 and a scale per 128 elements
// along d, on the 5th-generation tensor cores.
//
// flashrec 0.1.0 (PyPI page), Features: W8A8 FP8; Features > Decoding ("SID
// constraint"): the lm_head covers the SID token range only.
//
//   z[m][c] = sum_b sa[m][b] * sw[c / 128][b] * (sum_{k in b} q[m][k] * w[c][k])
//
// The scales change every 128 columns of d, so the tensor core cannot carry one
// accumulator through the whole dot product: each block's sum (4 MMAs of K = 32)
// goes to a TMEM accumulator of its own, and the epilogue warps add it, times
// the row's and the code block's scale, to fp32 registers while the MMAs of the
// next block run into the other accumulators.
#include <cuda_bf16.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "internal.h"
#include "tcgen05.cuh"

namespace sidbeam {
namespace {

using namespace dev;

constexpr int kBlock = SIDBEAM_FP8_BLOCK;  // 128 e4m3: 128 bytes, one swizzle row

// Instruction descriptor of kind::f8f6f4: fp32 accumulator, e4m3 A and B (format
// 0), both K-major, M = 128.
constexpr uint32_t idesc_f8(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | ((128u >> 4) << 24);
}

struct Fp8Args {
  int M, V, nb;               // rows, codes, blocks of 128 along d
  const float* sa;            // [M][nb]
  const float* sw;            // [ceil(V/128)][nb]
  void* out;                  // [M][ld]
  int64_t ld;
  uint32_t* status;
};

// ------------------------------------------------------------ many rows
// Persistent over tiles of 128 rows x kTileN codes. Two warp groups are the epilogue,
// each on half of a tile's columns: 128 (or 64) fp32 sums per thread. The third issues
// (warp 8: TMA, warp 9: MMA). A block's MMAs take 512 cycles, and so at least does
// its way out: 128 KB of TMEM reads and 32K FMAs per SM; the epilogue keeps three
// loads of 32 columns in turn, so that neither waits for the other.
//
// 4096 x 8192 x 2048 to fp32: 84 us at the full clock of 1,965 MHz (1,630 TFLOP/s, half of
// the 8-bit rate), 96.5 us in seconds of calls, where the 1,000 W power cap holds the
// clock at 1,620 MHz (1,425 TFLOP/s); to bf16 74.5 and 85.5. The figures below are at full clock.
// A block takes about 1,130 cycles, and a tile's store about 6,700 that overlap the
// next tile's first blocks only. No unit is full: the tensor pipe 41%, issue slots
// 48%, L2 26%, DRAM 18% of its rate; each SM takes in 48 KB a block, 43 bytes a
// cycle (12 TB/s over all SMs). Twice the epilogue warps with half the columns each
// measured 88 us against 83, so it is not their latency alone.
constexpr int kTileM = 128;
constexpr int kABytes = kTileM * kBlock;
constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
constexpr int kChunk = 128;                              // bytes of a row per store chunk
constexpr int kStore = kEpiWarps * 32 * kChunk;          // 32 KiB
template <int kTileN>
struct GemmPlan {
  static constexpr int kStages = kTileN == 256 ? 4 : 6;  // of 48 or 32 KiB
  static constexpr int kStageBytes = (kTileM + kTileN) * kBlock;
  static constexpr int kAccs = 512 / kTileN;             // TMEM accumulators
  static constexpr int kCols = kTileN / 2;               // columns of an epilogue warp
  static constexpr int kSmem = kStages * kStageBytes + kStore + 1024 + 256;
};

template <int kTileN, typename T>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_h,
                    const __grid_constant__ CUtensorMap map_w, const Fp8Args a) {
  using P = GemmPlan<kTileN>;
  constexpr int kStages = P::kStages, kStageBytes = P::kStageBytes, kAccs = P::kAccs;
  constexpr int kCols = P::kCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* store = smem + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(store + kStore);
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;  // [kAccs]
  uint64_t* acc_empty = acc_full + kAccs;
  uint64_t* drain = acc_empty + kAccs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int m_tiles = (a.M + kTileM - 1) / kTileM;
  const int n_tiles = (a.V + kTileN - 1) / kTileN;
  const int tiles = m_tiles * n_tiles;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kAccs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) tmem_alloc(tmem_slot, 512);
  wait_prior();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  release_next();
  constexpr uint32_t tmem = 0u;  // all 512 columns: they begin at column 0

  // Registers: 384 threads start with 168 each; 232 + 232 + 40 = 3 * 168.
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 8) {
      if (lane == 0) {
        prefetch_map(&map_h);
        prefetch_map(&map_w);
        uint32_t it = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
          const int nt = t / m_tiles, mt = t - nt * m_tiles;
          for (int k = 0; k < a.nb; ++k, ++it) {
            const uint32_t s = it % kStages;
            if (it >= kStages && !lane_wait(&empty[s], it / kStages - 1, abort_flag, a.status)) {
              ok = false;
              break;
            }
            uint8_t* st = smem + s * kStageBytes;
            mbar_arrive_expect_tx(&full[s], kStageBytes);
            tma_load_2d(st, &map_h, k * kBlock, mt * kTileM, &full[s]);
            tma_load_2d(st + kABytes, &map_w, k * kBlock, nt * kTileN, &full[s]);
          }
        }
        for (uint32_t j = it > kStages ? it - kStages : 0u; j < it; ++j)
          drain_wait(&full[j % kStages], (j / kStages) & 1u);
      }
    } else if (warp == 9) {
      if (elect_one()) {
        uint32_t it = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
          for (int k = 0; k < a.nb; ++k, ++it) {
            const uint32_t s = it % kStages, ab = it % kAccs;
            if (!lane_wait(&full[s], it / kStages, abort_flag, a.status) ||
                (it >= kAccs && !lane_wait(&acc_empty[ab], it / kAccs - 1, abort_flag, a.status))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t da = smem_desc(smem_addr(smem + s * kStageBytes));
            const uint64_t db = smem_desc(smem_addr(smem + s * kStageBytes + kABytes));
#pragma unroll
            for (int kk = 0; kk < kBlock / 32; ++kk)
              umma_f8(tmem + ab * kTileN, da + kk * 2, db + kk * 2, idesc_f8(kTileN),
                      kk > 0 ? 1u : 0u);
            umma_commit(&acc_full[ab]);
            umma_commit(&empty[s]);
          }
        }
        umma_commit(drain);
        drain_wait(drain, 0u);
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    const int quarter = warp & 3;       // TMEM lanes 32 * quarter .. + 31
    const int col0 = (warp >> 2) * kCols;  // first of its columns in the tile
    uint8_t* chunk = store + warp * 32 * kChunk;
    uint32_t it = 0;
    bool ok = true;
    for (int t = blockIdx.x; ok && t < tiles; t += gridDim.x) {
      const int nt = t / m_tiles, mt = t - nt * m_tiles;
      const int row = mt * kTileM + quarter * 32 + lane;
      const int n0 = nt * kTileN + col0;
      const float* sa = a.sa + static_cast<int64_t>(min(row, a.M - 1)) * a.nb;
      const float* sw = a.sw + static_cast<int64_t>(min(n0, a.V - 1) / kBlock) * a.nb;
      float acc[kCols];
#pragma unroll
      for (int e = 0; e < kCols; ++e) acc[e] = 0.f;
      float s = sa[0] * sw[0];
#pragma unroll 1
      for (int k = 0; k < a.nb; ++k, ++it) {
        const uint32_t ab = it % kAccs;
        const float f = s;
        if (k + 1 < a.nb) s = sa[k + 1] * sw[k + 1];
        if (!warp_wait(&acc_full[ab], it / kAccs, abort_flag, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem + ab * kTileN + col0 +
                               (static_cast<uint32_t>(quarter * 32) << 16);
        uint32_t v0[32], v1[32], v2[32];
        auto add = [&](int j, const uint32_t (&v)[32]) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            acc[j * 32 + e] = fmaf(__uint_as_float(v[e]), f, acc[j * 32 + e]);
        };
        auto release = [&] {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[ab]);
        };
        tmem_ld32_async(taddr, v0);
        tmem_ld32_async(taddr + 32, v1);
        tmem_wait_ld32(v0);
        tmem_wait_ld32(v1);
        if constexpr (kCols == 64) {
          release();
          add(0, v0);
          add(1, v1);
        } else {
          tmem_ld32_async(taddr + 64, v2);
          add(0, v0);
          tmem_ld32_async(taddr + 96, v0);
          add(1, v1);
          tmem_wait_ld32(v2);
          tmem_wait_ld32(v0);
          release();
          add(2, v2);
          add(3, v0);
        }
      }
      if (!ok) break;
      // 128-byte pieces of the warp's 32 rows through shared memory (16-byte
      // units, unit u of row l at u ^ (l & 7)), so that global stores cover
      // whole lines.
      constexpr int kPiece = kChunk / static_cast<int>(sizeof(T));  // 32 fp32 or 64 bf16
#pragma unroll
      for (int j = 0; j < kCols / kPiece; ++j) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          uint4 w;
          if constexpr (sizeof(T) == 4) {
            const float* f = acc + j * 32 + u * 4;
            w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                           __float_as_uint(f[3]));
          } else {
            const float* f = acc + j * 64 + u * 8;
            w = make_uint4(bf16x2(f[0], f[1]), bf16x2(f[2], f[3]), bf16x2(f[4], f[5]),
                           bf16x2(f[6], f[7]));
          }
          *reinterpret_cast<uint4*>(chunk + lane * kChunk + ((u ^ (lane & 7)) << 4)) = w;
        }
        __syncwarp();
        constexpr int kUnit = 16 / static_cast<int>(sizeof(T));
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const int l = p * 4 + (lane >> 3), u = lane & 7;
          const uint4 w = *reinterpret_cast<const uint4*>(chunk + l * kChunk + ((u ^ (l & 7)) << 4));
          const int r = mt * kTileM + quarter * 32 + l;
          const int c = n0 + j * kPiece + u * kUnit;
          if (r < a.M) {
            T* o = static_cast<T*>(a.out) + static_cast<int64_t>(r) * a.ld + c;
            if (c + kUnit <= a.V) {
              *reinterpret_cast<uint4*>(o) = w;
            } else {
              T f[kUnit];
              *reinterpret_cast<uint4*>(f) = w;
#pragma unroll
              for (int e = 0; e < kUnit; ++e)
                if (c + e < a.V) o[e] = f[e];
            }
          }
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free(tmem, 512);
}

// ------------------------------------------------------------ few rows
// The operands change places: a tile is 128 codes (M of the MMA) x NB rows, so a
// handful of rows does not leave most of a 128-row tile empty, and the weight,
// which is all that counts here, is read once. The CTAs of a cluster share a
// tile and split d; each adds up its part in registers, and the parts meet
// through distributed shared memory in rank order (the same sum every time).
//
// Bound by the weight's bytes and the start and end of a call: 32 rows of
// 8192 x 2048 take 7.5 us, a third of the copy bandwidth (2.7 us of bytes, about
// 2 us for an empty kernel, then the first loads' and the cluster's latency). Few rows
// do not reach the power cap: the figures here and at the rules on the host side hold
// in seconds of calls too (but 15.7 us for the 15.1 of 512 rows).
constexpr int kRowThreads = 192;  // TMA warp, MMA warp, 4 epilogue warps

template <int NB>
struct RowPlan {
  static constexpr int kStage = (kTileM + NB) * kBlock;
  static constexpr int kAcc = 8;                      // TMEM accumulators of NB columns
  static constexpr int kTmemCols = NB * kAcc < 32 ? 32 : NB * kAcc;
};

template <int NB, typename T>
__global__ void __launch_bounds__(kRowThreads, 1)
    fp8_rows_kernel(const __grid_constant__ CUtensorMap map_h,
                    const __grid_constant__ CUtensorMap map_w, const Fp8Args a, int split,
                    int stages) {
  using P = RowPlan<NB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[8], empty[8], acc_full[8], acc_empty[8], drain;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = blockIdx.x / split;
  const int m0 = blockIdx.y * NB;
  const int kb0 = a.nb * rank / split, kb1 = a.nb * (rank + 1) / split;
  const int n = kb1 - kb0;
  float* table = reinterpret_cast<float*>(smem + stages * P::kStage);  // [n][NB]

  if (threadIdx.x == 0) {
    for (int s = 0; s < 8; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&acc_full[s], 1);
      mbar_init(&acc_empty[s], 4);
    }
    mbar_init(&drain, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(&tmem_slot, P::kTmemCols);
  wait_prior();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  release_next();
  const uint32_t tmem = tmem_slot;

  float acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j) acc[j] = 0.f;
  if (warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (; i < n; ++i) {
        const int s = i % stages;
        if (i >= stages && !lane_wait(&empty[s], i / stages - 1, &abort_flag, a.status)) break;
        uint8_t* st = smem + s * P::kStage;
        mbar_arrive_expect_tx(&full[s], P::kStage);
        tma_load_2d(st, &map_w, (kb0 + i) * kBlock, tile * kTileM, &full[s]);
        tma_load_2d(st + kABytes, &map_h, (kb0 + i) * kBlock, m0, &full[s]);
      }
      for (int j = max(0, i - stages); j < i; ++j)
        drain_wait(&full[j % stages], (j / stages) & 1u);
    }
  } else if (warp == 1) {
    if (elect_one()) {
      for (int i = 0; i < n; ++i) {
        const int s = i % stages, ab = i % P::kAcc;
        if ((i >= P::kAcc &&
             !lane_wait(&acc_empty[ab], i / P::kAcc - 1, &abort_flag, a.status)) ||
            !lane_wait(&full[s], i / stages, &abort_flag, a.status))
          break;
        tc_fence_after();
        const uint32_t sw = smem_addr(smem + s * P::kStage);
#pragma unroll
        for (int kk = 0; kk < kBlock / 32; ++kk)
          umma_f8(tmem + ab * NB, smem_desc(sw + kk * 32), smem_desc(sw + kABytes + kk * 32),
                  idesc_f8(NB), kk > 0 ? 1u : 0u);
        umma_commit(&empty[s]);
        umma_commit(&acc_full[ab]);
      }
      umma_commit(&drain);
      drain_wait(&drain, 0u);
    }
  } else {
    // table[i][j] = the factor of row m0 + j in block kb0 + i for this tile.
    const int e0 = threadIdx.x - 64;
    for (int e = e0; e < n * NB; e += 128) {
      const int j = e / n, i = e - j * n;
      table[i * NB + j] = m0 + j < a.M
                              ? a.sa[static_cast<int64_t>(m0 + j) * a.nb + kb0 + i] *
                                    a.sw[static_cast<int64_t>(tile) * a.nb + kb0 + i]
                              : 0.f;
    }
    named_sync(1, 128);
    const int quarter = warp & 3;
    for (int i = 0; i < n; ++i) {
      const int ab = i % P::kAcc;
      if (!warp_wait(&acc_full[ab], i / P::kAcc, &abort_flag, a.status)) break;
      tc_fence_after();
      const uint32_t taddr = tmem + ab * NB + (static_cast<uint32_t>(quarter * 32) << 16);
#pragma unroll
      for (int j0 = 0; j0 < NB; j0 += 16) {
        uint32_t v[16];
        tmem_ld16(taddr + j0, v);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(table + i * NB + j0 + j);
          acc[j0 + j] = fmaf(__uint_as_float(v[j]), f.x, acc[j0 + j]);
          acc[j0 + j + 1] = fmaf(__uint_as_float(v[j + 1]), f.y, acc[j0 + j + 1]);
          acc[j0 + j + 2] = fmaf(__uint_as_float(v[j + 2]), f.z, acc[j0 + j + 2]);
          acc[j0 + j + 3] = fmaf(__uint_as_float(v[j + 3]), f.w, acc[j0 + j + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[ab]);
    }
  }
  // The stages are free now (every block has been multiplied).
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem, P::kTmemCols);
  float* part = reinterpret_cast<float*>(smem);  // [NB][128]
  const int c_local = (warp & 3) * 32 + lane;
  const int c = tile * kTileM + c_local;
  T* out = static_cast<T*>(a.out) + c;
  if (split == 1) {
    if (warp >= 2 && c < a.V) {
#pragma unroll
      for (int j = 0; j < NB; ++j)
        if (m0 + j < a.M) out[static_cast<int64_t>(m0 + j) * a.ld] = static_cast<T>(acc[j]);
    }
    return;
  }
  if (warp >= 2) {
#pragma unroll
    for (int j = 0; j < NB; ++j) part[j * 128 + c_local] = acc[j];
  }
  cluster_sync();
  if (warp >= 2 && c < a.V) {
    // Eight rows' parts in flight at a time (a remote load takes long).
    const int rows = min(NB, a.M - m0);
    for (int j0 = rank; j0 < rows; j0 += 8 * split) {
      float z[8] = {};
#pragma unroll 2
      for (int p = 0; p < split; ++p) {
        const uint32_t at = peer_addr(&part[c_local], p);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = j0 + e * split;
          v[e] = j < rows ? ld_peer(at + j * 512) : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] += v[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j0 + e * split < rows)
          out[static_cast<int64_t>(m0 + j0 + e * split) * a.ld] = static_cast<T>(z[e]);
    }
  }
  cluster_sync();  // no CTA leaves while another still reads its part
}

// ------------------------------------------------------------ host side
// 2-D e4m3 tensor map over a row-major [rows][cols] matrix, box [box_rows][128].
bool make_map(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_rows) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBlock), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Opts `kernel` into `smem` bytes of shared memory, once per device and kernel
// (`done`: that kernel's flags).
template <typename K>
cudaError_t opt_in(K kernel, int smem, bool (&done)[64]) {
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  return e;
}

template <int kTileN, typename T>
int launch_gemm(const void* h, const void* w, const Fp8Args& a, int d, cudaStream_t stream) {
  CUtensorMap mh, mw;
  if (!make_map(&mh, h, a.M, d, kTileM) || !make_map(&mw, w, a.V, d, kTileN))
    return set_error(SIDBEAM_ERR_CUDA, "lmhead_logits_fp8: tensor map encoding failed");
  static bool done[64] = {};
  cudaError_t e = opt_in(fp8_gemm_kernel<kTileN, T>, GemmPlan<kTileN>::kSmem, done);
  if (e != cudaSuccess) return cuda_error(e, "lmhead_logits_fp8: cudaFuncSetAttribute");
  const int64_t tiles =
      static_cast<int64_t>((a.M + kTileM - 1) / kTileM) * ((a.V + kTileN - 1) / kTileN);
  const int grid = static_cast<int>(std::min<int64_t>(tiles, device_sm_count()));
  e = launch_dependent(fp8_gemm_kernel<kTileN, T>, dim3(static_cast<unsigned>(grid)), kThreads,
                       GemmPlan<kTileN>::kSmem, 1, stream, mh, mw, a);
  return e == cudaSuccess ? SIDBEAM_OK : cuda_error(e, "lmhead_logits_fp8: launch");
}

template <int NB, typename T>
int launch_rows(const void* h, const void* w, const Fp8Args& a, int d, cudaStream_t stream) {
  using P = RowPlan<NB>;
  CUtensorMap mh, mw;
  if (!make_map(&mh, h, a.M, d, NB) || !make_map(&mw, w, a.V, d, kTileM))
    return set_error(SIDBEAM_ERR_CUDA, "lmhead_logits_fp8: tensor map encoding failed");
  const int tiles = (a.V + kTileM - 1) / kTileM;
  const int groups = (a.M + NB - 1) / NB;
  const int sms = device_sm_count();
  // CTAs per tile: up to 8 while all clusters run at once, one CTA to an SM, and
  // every CTA has a block (1 x 8192 x 2048: 6.2 us, unsplit 8.7; 16 x 4096 x 8192:
  // 11.8, unsplit 28.6; for 16 tiles, 8 CTAs each instead of 4 would not run at once:
  // 32 x 2048 x 2048 6.2 instead of 5.7).
  int log2 = 0;
  while (log2 < 3 && (2 << log2) <= a.nb && tiles * groups << (log2 + 1) <= sms) {
    static std::mutex mu;
    static int cache[64][4] = {};
    int fit = 0;
    const cudaError_t e =
        clusters_at_once(fp8_rows_kernel<NB, T>, kRowThreads, 224 * 1024, log2 + 1, mu, cache, &fit);
    if (e != cudaSuccess)
      return cuda_error(e, "lmhead_logits_fp8: cudaOccupancyMaxActiveClusters");
    if (tiles * groups > fit) break;
    ++log2;
  }
  const int split = 1 << log2;
  const int n = (a.nb + split - 1) / split;
  const int table = n * NB * 4;
  // More CTAs than SMs: two to an SM (32 x 32768 x 2048: 16.7 us, one to an SM 22.8).
  const int room = tiles * groups * split > sms ? 112 : 224;
  const int left = room * 1024 - 1024 - table;
  const int stages = std::max(2, std::min({8, n, left / P::kStage}));
  const int smem = 1024 + std::max(stages * P::kStage + table, NB * 128 * 4);
  static bool done[64] = {};
  cudaError_t e = opt_in(fp8_rows_kernel<NB, T>, 224 * 1024, done);
  if (e != cudaSuccess) return cuda_error(e, "lmhead_logits_fp8: cudaFuncSetAttribute");
  e = launch_dependent(fp8_rows_kernel<NB, T>,
                       dim3(static_cast<unsigned>(tiles * split), static_cast<unsigned>(groups)),
                       kRowThreads, smem, split, stream, mh, mw, a, split, stages);
  return e == cudaSuccess ? SIDBEAM_OK : cuda_error(e, "lmhead_logits_fp8: launch");
}

// Few rows up to 32: with 64 rows of 8192 x 2048 the few-rows kernel took 9.8 us, the
// other 8.1. 16 or 32 of them a tile, since a tile's promotion costs its whole width.
// Above, 128 codes a tile while 256 would leave half of the SMs without one:
// 129 rows (64 wide tiles) 9.3 us against 13.4, 512 rows (128 wide tiles) 17.0
// against 15.0.
template <typename T>
int launch(const void* h, const void* w, const Fp8Args& a, int d, cudaStream_t stream) {
  if (a.M <= 16) return launch_rows<16, T>(h, w, a, d, stream);
  if (a.M <= 32) return launch_rows<32, T>(h, w, a, d, stream);
  const int64_t tiles = static_cast<int64_t>((a.M + kTileM - 1) / kTileM) * ((a.V + 255) / 256);
  return 2 * tiles <= device_sm_count() ? launch_gemm<128, T>(h, w, a, d, stream)
                                        : launch_gemm<256, T>(h, w, a, d, stream);
}

bool misaligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0;
}

}  // namespace
}  // namespace sidbeam

using namespace sidbeam;

extern "C" int lmhead_logits_fp8(const void* hidden_q, const float* hidden_scale, const void* w_q,
                                 const float* w_scale, int M, int V, int d, void* logits,
                                 sidbeam_dtype dtype, int64_t ld, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (dtype != SIDBEAM_F32 && dtype != SIDBEAM_BF16)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "lmhead_logits_fp8: unknown dtype %d",
                     static_cast<int>(dtype));
  if (M < 0 || V < 1 || V > SIDBEAM_MAX_V || d < 16 || d > SIDBEAM_MAX_HIDDEN || (d & 15) != 0)
    return set_error(SIDBEAM_ERR_INVALID_ARG,
                     "lmhead_logits_fp8: bad shape M=%d V=%d d=%d (d a multiple of 16, at most %d)",
                     M, V, d, SIDBEAM_MAX_HIDDEN);
  if (M == 0) return SIDBEAM_OK;
  if (!hidden_q || !hidden_scale || !w_q || !w_scale || !logits)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "lmhead_logits_fp8: NULL pointer argument");
  if (M > 0x7FFFFFFF - kTileM ||
      (static_cast<int64_t>(M) + 127) / 128 * ((V + 127) / 128) > 0x3FFFFFFF)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "lmhead_logits_fp8: M=%d x V=%d too large", M, V);
  const int esize = dtype == SIDBEAM_BF16 ? 2 : 4;
  if (ld < V)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "lmhead_logits_fp8: ld=%lld < V=%d",
                     static_cast<long long>(ld), V);
  if (misaligned(hidden_q, 16) || misaligned(w_q, 16) || misaligned(logits, 16) ||
      misaligned(hidden_scale, 4) || misaligned(w_scale, 4) || (ld * esize) % 16 != 0)
    return set_error(SIDBEAM_ERR_ALIGNMENT,
                     "lmhead_logits_fp8: hidden_q, w_q and logits must be 16-byte aligned, "
                     "ld * sizeof(dtype) %% 16 == 0");
  if (!workspace || workspace_bytes < 256 || misaligned(workspace, 256))
    return set_error(SIDBEAM_ERR_WORKSPACE,
                     "lmhead_logits_fp8: workspace of >= 256 bytes, 256-byte aligned");
  Fp8Args a{};
  a.M = M;
  a.V = V;
  a.nb = (d + kBlock - 1) / kBlock;
  a.sa = hidden_scale;
  a.sw = w_scale;
  a.out = logits;
  a.ld = ld;
  a.status = static_cast<uint32_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return dtype == SIDBEAM_BF16 ? launch<__nv_bfloat16>(hidden_q, w_q, a, d, s)
                               : launch<float>(hidden_q, w_q, a, d, s);
}
