// The 8-bit operands of the lm_head product: residual_rmsnorm_fp8 (the rows)
// and lmhead_quantize_fp8 (the weight).
//
// flashrec 0.1.0 (PyPI page), Features: W8A8 FP8 weights and activations, the
// RMS norm fused with the quantisation of its output.
//
// A block of 128 elements y shares scale = max(max |y|, 448 * 2^-100) / 448 and
// holds q = e4m3(y * (1 / scale)): the largest element lands on the largest
// e4m3 value, every other keeps a relative rounding of at most 2^-4. The
// quotient and the reciprocal are rounded once each in fp32, so q depends on y
// alone. The floor 2^-100 keeps the reciprocal finite for blocks of zeros.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "tcgen05.cuh"

namespace sidbeam {
namespace {

using namespace dev;

constexpr int kBlock = SIDBEAM_FP8_BLOCK;
constexpr float kFp8Max = 448.f;
constexpr float kMinAmax = 448.f * 7.888609052210118e-31f;  // 448 * 2^-100

__device__ __forceinline__ float2 bf16x2_to_f32(uint32_t u) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

// Four e4m3 values, round to nearest even; magnitudes above 448 (a product
// rounded up past it) become 448.
__device__ __forceinline__ uint32_t f32x4_to_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

// Scale of a block whose largest magnitude is amax, and its reciprocal.
__device__ __forceinline__ float block_scale(float amax, float& inv) {
  const float scale = __fdiv_rn(fmaxf(amax, kMinAmax), kFp8Max);
  inv = __frcp_rn(scale);
  return scale;
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = bf16x2_to_f32(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

// ------------------------------------------------------------ residual RMS norm
// T threads own a row, each K chunks of 8 consecutive elements, chunk i + k * T
// (16-byte loads; 16 neighbouring threads hold one scale block). The row stays
// in registers between its sum of squares and its quantisation, so it is read
// once: 7 bytes per element in all, the bound of this kernel (8192 rows of 2048:
// 20.4 us at full clock, 89% of the copy bandwidth; 21.3 in seconds of calls, where the
// power cap holds the clock at 1,777 MHz). T threads a row by its size (us per call at
// full clock; up to d = 512 part of the inputs stays in L2, 16384 rows up to 1024, 8192
// of 2048, 4096 above; T = 32: four rows to a CTA):
//   d      256    512    1024   2048   4096   8192
//   32     6.0   11.3    20.9   23.6
//   128   17.2   18.1    20.5   20.2   21.3   41.4
//   256                         21.4   20.9   40.4
// up to 512 a warp wins, its shuffles being the whole sum; at 1024 the two are
// level with many rows and 128 threads win with few (512 rows: 1.9 against 2.4);
// above, a warp's registers hold too few rows in flight. 256 threads, level with 128 at
// 4096 and 8192, only where 128 would need more than 8 chunks each.
template <int T, int K>
__global__ void __launch_bounds__(T == 32 ? 128 : T)
    rmsnorm_kernel(const uint4* x, const uint4* residual, const uint4* weight,
                   float eps, int M, int d, uint4* residual_out, uint2* __restrict__ q,
                   float* __restrict__ scale) {
  constexpr int kRows = T == 32 ? 4 : 1;
  wait_prior();
  release_next();
  const int t = T == 32 ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + (T == 32 ? threadIdx.x >> 5 : 0);
  if (row >= M) return;
  const int chunks = d >> 3;
  const int64_t base = row * chunks;
  float h[K][8];
  float sum = 0.f;
  uint4 a[K], b[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = t + k * T;
    a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
    if (c < chunks) {
      a[k] = x[base + c];
      if (residual) b[k] = residual[base + c];
    }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = t + k * T;
    float r[8];
    unpack8(a[k], h[k]);
    unpack8(b[k], r);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[k][e] += r[e];
      sum = fmaf(h[k][e], h[k][e], sum);
    }
    if (residual_out && c < chunks)
      residual_out[base + c] =
          make_uint4(bf16x2(h[k][0], h[k][1]), bf16x2(h[k][2], h[k][3]),
                     bf16x2(h[k][4], h[k][5]), bf16x2(h[k][6], h[k][7]));
  }
  // The weight, on its way during the sum. (No read-only loads here: they are not
  // ordered behind wait_prior().)
#pragma unroll
  for (int k = 0; k < K; ++k) {
    a[k] = make_uint4(0u, 0u, 0u, 0u);
    if (t + k * T < chunks) a[k] = weight[t + k * T];
  }
  sum = warp_sum(sum);
  if constexpr (T > 32) {
    __shared__ float part[T / 32];
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) sum += part[w];
  }
  const float rinv = __frsqrt_rn(sum / static_cast<float>(d) + eps);
  const int nb = (d + kBlock - 1) / kBlock;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = t + k * T;
    const bool in = c < chunks;
    float w[8];
    unpack8(a[k], w);
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[k][e] = h[k][e] * rinv * w[e];
      amax = fmaxf(amax, fabsf(h[k][e]));
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    float inv;
    const float s = block_scale(amax, inv);
    if (in) {
      q[base + c] = make_uint2(
          f32x4_to_e4m3(h[k][0] * inv, h[k][1] * inv, h[k][2] * inv, h[k][3] * inv),
          f32x4_to_e4m3(h[k][4] * inv, h[k][5] * inv, h[k][6] * inv, h[k][7] * inv));
      if ((c & 15) == 0) scale[row * nb + (c >> 4)] = s;
    }
  }
}

// ------------------------------------------------------------ weight quantisation
// One CTA per block of 128 codes x 128 columns, kept in registers between its
// maximum and its rounding: 16 threads per row, 16 rows per pass, 8 passes.
// Bound by the 3 bytes per element it moves (8192 x 2048: 11.3 us, 68% of the copy
// bandwidth, the same in seconds of calls: each CTA reads once and writes once, and 1024
// of them are one wave whose start and end count); a small weight (500 x 1040) by its
// 2 us of latency.
constexpr int kQuantThreads = 256;

__global__ void __launch_bounds__(kQuantThreads)
    quantize_kernel(const uint4* w, int V, int d, uint2* __restrict__ q,
                    float* __restrict__ scale) {
  __shared__ float part[kQuantThreads / 32];
  wait_prior();
  release_next();
  const int nb = (d + kBlock - 1) / kBlock;
  const int bc = blockIdx.x, br = blockIdx.y;
  const int chunks = d >> 3;
  const int c = bc * 16 + (threadIdx.x & 15);
  const int row0 = br * kBlock + (threadIdx.x >> 4);
  uint4 v[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int row = row0 + p * 16;
    v[p] = make_uint4(0u, 0u, 0u, 0u);
    if (row < V && c < chunks) v[p] = w[static_cast<int64_t>(row) * chunks + c];
  }
  float amax = 0.f;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    float f[8];
    unpack8(v[p], f);
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(f[e]));
  }
  amax = warp_max(amax);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQuantThreads / 32; ++i) amax = fmaxf(amax, part[i]);
  float inv;
  const float s = block_scale(amax, inv);
  if (threadIdx.x == 0) scale[static_cast<int64_t>(br) * nb + bc] = s;
#pragma unroll
  for (int p = 0; p < 8; ++p) {
    const int row = row0 + p * 16;
    float f[8];
    unpack8(v[p], f);
    if (row < V && c < chunks)
      q[static_cast<int64_t>(row) * chunks + c] =
          make_uint2(f32x4_to_e4m3(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv),
                     f32x4_to_e4m3(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv));
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int T, int K>
cudaError_t launch_rmsnorm(const void* x, const void* residual, const void* weight, float eps,
                           int M, int d, void* residual_out, void* q, float* scale,
                           cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(T == 32 ? (static_cast<int64_t>(M) + 3) / 4 : M));
  return launch_dependent(rmsnorm_kernel<T, K>, grid, T == 32 ? 128 : T, 0, 1, s,
                          static_cast<const uint4*>(x), static_cast<const uint4*>(residual),
                          static_cast<const uint4*>(weight), eps, M, d,
                          static_cast<uint4*>(residual_out), static_cast<uint2*>(q), scale);
}

}  // namespace
}  // namespace sidbeam

using namespace sidbeam;

extern "C" int residual_rmsnorm_fp8(const void* x, const void* residual, const void* weight,
                                    float eps, int M, int d, void* residual_out, void* hidden_q,
                                    float* hidden_scale, void* stream) {
  if (M < 0 || d < 16 || d > SIDBEAM_MAX_HIDDEN || (d & 15) != 0)
    return set_error(SIDBEAM_ERR_INVALID_ARG,
                     "residual_rmsnorm_fp8: M=%d, d=%d (a multiple of 16, at most %d)", M, d,
                     SIDBEAM_MAX_HIDDEN);
  if (!(eps >= 0.f) || eps > 3.0e38f)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "residual_rmsnorm_fp8: eps must be finite, >= 0");
  if (M == 0) return SIDBEAM_OK;
  if (!x || !weight || !hidden_q || !hidden_scale)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "residual_rmsnorm_fp8: NULL pointer argument");
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) ||
      !aligned16(hidden_q) || (reinterpret_cast<uintptr_t>(hidden_scale) & 3u) != 0)
    return set_error(SIDBEAM_ERR_ALIGNMENT, "residual_rmsnorm_fp8: pointers must be 16-byte aligned");
  const int chunks = d / 8;  // T * K of them at most
  const auto launch = chunks <= 32        ? launch_rmsnorm<32, 1>
                      : chunks <= 64      ? launch_rmsnorm<32, 2>
                      : chunks <= 128     ? launch_rmsnorm<128, 1>
                      : chunks <= 128 * 2 ? launch_rmsnorm<128, 2>
                      : chunks <= 128 * 4 ? launch_rmsnorm<128, 4>
                      : chunks <= 128 * 8 ? launch_rmsnorm<128, 8>
                                          : launch_rmsnorm<256, 8>;
  const cudaError_t e = launch(x, residual, weight, eps, M, d, residual_out, hidden_q,
                               hidden_scale, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SIDBEAM_OK : cuda_error(e, "residual_rmsnorm_fp8: launch");
}

extern "C" int lmhead_quantize_fp8(const void* w_sid, int V, int d, void* w_q, float* w_scale,
                                   void* stream) {
  if (!w_sid || !w_q || !w_scale)
    return set_error(SIDBEAM_ERR_INVALID_ARG, "lmhead_quantize_fp8: NULL pointer argument");
  if (V < 1 || V > SIDBEAM_MAX_V || d < 16 || d > SIDBEAM_MAX_HIDDEN || (d & 15) != 0)
    return set_error(SIDBEAM_ERR_INVALID_ARG,
                     "lmhead_quantize_fp8: V=%d, d=%d (a multiple of 16, at most %d)", V, d,
                     SIDBEAM_MAX_HIDDEN);
  if (!aligned16(w_sid) || !aligned16(w_q) || (reinterpret_cast<uintptr_t>(w_scale) & 3u) != 0)
    return set_error(SIDBEAM_ERR_ALIGNMENT, "lmhead_quantize_fp8: pointers must be 16-byte aligned");
  const dim3 grid(static_cast<unsigned>((d + kBlock - 1) / kBlock),
                  static_cast<unsigned>((V + kBlock - 1) / kBlock));
  const cudaError_t e = launch_dependent(
      quantize_kernel, grid, kQuantThreads, 0, 1, static_cast<cudaStream_t>(stream),
      static_cast<const uint4*>(w_sid), V, d, static_cast<uint2*>(w_q), w_scale);
  return e == cudaSuccess ? SIDBEAM_OK : cuda_error(e, "lmhead_quantize_fp8: launch");
}
