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

// One warp per (row, head); lane l holds elements l * D/32 .. of q, k, v, o.
template <int D>
__global__ void __launch_bounds__(128) attention_kernel(const AttnArgs a) {
  constexpr int E = D / 32;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t row = w / a.H;
  if (row >= static_cast<int64_t>(a.R) * a.B) return;
  const int h = static_cast<int>(w - row * a.H);
  const int g = h / (a.H / a.Hkv);
  const int r = static_cast<int>(row / a.B), b = static_cast<int>(row - static_cast<int64_t>(r) * a.B);
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(a.q[row * a.q_stride + h * D + lane * E + e]) * a.scale_log2;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  auto add = [&](const __nv_bfloat16* k, const __nv_bfloat16* v) {
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) x = fmaf(q[e], __bfloat162float(k[lane * E + e]), x);
    x = warp_sum(x);
    const float mn = fmaxf(m, x);
    const float f = exp2f(m - mn), p = exp2f(x - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * __bfloat162float(v[lane * E + e]);
    m = mn;
  };
  const int64_t cap = a.table ? static_cast<int64_t>(a.table_stride) * a.page_size : a.page_size;
  int64_t len = a.len[r];
  if (len < 0 || len > cap) {
    if (lane == 0) atomicOr(a.status, kStatusBadCache);
    len = len < 0 ? 0 : cap;
  }
  bool dead = false;
  int slot = b;
  for (int u = a.level - 1; u >= 0; --u) {
    const int64_t at = (static_cast<int64_t>(u) * a.R + r) * a.B + slot;
    const int p = a.bp[at];
    if (p < 0 || (u > 0 && p >= a.B)) {
      dead = true;
      break;
    }
    slot = p;
  }
  if (!dead) {
    slot = b;
    for (int u = a.level - 1; u >= 0; --u) {
      const int64_t at = (static_cast<int64_t>(u) * a.R + r) * a.B + slot;
      add(a.kb + (at * a.Hkv + g) * D, a.vb + (at * a.Hkv + g) * D);
      slot = a.bp[at];
    }
    for (int64_t i = 0; i < len; ++i) {
      int64_t page = r, t = i;
      if (a.table) {
        page = a.table[static_cast<int64_t>(r) * a.table_stride + i / a.page_size];
        t = i % a.page_size;
        if (page < 0 || page >= a.n_pages) {
          if (lane == 0) atomicOr(a.status, kStatusBadCache);
          const float mn = fmaxf(m, 0.f), f = exp2f(m - mn);
          l = l * f + exp2f(-mn);
          for (int e = 0; e < E; ++e) o[e] *= f;
          m = mn;
          continue;
        }
      }
      const int64_t at = page * a.page_stride + t * a.token_stride + g * D;
      add(a.k + at, a.v + at);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    a.out[row * a.out_stride + h * D + lane * E + e] = __float2bfloat16(o[e] * inv);
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
  const int64_t warps = static_cast<int64_t>(R) * B * H;
  const unsigned grid = static_cast<unsigned>((warps + 3) / 4);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (D == 64)
    attention_kernel<64><<<grid, 128, 0, s>>>(a);
  else
    attention_kernel<128><<<grid, 128, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SIDBEAM_OK : cuda_error(e, "beam_attention: launch");
}
