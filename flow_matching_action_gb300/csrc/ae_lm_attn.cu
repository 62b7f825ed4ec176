// Attention of single tokens, first form: one warp per
// (query row, head) walks the row's keys with a running maximum and sum; a
// lane holds DH / 32 consecutive dims of q, k, v and o.
#include <math.h>

#include "ae_internal.h"
#include "ae_tc.cuh"

namespace ae {
namespace {

template <int E>
__device__ __forceinline__ void load_row(const bf16* p, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = __bfloat162float(p[i]);
}

template <int DH>
__device__ void attend_row(const bf16* q, const bf16* k, const bf16* v, int64_t kv_stride, const uint8_t* mask,
                           int n_keys, float scale, bf16* out) {
  constexpr int E = DH / 32;
  const int lane = threadIdx.x & 31;
  float qr[E], o[E], x[E];
  load_row<E>(q + lane * E, qr);
#pragma unroll
  for (int i = 0; i < E; ++i) o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < n_keys; ++j) {
    if (mask != nullptr && mask[j] == 0) continue;
    load_row<E>(k + (int64_t)j * kv_stride + lane * E, x);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) s += qr[i] * x[i];
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= scale;
    const float mn = fmaxf(m, s);
    const float f = m == -INFINITY ? 0.f : __expf(m - mn), p = __expf(s - mn);
    m = mn;
    l = l * f + p;
    load_row<E>(v + (int64_t)j * kv_stride + lane * E, x);
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = o[i] * f + p * x[i];
  }
  const float r = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) out[lane * E + i] = __float2bfloat16(o[i] * r);
}

template <int DH>
__global__ void k_token_rows(const __grid_constant__ TokenAttnArgs a) {
  const int b = blockIdx.x, h = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (h >= a.Hq) return;
  int64_t r0 = a.kv_row0[b], n = a.kv_len[b];
  if (r0 < 0 || n < 0 || n > a.max_len || r0 > a.cache_rows || n > a.cache_rows - r0) {
    tc::report(a.status, kDevBounds);
    if (r0 < 0) {
      n += r0;
      r0 = 0;
    }
    n = min(n, (int64_t)a.max_len);
    n = max(min(n, a.cache_rows - r0), (int64_t)0);
  }
  const int64_t col = (int64_t)(h / (a.Hq / a.Hkv)) * DH;
  attend_row<DH>(a.q + b * a.q_stride + (int64_t)h * DH, a.k + r0 * a.kv_stride + col, a.v + r0 * a.kv_stride + col,
                 a.kv_stride, a.key_mask ? a.key_mask + r0 : nullptr, (int)n, a.scale,
                 a.out + b * a.out_stride + (int64_t)h * DH);
}

}  // namespace

cudaError_t launch_token_attention(const TokenAttnArgs& a, int dh, int sm_count, cudaStream_t s) {
  (void)sm_count;
  const dim3 grid(a.batch, (a.Hq + 3) / 4);
  if (dh == 64) return launch_k(k_token_rows<64>, grid, dim3(128), 0, s, false, a);
  if (dh == 128) return launch_k(k_token_rows<128>, grid, dim3(128), 0, s, false, a);
  return launch_k(k_token_rows<256>, grid, dim3(128), 0, s, false, a);
}

cudaError_t lm_kernel_setup() { return prompt_kernel_setup(); }

}  // namespace ae
