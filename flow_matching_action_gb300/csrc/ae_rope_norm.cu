// Per-head RMS norm of queries and keys, rotary positions and the K/V cache
// write in one pass over the merged projection (ae_qk_norm_rope).
//
// DH / 16 lanes hold one head: lane l has dims 8l .. 8l+7 and their rotation
// partners DH/2 + 8l .. +7 (two 16-byte loads, every pair within a thread), so
// a head's sum of squares is one shuffle reduction over its lanes and nothing
// is exchanged for the rotation.  The angle's cosine and sine are computed once
// per (token, pair) of the block and shared by the token's heads through
// shared memory.
// An angle is positions * frequency modulo one turn: the frequency as a 64-bit
// fraction of a turn times the integer position wraps modulo 2^64, which is
// the reduction, exact for every int32 position; its top 32 bits leave an
// error of 2^-33 turns.
#include "ae_internal.h"
#include "ae_tc.cuh"

namespace ae {
namespace {

constexpr int kThreads = 256;

struct Vec8 {
  uint4 u;
};

__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int DH>
__global__ void __launch_bounds__(kThreads) k_qk_norm_rope(const __grid_constant__ RopeNormArgs a, int toks_per_block) {
  constexpr int HALF = DH / 2;
  constexpr int LPH = DH / 16;       // lanes of a head
  constexpr int HPW = 32 / LPH;      // heads a warp works on at once
  extern __shared__ float2 cs[];     // [toks_per_block][HALF] (cos, sin)
  const int tok0 = blockIdx.x * toks_per_block;
  const int ntok = min(toks_per_block, a.tokens - tok0);
  for (int i = threadIdx.x; i < ntok * HALF; i += kThreads) {
    const int t = i / HALF, j = i - t * HALF;
    const int64_t pos = a.positions[(int64_t)a.axis[j] * a.tokens + tok0 + t];
    const int32_t frac = (int32_t)(uint32_t)(((uint64_t)pos * a.turn[j]) >> 32);  // in [-1/2, 1/2) turns
    float s, c;
    sincospif((float)frac * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    cs[i] = make_float2(c, s);
  }
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPH, l = lane % LPH;
  const int heads = a.Hq + 2 * a.Hkv;
  const int units = ntok * heads;
  for (int u0 = warp * HPW; u0 < units; u0 += (kThreads / 32) * HPW) {  // uniform for the warp
    const int u = u0 + sub;
    const bool on = u < units;
    const int t = on ? u / heads : 0, h = on ? u - t * heads : 0;
    const bf16* src = a.qkv + (int64_t)(tok0 + t) * a.qkv_stride + (int64_t)h * DH + 8 * l;
    uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
    if (on) {
      lo = *reinterpret_cast<const uint4*>(src);
      hi = *reinterpret_cast<const uint4*>(src + HALF);
    }
    bf16* dst = nullptr;
    if (on && h < a.Hq) {
      dst = a.q_out + (int64_t)(tok0 + t) * a.q_stride + (int64_t)h * DH;
    } else if (on) {
      const int64_t row = a.kv_rows ? a.kv_rows[tok0 + t] : tok0 + t;
      if (row >= a.cache_rows) {
        tc::report(a.status, kDevBounds);
      } else if (row >= 0) {
        const int kh = h - a.Hq;
        dst = (kh < a.Hkv ? a.k_cache + row * a.kv_stride + (int64_t)kh * DH
                          : a.v_cache + row * a.kv_stride + (int64_t)(kh - a.Hkv) * DH);
      }
    }
    float x[8], y[8];
    unpack8(lo, x);
    unpack8(hi, y);
    const bf16* w = h < a.Hq ? a.q_norm : a.k_norm;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += x[i] * x[i] + y[i] * y[i];
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (h < a.Hq + a.Hkv && on) {
      if (w != nullptr) {
        const float r = rsqrtf(ss * (1.f / DH) + a.eps);
        float wl[8], wh[8];
        unpack8(*reinterpret_cast<const uint4*>(w + 8 * l), wl);
        unpack8(*reinterpret_cast<const uint4*>(w + HALF + 8 * l), wh);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= r * (a.norm_offset + wl[i]);
          y[i] *= r * (a.norm_offset + wh[i]);
        }
      }
      const float2* c = cs + t * HALF + 8 * l;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 z = c[i];
        const float p = x[i] * z.x - y[i] * z.y;
        y[i] = y[i] * z.x + x[i] * z.y;
        x[i] = p;
      }
      lo = pack8(x);
      hi = pack8(y);
    }
    if (dst != nullptr) {
      *reinterpret_cast<uint4*>(dst + 8 * l) = lo;
      *reinterpret_cast<uint4*>(dst + HALF + 8 * l) = hi;
    }
  }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeNormArgs& a, int dh, int sm_count, cudaStream_t s) {
  const int tpb = a.tokens >= 8 * sm_count ? 4 : 1;
  const int grid = (a.tokens + tpb - 1) / tpb;
  const size_t smem = (size_t)tpb * (dh / 2) * sizeof(float2);
  if (dh == 64) return launch_k(k_qk_norm_rope<64>, dim3(grid), dim3(kThreads), smem, s, false, a, tpb);
  if (dh == 128) return launch_k(k_qk_norm_rope<128>, dim3(grid), dim3(kThreads), smem, s, false, a, tpb);
  return launch_k(k_qk_norm_rope<256>, dim3(grid), dim3(kThreads), smem, s, false, a, tpb);
}

}  // namespace ae
