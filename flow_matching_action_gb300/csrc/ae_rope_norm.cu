// Per-head RMS norm of queries and keys, rotary positions and the K/V cache
// write in one pass over the merged projection (ae_qk_norm_rope).
//
// DH / 16 lanes hold one head: lane l has dims 8l .. 8l+7 and their rotation
// partners DH/2 + 8l .. +7 (two 16-byte loads, every pair within a thread), so
// a head's sum of squares is one shuffle reduction over its lanes and nothing
// is exchanged for the rotation.  A warp works alone on a token (or on a part of
// its heads when tokens are few): its lanes compute the token's cosines and
// sines once, share them through the warp's slice of shared memory, and stream
// the heads with the loads two steps ahead; no barrier between warps.
// An angle is positions * frequency modulo one turn: the frequency as a 64-bit
// fraction of a turn times the integer position wraps modulo 2^64, which is
// the reduction, for every int32 position.  Its top 32 bits (cut by less than
// 2^-32 turns) become an fp32 part of half a turn: at most 2^-26 turns off.
// Bound by the bytes of the rows, read once and written once: 32768 tokens
// 32/8/128 with norms and scattered rows 136 us, 5.9 TB/s (89% of a plain copy);
// 5003 tokens 12/4/64 without norms 6.5 us, 3.9 TB/s (a launch and one short wave);
// 12 tokens 8/1/256 2.5 to 4 us, a launch.  (A block a token with the angles behind
// barriers took 149.5, 10.2 and 10.4 us.)
// Arithmetic is fp32; a result is rounded once, to the bf16 of the caches.
#include "ae_internal.h"
#include "ae_tc.cuh"

namespace ae {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocks = 3;  // resident a SM

// Two fp32 lanes of one 64-bit register (packed multiply-adds).
typedef uint64_t f2;
__device__ __forceinline__ f2 pair(float a, float b) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(f2 v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Eight bf16 as four pairs of fp32.
__device__ __forceinline__ void unpack8(const uint4& u, f2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

__device__ __forceinline__ uint4 pack8(const f2 (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    split(x[i], a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Eight fp32 of shared memory as four pairs.
__device__ __forceinline__ void load8(const float* p, f2 (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 v = reinterpret_cast<const float4*>(p)[i];
    x[2 * i] = pair(v.x, v.y);
    x[2 * i + 1] = pair(v.z, v.w);
  }
}

template <int DH>
__global__ void __launch_bounds__(kThreads, kBlocks)
    k_qk_norm_rope(const __grid_constant__ RopeNormArgs a, int parts) {
  constexpr int HALF = DH / 2;
  constexpr int LPH = DH / 16;       // lanes of a head
  constexpr int HPW = 32 / LPH;      // heads a warp works on at once
  constexpr int PAIRS = HALF / 32;   // rotation pairs whose angles a lane computes
  __shared__ __align__(16) float trig_all[kThreads / 32][3][HALF];  // cos, sin, -sin of the warp's token
  __shared__ __align__(16) float norm_w[2][DH];                     // norm_offset + w of queries, keys
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPH, l = lane % LPH;
  const int heads = a.Hq + 2 * a.Hkv, n_rot = a.Hq + a.Hkv;
  float(*trig)[HALF] = trig_all[warp];
  const int items = a.tokens * parts, stride = gridDim.x * (kThreads / 32);
  int item = blockIdx.x * (kThreads / 32) + warp;

  auto fetch = [&](int t, int h, uint4& lo, uint4& hi) {
    if (h >= heads) return;
    const bf16* src = a.qkv + (int64_t)t * a.qkv_stride + (int64_t)h * DH + 8 * l;
    lo = *reinterpret_cast<const uint4*>(src);
    hi = *reinterpret_cast<const uint4*>(src + HALF);
  };
  int t = item / parts, h0 = (item - t * parts) * HPW;
  uint4 lo1 = make_uint4(0, 0, 0, 0), hi1 = lo1;  // the next step's pieces
  if (item < items) fetch(t, h0 + sub, lo1, hi1);

  // the lane's pairs, the same for every token: read once (the argument's
  // entries are constants, which lanes at different addresses read one by one)
  uint64_t turn[PAIRS];
  int axis[PAIRS], pos[PAIRS];
  int64_t row = 0;
#pragma unroll
  for (int i = 0; i < PAIRS; ++i) {
    turn[i] = a.turn_table ? a.turn_table[lane + 32 * i] : a.turn[lane + 32 * i];
    axis[i] = a.n_axes > 1 ? a.axis[lane + 32 * i] : 0;
    pos[i] = item < items ? a.positions[(int64_t)axis[i] * a.tokens + t] : 0;
  }
  if (item < items) row = a.kv_rows ? a.kv_rows[t] : t;
  if (a.q_norm != nullptr || a.k_norm != nullptr)
    for (int i = threadIdx.x; i < DH; i += kThreads) {
      norm_w[0][i] = a.q_norm ? a.norm_offset + __bfloat162float(a.q_norm[i]) : 0.f;
      norm_w[1][i] = a.k_norm ? a.norm_offset + __bfloat162float(a.k_norm[i]) : 0.f;
    }
  __syncthreads();

  while (item < items) {  // uniform for the warp
    __syncwarp();
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      const int32_t frac = (int32_t)(uint32_t)(((uint64_t)(int64_t)pos[i] * turn[i]) >> 32);  // in [-1/2, 1/2) turns
      float sn, cn;
      sincospif((float)frac * 4.656612873077393e-10f, &sn, &cn);  // 2^-31: half turns
      trig[0][lane + 32 * i] = cn;
      trig[1][lane + 32 * i] = sn;
      trig[2][lane + 32 * i] = -sn;
    }
    __syncwarp();
    const int64_t tok = t, dst_row = row;
    item += stride;
    const int t1 = item / parts, h1 = (item - t1 * parts) * HPW;
    if (item < items) {  // the next token's positions and cache row
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) pos[i] = a.positions[(int64_t)axis[i] * a.tokens + t1];
      row = a.kv_rows ? a.kv_rows[t1] : t1;
    }
    bf16* q_row = a.q_out + tok * a.q_stride + 8 * l;
    const bool store_kv = dst_row >= 0 && dst_row < a.cache_rows;
    if (dst_row >= a.cache_rows) tc::report(a.status, kDevBounds);
    for (; h0 < heads; h0 += parts * HPW) {
      uint4 lo = lo1, hi = hi1;
      const int hn = h0 + parts * HPW;
      if (hn < heads) fetch((int)tok, hn + sub, lo1, hi1);
      else if (item < items) fetch(t1, h1 + sub, lo1, hi1);
      const int h = h0 + sub;
      f2 x[4], y[4];
      unpack8(lo, x);
      unpack8(hi, y);
      if (h0 < n_rot) {  // a step of values only skips the arithmetic
        f2 s2 = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) s2 = fma2(y[i], y[i], fma2(x[i], x[i], s2));
        float ss, se;
        split(s2, ss, se);
        ss += se;
#pragma unroll
        for (int o = LPH / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (h < n_rot) {
          const bool is_k = h >= a.Hq;
          if ((is_k ? a.k_norm : a.q_norm) != nullptr) {
            const float r = rsqrtf(ss * (1.f / DH) + a.eps);
            const f2 r2 = pair(r, r);
            f2 wl[4], wh[4];
            load8(norm_w[is_k] + 8 * l, wl);
            load8(norm_w[is_k] + HALF + 8 * l, wh);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = mul2(x[i], mul2(r2, wl[i]));
              y[i] = mul2(y[i], mul2(r2, wh[i]));
            }
          }
          f2 c[4], sn[4], ns[4];
          load8(trig[0] + 8 * l, c);
          load8(trig[1] + 8 * l, sn);
          load8(trig[2] + 8 * l, ns);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f2 p = fma2(y[i], ns[i], mul2(x[i], c[i]));
            y[i] = fma2(x[i], sn[i], mul2(y[i], c[i]));
            x[i] = p;
          }
          lo = pack8(x);
          hi = pack8(y);
        }
      }
      bf16* dst = nullptr;
      if (h < a.Hq) dst = q_row + (int64_t)h * DH;
      else if (h < heads && store_kv)
        dst = (h < n_rot ? a.k_cache + (int64_t)(h - a.Hq) * DH : a.v_cache + (int64_t)(h - n_rot) * DH) +
              dst_row * a.kv_stride + 8 * l;
      if (dst != nullptr) {
        *reinterpret_cast<uint4*>(dst) = lo;
        *reinterpret_cast<uint4*>(dst + HALF) = hi;
      }
    }
    t = t1;
    h0 = h1;
  }
}

template <int DH>
cudaError_t launch(const RopeNormArgs& a, int sm_count, cudaStream_t s) {
  constexpr int HPW = 512 / DH, W = kThreads / 32;
  // tokens that do not fill the GPU's warps are split by heads
  const int warps = kBlocks * W * sm_count, steps = (a.Hq + 2 * a.Hkv + HPW - 1) / HPW;
  int parts = warps / a.tokens;
  parts = parts < 1 ? 1 : (parts > steps ? steps : parts);
  const int64_t blocks = ((int64_t)a.tokens * parts + W - 1) / W;
  const unsigned grid = (unsigned)(blocks < kBlocks * sm_count ? blocks : kBlocks * sm_count);
  return launch_k(k_qk_norm_rope<DH>, dim3(grid), dim3(kThreads), 0, s, false, a, parts);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeNormArgs& a, int dh, int sm_count, cudaStream_t s) {
  if (dh == 64) return launch<64>(a, sm_count, s);
  if (dh == 128) return launch<128>(a, sm_count, s);
  return launch<256>(a, sm_count, s);
}

}  // namespace ae
