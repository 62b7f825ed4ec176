// Attention of one new token per request over its cached rows
// (ae_token_attention).
//
// Every cached row is read once for the whole group of query heads: S = Q K^T
// and O += P V run on m16n8k16 tensor-core tiles whose 16 rows are the group's
// heads (mma.sync: a token has at most 16 rows, far below a tcgen05 tile, and
// the bytes of K and V bound the operator; at 23 bytes per clock and SM the
// tiles need under a fifth of the mma.sync rate).
// One warp works alone on tiles of 16 keys: it copies its K and V rows
// (cp.async, 16-byte pieces XORed by row so that ldmatrix reads are free of
// bank conflicts) into a ring of its own, so no barrier sits between the
// copies and the math; masked rows and rows past the end are zero-filled, not
// read.  Four warps of a CTA interleave their tiles over the CTA's key range.
// The key range of a request is split over the CTAs of a cluster, which merge
// their (m, l, O) through distributed shared memory: one launch, no workspace,
// sums in rank order.  The ranges follow the lengths on the device, whatever
// the lengths of the capture were.
#include <math.h>

#include "ae_internal.h"
#include "ae_tc.cuh"

namespace ae {
namespace {

using namespace tc;

constexpr int kWarps = 4;
constexpr int kKeys = 16;      // keys of a warp's tile
constexpr float kRaise = 8.f;  // log2: raise the exponent reference past this

template <int DH>
struct Cfg {
  static constexpr int STAGES = DH == 64 ? 4 : 3;
  static constexpr int TILE = kKeys * DH * 2;         // bytes of a K (or V) tile
  static constexpr int RING = kWarps * STAGES * 2 * TILE;
  static constexpr int PART = kWarps * 16 * DH * 4;   // fp32 partials, over the ring
  static constexpr int ML = RING > PART ? RING : PART;  // [kWarps][16] (m, l), then [16] of the CTA
  static constexpr int BYTES = ML + (kWarps + 1) * 16 * 8;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// d += a b: a 16 x 16 (row), b 16 x 8 (col)
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// H16: the tile's heads fill more than 8 rows (else rows 8..15 are zero and
// neither held nor stored).
template <int DH, bool H16>
__global__ void __launch_bounds__(kWarps * 32) k_token_attn(const __grid_constant__ TokenAttnArgs a, int split, int hc,
                                                            int gc) {
  using C = Cfg<DH>;
  constexpr int ST = C::STAGES, KS = DH / 16, NT = DH / 8;
  constexpr int R = H16 ? 2 : 1;  // 8-row halves held
  extern __shared__ __align__(1024) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % split;
  int u = blockIdx.x / split;
  const int G = a.Hq / a.Hkv;
  const int h = u % (a.Hkv * hc), b = u / (a.Hkv * hc);
  const int kvh = h / hc, g0 = (h - kvh * hc) * gc;

  int64_t r0 = a.kv_row0[b], len = a.kv_len[b];
  if (r0 < 0 || len < 0 || len > a.max_len || r0 > a.cache_rows || len > a.cache_rows - r0) {
    report(a.status, kDevBounds);
    if (r0 < 0) {
      len += r0;
      r0 = 0;
    }
    len = min(len, (int64_t)a.max_len);
    len = max(min(len, a.cache_rows - r0), (int64_t)0);
  }
  // this CTA's keys [lo, hi), whole tiles except the last
  const int n_all = (int)((len + kKeys - 1) / kKeys);
  const int t_lo = (int)((int64_t)n_all * rank / split), t_hi = (int)((int64_t)n_all * (rank + 1) / split);
  const int n = t_hi - t_lo > warp ? (t_hi - t_lo - warp + kWarps - 1) / kWarps : 0;  // tiles of this warp
  const uint8_t* mask = a.key_mask ? a.key_mask + r0 : nullptr;
  const bf16* kb = a.k + r0 * a.kv_stride + (int64_t)kvh * DH;
  const bf16* vb = a.v + r0 * a.kv_stride + (int64_t)kvh * DH;

  // Q fragments: rows lane / 4 (+ 8), dims 16 ks + 2 (lane % 4) + {0, 1} (+ 8)
  uint32_t q[KS][2 * R];
  {
    const int hr = lane >> 2;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int g = g0 + hr + 8 * i;
      const bool on = hr + 8 * i < gc && g < G;
      const bf16* qr = a.q + (int64_t)b * a.q_stride + (int64_t)(kvh * G + (on ? g : 0)) * DH + 2 * (lane & 3);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        q[ks][i] = on ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks) : 0u;
        q[ks][R + i] = on ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8) : 0u;
      }
    }
  }

  uint8_t* ring = smem + warp * (ST * 2 * C::TILE);
  const uint32_t ring_u = smem_u32(ring);
  // valid keys of the warp's j-th tile (bit = key), from its mask byte held by lanes 0..15
  auto tile_key0 = [&](int j) { return (t_lo + warp + j * kWarps) * kKeys; };
  auto mask_byte = [&](int j) -> uint32_t {
    const int key = tile_key0(j) + lane;
    return mask != nullptr && j < n && lane < kKeys && key < len ? mask[key] : 0u;
  };
  auto bits_of = [&](int j, uint32_t byte) -> uint32_t {
    if (j >= n) return 0u;
    if (mask != nullptr) return __ballot_sync(0xffffffffu, byte != 0);
    const int left = (int)len - tile_key0(j);
    return left >= kKeys ? 0xffffu : (1u << left) - 1u;
  };
  auto issue = [&](int j, uint32_t bits) {
    if (j < n) {
      constexpr int CPR = DH / 8;      // 16-byte pieces of a row
      uint8_t* ks = ring + (j % ST) * 2 * C::TILE;
      const int64_t row0 = tile_key0(j);
#pragma unroll
      for (int e = 0; e < kKeys * CPR / 32; ++e) {
        const int i = lane + 32 * e, r = i / CPR, ch = i % CPR;
        const bool on = (bits >> r) & 1u;
        const int64_t off = on ? (row0 + r) * a.kv_stride + ch * 8 : 0;
        // pieces XORed by row within each 128-byte group
        uint8_t* dst = ks + r * (DH * 2) + ((ch ^ (r & 7)) << 4);
        cp_async16(dst, on ? kb + off : (const bf16*)a.q, on ? 16u : 0u);
        cp_async16(dst + C::TILE, on ? vb + off : (const bf16*)a.q, on ? 16u : 0u);
      }
    }
    cp_async_commit();
  };

  float o[NT][2 * R];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 2 * R; ++j) o[i][j] = 0.f;
  float m[R], l[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  const float c = a.scale * 1.4426950408889634f;

  uint64_t inflight = 0;  // 16 bits a tile, the oldest in the low bits
  int queued = 0;
  uint32_t byte = mask_byte(0);
#pragma unroll
  for (int j = 0; j < ST - 1; ++j) {
    const uint32_t bits = bits_of(j, byte);
    byte = mask_byte(j + 1);
    issue(j, bits);
    inflight |= (uint64_t)bits << (16 * queued++);
  }
  for (int j = 0; j < n; ++j) {
    {
      const uint32_t bits = bits_of(j + ST - 1, byte);
      byte = mask_byte(j + ST);
      issue(j + ST - 1, bits);
      inflight |= (uint64_t)bits << (16 * (ST - 1));
    }
    const uint32_t bits = (uint32_t)inflight & 0xffffu;
    inflight >>= 16;
    cp_async_wait<ST - 1>();
    __syncwarp();
    const uint32_t ks_u = ring_u + (j % ST) * 2 * C::TILE, vs_u = ks_u + C::TILE;

    // S = Q K^T: two 8-key tiles
    float s[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[t][i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      // matrices: keys 0..7 dims lo, hi; keys 8..15 dims lo, hi of this 16-dim step
      uint32_t kf[4];
      const int r = (lane & 7) + ((lane >> 4) << 3), ch = 2 * ks + ((lane >> 3) & 1);
      ldsm4(ks_u + r * (DH * 2) + ((ch ^ (r & 7)) << 4), kf);
      mma16(s[0], q[ks][0], H16 ? q[ks][R - 1] : 0u, q[ks][R], H16 ? q[ks][2 * R - 1] : 0u, kf[0], kf[1]);
      mma16(s[1], q[ks][0], H16 ? q[ks][R - 1] : 0u, q[ks][R], H16 ? q[ks][2 * R - 1] : 0u, kf[2], kf[3]);
    }
    // mask, running maximum (rows are shared by four lanes)
    float factor[R];
    bool raise = false;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = 8 * t + 2 * (lane & 3) + e;
          float& x = s[t][2 * i + e];
          x = ((bits >> key) & 1u) ? x * c : -INFINITY;
          top = fmaxf(top, x);
        }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      factor[i] = 1.f;
      if (top > m[i] + kRaise) {
        factor[i] = ex2_fast(m[i] - top);
        m[i] = top;
        raise = true;
      }
    }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        l[i] *= factor[i];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          o[t][2 * i] *= factor[i];
          o[t][2 * i + 1] *= factor[i];
        }
      }
    }
    uint32_t p[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float base = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float x = ex2_fast(s[t][2 * i] - base), y = ex2_fast(s[t][2 * i + 1] - base);
        l[i] += x + y;
        p[2 * t + i] = bf16x2(x, y);
      }
    }
    // O += P V: V rows read transposed, two 8-dim tiles a load
#pragma unroll
    for (int t = 0; t < NT; t += 2) {
      uint32_t vf[4];
      const int r = (lane & 7) + (((lane >> 3) & 1) << 3), ch = t + (lane >> 4);
      ldsm4_t(vs_u + r * (DH * 2) + ((ch ^ (r & 7)) << 4), vf);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float d[4] = {o[t + e][0], o[t + e][1], H16 ? o[t + e][2 * R - 2] : 0.f, H16 ? o[t + e][2 * R - 1] : 0.f};
        mma16(d, p[0], p[1], p[2], p[3], vf[2 * e], vf[2 * e + 1]);
        o[t + e][0] = d[0];
        o[t + e][1] = d[1];
        if (H16) {
          o[t + e][2 * R - 2] = d[2];
          o[t + e][2 * R - 1] = d[3];
        }
      }
    }
    __syncwarp();  // the stage is overwritten next
  }
  cp_async_wait<0>();
  __syncthreads();

  // ---- merge the warps, then the cluster
  float2* ml = reinterpret_cast<float2*>(smem + C::ML);  // [kWarps][16], then [16]
  float* part = reinterpret_cast<float*>(smem);          // [kWarps][8 R][DH]
  constexpr int ROWS = 8 * R;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
    l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    const int r = (lane >> 2) + 8 * i;
    if ((lane & 3) == 0) ml[warp * 16 + r] = make_float2(m[i], l[i]);
    float* pr = part + (warp * ROWS + r) * DH + 2 * (lane & 3);
#pragma unroll
    for (int t = 0; t < NT; ++t) *reinterpret_cast<float2*>(pr + 8 * t) = make_float2(o[t][2 * i], o[t][2 * i + 1]);
  }
  __syncthreads();
  constexpr int PER = DH / 4;
  auto store = [&](int r, int p4, float l_sum, const float4& v) {
    if (r >= gc || g0 + r >= G) return;
    const float inv = l_sum > 0.f ? 1.f / l_sum : 0.f;
    *reinterpret_cast<uint2*>(a.out + (int64_t)b * a.out_stride + (int64_t)(kvh * G + g0 + r) * DH + 4 * p4) =
        make_uint2(bf16x2(v.x * inv, v.y * inv), bf16x2(v.z * inv, v.w * inv));
  };
  for (int i = threadIdx.x; i < ROWS * PER; i += kWarps * 32) {
    const int r = i / PER, p4 = i % PER;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, ml[w * 16 + r].x);
    float l_sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 x = ml[w * 16 + r];
      const float f = x.x == -INFINITY ? 0.f : ex2_fast(x.x - top);
      const float4 y = *reinterpret_cast<const float4*>(part + (w * ROWS + r) * DH + 4 * p4);
      l_sum += f * x.y;
      v.x += f * y.x;
      v.y += f * y.y;
      v.z += f * y.z;
      v.w += f * y.w;
    }
    if (split == 1) {
      store(r, p4, l_sum, v);
    } else {
      *reinterpret_cast<float4*>(part + r * DH + 4 * p4) = v;  // over warp 0's, read by this thread alone
      if (p4 == 0) ml[kWarps * 16 + r] = make_float2(top, l_sum);
    }
  }
  if (split > 1) {
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    const uint32_t part_u = smem_u32(part), ml_u = smem_u32(ml + kWarps * 16);
    for (int i = rank * kWarps * 32 + threadIdx.x; i < ROWS * PER; i += split * kWarps * 32) {
      const int r = i / PER, p4 = i % PER;
      float top = -INFINITY;
      for (int k = 0; k < split; ++k) top = fmaxf(top, ld_cluster_f2(mapa(ml_u + r * 8, k)).x);
      float l_sum = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int k = 0; k < split; ++k) {
        const float2 x = ld_cluster_f2(mapa(ml_u + r * 8, k));
        const float4 y = ld_cluster_f4(mapa(part_u + (r * DH + 4 * p4) * 4, k));
        const float f = x.x == -INFINITY ? 0.f : ex2_fast(x.x - top);
        l_sum += f * x.y;
        v.x += f * y.x;
        v.y += f * y.y;
        v.z += f * y.z;
        v.w += f * y.w;
      }
      store(r, p4, l_sum, v);
    }
    __syncthreads();
    cluster_arrive();  // no CTA leaves while a peer reads its partials
    cluster_wait();
  }
}

template <int DH, bool H16>
cudaError_t launch(const TokenAttnArgs& a, int gc, int hc, int split, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.batch * a.Hkv * hc * split));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = Cfg<DH>::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_token_attn<DH, H16>, a, split, hc, gc);
}

template <int DH, bool H16>
cudaError_t setup() {
  return cudaFuncSetAttribute(k_token_attn<DH, H16>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<DH>::BYTES);
}

}  // namespace

cudaError_t launch_token_attention(const TokenAttnArgs& a, int dh, int sm_count, cudaStream_t s) {
  // heads of a group in chunks of at most 16 rows
  const int G = a.Hq / a.Hkv, hc = (G + 15) / 16, gc = (G + hc - 1) / hc;
  const int64_t units = (int64_t)a.batch * a.Hkv * hc;
  if (units > 0x7fffffff / 8) return cudaErrorInvalidConfiguration;
  // split the keys while CTAs are fewer than two a SM and keep a tile for every warp
  int split = 1;
  while (split < 8 && units * split < 2 * sm_count && a.max_len > split * kWarps * kKeys) split *= 2;
  const bool wide = gc > 8;
  if (dh == 64) return wide ? launch<64, true>(a, gc, hc, split, s) : launch<64, false>(a, gc, hc, split, s);
  if (dh == 128) return wide ? launch<128, true>(a, gc, hc, split, s) : launch<128, false>(a, gc, hc, split, s);
  return wide ? launch<256, true>(a, gc, hc, split, s) : launch<256, false>(a, gc, hc, split, s);
}

cudaError_t token_kernel_setup() {
  cudaError_t e = setup<64, false>();
  if (e == cudaSuccess) e = setup<64, true>();
  if (e == cudaSuccess) e = setup<128, false>();
  if (e == cudaSuccess) e = setup<128, true>();
  if (e == cudaSuccess) e = setup<256, false>();
  if (e == cudaSuccess) e = setup<256, true>();
  return e;
}

}  // namespace ae
