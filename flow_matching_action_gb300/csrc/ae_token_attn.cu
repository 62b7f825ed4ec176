// Attention of one new token per request over its cached rows
// (ae_token_attention).
//
// Every cached row is read once for the whole group of query heads.  The
// transposed products S^T = K Q^T and O^T += V^T P^T put the 16 keys (or 16
// dims) of a tile in the rows of an m16n8k16 tensor-core tile and the heads in
// its eight columns (mma.sync: a token has a few heads, far below a tcgen05
// tile, and the bytes of K and V bound the operator); P^T becomes the second
// product's operand by an 8 x 8 transpose across the warp.
// One warp works alone on tiles of 16 keys: it loads a tile's K and V rows with
// one TMA box each (128-byte swizzle, so that ldmatrix reads are free of bank
// conflicts) into a ring of its own, so no barrier sits between the copies and
// the math.  (Measured on one warp at head_dim 256: issuing a tile takes 130
// clocks this way, 1190 as 32 cp.async a lane, 2060 as one bulk copy a row.)
// Scores of masked rows and of rows past the end become -inf and their V rows
// are zeroed in shared memory, since 0 * NaN would reach every head; a tile
// without valid keys is not read.  Four warps of a CTA interleave their tiles
// over the CTA's key range.
// The key range of a request is split over the CTAs of a cluster.  The warps of
// a CTA merge their (m, l, O), every CTA sends each peer the dims that peer owns
// (remote shared memory), and after one cluster barrier each owner merges its
// dims: one launch, no workspace, sums in a fixed order.  The ranges follow the
// lengths on the device, whatever the lengths of the capture were.
// Bound by the bytes of K and V where requests fill the GPU: 64 of 8k keys
// 32/8/128 290 to 298 us, 7.1 TB/s.  Few or short requests are bound by a launch,
// the first loads, and the two merges: 712 keys 8/1/256 5.6 us; twelve requests of up
// to 2048 keys, a camera slot masked, 7.7 us (1.4 TB/s).  Groups of nine to sixteen
// heads (NB = 2): 64 of 8k keys 16/1/128 44.5 us, 5.9 TB/s.
// Scores, statistics and O are fp32; weights are rounded to bf16 because the
// tensor cores multiply bf16 (an error of at most 2^-8 of each term), O once.
#include <math.h>

#include "ae_internal.h"
#include "ae_tc.cuh"

namespace ae {
namespace {

using namespace tc;

constexpr int kWarps = 4;
constexpr int kKeys = 16;      // keys of a warp's tile
constexpr int kMaxSplit = 8;
constexpr float kRaise = 8.f;  // log2: raise the exponent reference past this

// NB: 8-head column tiles of the group.
template <int DH, int NB>
struct Cfg {
  static constexpr int ST = DH == 64 ? 4 : 3;            // ring stages of a warp
  static constexpr int DB = DH / 64;                     // 64-dim blocks of a row
  static constexpr int TILE = kKeys * DH * 2;            // a K (or V) tile: [DB][16 rows][128 bytes]
  static constexpr int HEADS = 8 * NB;
  static constexpr int RING = kWarps * ST * 2 * TILE;    // then, over it, the warps' [DH][HEADS] fp32 and (m, l)
  static constexpr int WARP_ML = kWarps * DH * HEADS * 4;
  static constexpr int MERGE = RING;                     // [split][DH / split][HEADS] fp32 from the peers
  static constexpr int ML = MERGE + DH * HEADS * 4;      // [split][HEADS] (m, l)
  static constexpr int BARS = ML + kMaxSplit * HEADS * 8;
  static constexpr int BYTES = BARS + kWarps * ST * 8 + 16 + 1024;
  static_assert(WARP_ML + kWarps * HEADS * 8 <= RING, "the warps' partials fit over the ring");
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
  asm(
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
// Transpose of the warp's 8 x 8 matrix of 16-bit elements (row lane / 4, columns 2 (lane % 4), + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void st_cluster_f2(uint32_t addr, float x, float y) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}
__device__ __forceinline__ void st_cluster_f4(uint32_t addr, const float4& v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
// Byte offset of 16-byte piece c of row r in a tile.
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return (uint32_t)((c >> 3) * (kKeys * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

template <int DH, int NB, bool SPLIT>
__global__ void __launch_bounds__(kWarps * 32)
    k_token_attn(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                 const __grid_constant__ TokenAttnArgs a, int split, int hc, int gc) {
  using C = Cfg<DH, NB>;
  constexpr int KS = DH / 16, ST = C::ST, HEADS = C::HEADS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  if (SPLIT) cluster_arrive();            // before the first remote write every CTA must have started
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = blockIdx.x, b = blockIdx.z;
  const int G = a.Hq / a.Hkv;
  const int kvh = hc == 1 ? blockIdx.y : blockIdx.y / hc, g0 = (blockIdx.y - kvh * hc) * gc;
  int64_t r0 = a.kv_row0[b], len = a.kv_len[b];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BARS) + warp * ST;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::BARS + kWarps * ST * 8);
  if (lane == 0) {
    for (int i = 0; i < ST; ++i) mbar_init(&bars[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    if (a.cache_rows > 0) {  // without rows there are no maps
      prefetch_tensormap(&kmap);
      prefetch_tensormap(&vmap);
    }
  }

  // Q as the second operand: heads lane / 4 (+ 8), dims 16 ks + 2 (lane % 4) + {0, 1} (+ 8)
  uint32_t q[KS][NB][2];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int hr = (lane >> 2) + 8 * i;
    const bool on = hr < gc && g0 + hr < G;
    const bf16* qr = a.q + (int64_t)b * a.q_stride + (int64_t)(kvh * G + (on ? g0 + hr : 0)) * DH + 2 * (lane & 3);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[ks][i][0] = on ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks) : 0u;
      q[ks][i][1] = on ? *reinterpret_cast<const uint32_t*>(qr + 16 * ks + 8) : 0u;
    }
  }
  if (r0 < 0 || len < 0 || len > a.max_len || r0 > a.cache_rows || len > a.cache_rows - r0) {
    report(a.status, kDevBounds);
    if (r0 < 0) {
      len += r0;
      r0 = 0;
    }
    len = min(len, (int64_t)a.max_len);
    len = max(min(len, a.cache_rows - r0), (int64_t)0);
  }
  // this CTA's tiles [t_lo, t_hi), every fourth of them this warp's
  const int n_all = (int)((len + kKeys - 1) / kKeys);
  const int t_lo = SPLIT ? (int)((int64_t)n_all * rank / split) : 0;
  const int t_hi = SPLIT ? (int)((int64_t)n_all * (rank + 1) / split) : n_all;
  const int n = t_hi - t_lo > warp ? (t_hi - t_lo - warp + kWarps - 1) / kWarps : 0;
  const int key_first = (t_lo + warp) * kKeys;
  const uint8_t* mask = a.key_mask ? a.key_mask + r0 : nullptr;

  const int row_first = __shfl_sync(0xffffffffu, (int)r0 + key_first, 0);
  uint8_t* ring = smem + warp * (ST * 2 * C::TILE);
  const uint32_t ring_u = smem_u32(ring);
  // valid keys of the warp's j-th tile (bit = key), from its mask byte held by lanes 0..15
  auto mask_byte = [&](int j) -> uint32_t {
    const int key = key_first + j * (kWarps * kKeys) + lane;
    return mask != nullptr && j < n && lane < kKeys && key < len ? mask[key] : 0u;
  };
  auto bits_of = [&](int j, uint32_t byte) -> uint32_t {
    if (j >= n) return 0u;
    if (mask != nullptr) return __ballot_sync(0xffffffffu, byte != 0);
    const int left = (int)len - (key_first + j * (kWarps * kKeys));
    return left >= kKeys ? 0xffffu : (1u << left) - 1u;
  };
  auto issue = [&](int j, uint32_t bits) {
    if (j >= n) return;
    uint64_t* bar = &bars[j % ST];
    uint8_t* dst = ring + (j % ST) * 2 * C::TILE;
    const int row = row_first + j * (kWarps * kKeys), block = kvh * C::DB;
    if (elect_one()) {
      if (bits == 0u) {
        mbar_arrive(bar);
      } else {
        mbar_arrive_expect_tx(bar, 2 * C::TILE);
        tma_load_3d_nohint(dst, &kmap, bar, 0, row, block);
        tma_load_3d_nohint(dst + C::TILE, &vmap, bar, 0, row, block);
      }
    }
    __syncwarp();
  };

  // O^T: dims 16 t + lane / 4 (+ 8), heads 2 (lane % 4) + {0, 1} (+ 8 i)
  float o[KS][NB][4];
#pragma unroll
  for (int t = 0; t < KS; ++t)
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[t][i][e] = 0.f;
  float m[NB][2], l[NB][2];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[i][e] = -INFINITY;
      l[i][e] = 0.f;
    }
  const float c = a.scale * 1.4426950408889634f;

  uint64_t inflight = 0;  // valid bits of the tiles in the ring, 16 a tile, the oldest lowest
  uint32_t byte = mask_byte(0);
#pragma unroll
  for (int j = 0; j < ST - 1; ++j) {
    const uint32_t bits = bits_of(j, byte);
    byte = mask_byte(j + 1);
    issue(j, bits);
    inflight |= (uint64_t)bits << (16 * j);
  }
  bool ok = true;
  __syncwarp();
  for (int j = 0; j < n; ++j) {
    {
      const uint32_t bits = bits_of(j + ST - 1, byte);
      byte = mask_byte(j + ST);
      issue(j + ST - 1, bits);
      inflight |= (uint64_t)bits << (16 * (ST - 1));
    }
    const uint32_t bits = (uint32_t)inflight & 0xffffu;
    inflight >>= 16;
    ok = __all_sync(0xffffffffu, mbar_wait(&bars[j % ST], (uint32_t)(j / ST) & 1u, abort_flag, a.status));
    if (!ok) {
      // every copy in flight lands before the CTA's shared memory is reused
      for (int i = j; i < min(n, j + ST); ++i) mbar_drain(&bars[i % ST], (uint32_t)(i / ST) & 1u, a.status);
      break;
    }
    const uint32_t ks_u = ring_u + (j % ST) * 2 * C::TILE, vs_u = ks_u + C::TILE;
    if (bits != 0xffffu) {
      uint8_t* v = ring + (j % ST) * 2 * C::TILE + C::TILE;
#pragma unroll
      for (int e = 0; e < kKeys * 8 / 32; ++e) {
        const int r = (lane >> 3) + 4 * e;
        if (!((bits >> r) & 1u))
#pragma unroll
          for (int d = 0; d < C::DB; ++d)
            *reinterpret_cast<uint4*>(v + d * (kKeys * 128) + r * 128 + (lane & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();  // a later copy writes here again
      __syncwarp();
    }

    // S^T = K Q^T, even and odd steps apart (two short chains)
    float s[NB][2][4];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][0][e] = s[i][1][e] = 0.f;
#pragma unroll
    for (int k4 = 0; k4 < KS; k4 += 4) {
      uint32_t kf[4][4];  // matrices: keys 0..7, 8..15 of dims lo; keys 0..7, 8..15 of dims hi
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ldsm4(ks_u + piece(lane & 15, 2 * (k4 + e) + (lane >> 4)), kf[e]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < NB; ++i)
          mma16(s[i][e & 1], kf[e][0], kf[e][1], kf[e][2], kf[e][3], q[k4 + e][i][0], q[k4 + e][i][1]);
    }
    // rows lane / 4 (+ 8) are keys: the maximum of a head is over eight lanes and two rows
    const bool on0 = (bits >> (lane >> 2)) & 1u, on1 = (bits >> (8 + (lane >> 2))) & 1u;
    bool raise = false;
    float factor[NB][2];
    uint32_t p[NB][2];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float& x0 = s[i][0][e];
        float& x1 = s[i][0][2 + e];
        x0 = on0 ? (x0 + s[i][1][e]) * c : -INFINITY;
        x1 = on1 ? (x1 + s[i][1][2 + e]) * c : -INFINITY;
        float top = fmaxf(x0, x1);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        factor[i][e] = 1.f;
        if (top > m[i][e] + kRaise) {
          factor[i][e] = ex2_fast(m[i][e] - top);
          m[i][e] = top;
          raise = true;
        }
      }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[i][e] *= factor[i][e];
#pragma unroll
          for (int t = 0; t < KS; ++t) {
            o[t][i][e] *= factor[i][e];
            o[t][i][2 + e] *= factor[i][e];
          }
        }
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      float w[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float base = m[i][e] == -INFINITY ? 0.f : m[i][e];
        w[e] = ex2_fast(s[i][0][e] - base);
        w[2 + e] = ex2_fast(s[i][0][2 + e] - base);
        l[i][e] += w[e] + w[2 + e];
      }
      // P^T, keys down the rows: heads become the columns' owners
      p[i][0] = transpose8x8(bf16x2(w[0], w[1]));
      p[i][1] = transpose8x8(bf16x2(w[2], w[3]));
    }
    // O^T += V^T P^T: V rows read transposed, 16 dims a load
#pragma unroll
    for (int t4 = 0; t4 < KS; t4 += 4) {
      uint32_t vf[4][4];  // matrices (keys, dims): (lo, lo), (lo, hi), (hi, lo), (hi, hi)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        ldsm4_t(vs_u + piece((lane & 7) + ((lane >> 4) << 3), 2 * (t4 + e) + ((lane >> 3) & 1)), vf[e]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < NB; ++i)
          mma16(o[t4 + e][i], vf[e][0], vf[e][1], vf[e][2], vf[e][3], p[i][0], p[i][1]);
    }
    __syncwarp();  // the stage is overwritten next
  }

  // ---- merge the warps over the ring
  float* part = reinterpret_cast<float*>(smem);                       // [kWarps][DH][HEADS]
  float2* wml = reinterpret_cast<float2*>(smem + C::WARP_ML);          // [kWarps][HEADS]
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], d);
  __syncthreads();  // every warp is done with its tiles
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int h = 8 * i + 2 * (lane & 3);
    if (lane < 4) *reinterpret_cast<float4*>(wml + warp * HEADS + h) = make_float4(m[i][0], l[i][0], m[i][1], l[i][1]);
#pragma unroll
    for (int t = 0; t < KS; ++t)
#pragma unroll
      for (int half = 0; half < 2; ++half)
        *reinterpret_cast<float2*>(part + (warp * DH + 16 * t + 8 * half + (lane >> 2)) * HEADS + h) =
            make_float2(o[t][i][2 * half], o[t][i][2 * half + 1]);
  }
  __syncwarp();
  if (SPLIT) cluster_wait();
  __syncthreads();
  // a thread has four heads of every (512 / HEADS)-th dim
  const int own = DH / split;  // dims an owner merges
  const uint32_t merge_u = smem_u32(smem + C::MERGE), ml_u = smem_u32(smem + C::ML);
  {
    const int h4 = (threadIdx.x % (HEADS / 4)) * 4;
    float top[4], sum[4], f[kWarps][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      top[e] = -INFINITY;
      sum[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top[e] = fmaxf(top[e], wml[w * HEADS + h4 + e].x);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 x = wml[w * HEADS + h4 + e];
        f[w][e] = x.x == -INFINITY ? 0.f : ex2_fast(x.x - top[e]);
        sum[e] += f[w][e] * x.y;
      }
    }
    for (int d = threadIdx.x / (HEADS / 4); d < DH; d += kWarps * 32 / (HEADS / 4)) {
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(part + (w * DH + d) * HEADS + h4);
        v.x += f[w][0] * x.x;
        v.y += f[w][1] * x.y;
        v.z += f[w][2] * x.z;
        v.w += f[w][3] * x.w;
      }
      const int owner = SPLIT ? d / own : 0;
      const uint32_t at = merge_u + ((rank * own + d - owner * own) * HEADS + h4) * 4;
      st_cluster_f4(SPLIT ? mapa(at, owner) : at, v);
    }
    const int owner = threadIdx.x / (HEADS / 4);  // (m, l) of the thread's heads to one owner
    if (owner < split)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t at = ml_u + (rank * HEADS + h4 + e) * 8;
        st_cluster_f2(SPLIT ? mapa(at, owner) : at, top[e], sum[e]);
      }
  }
  __syncwarp();
  if (SPLIT) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  // a thread merges two neighbouring dims of one head
  const float* merge = reinterpret_cast<const float*>(smem + C::MERGE);
  const float2* ml = reinterpret_cast<const float2*>(smem + C::ML);
  for (int i = threadIdx.x; i < own / 2 * HEADS; i += kWarps * 32) {
    const int h = i % HEADS, d = 2 * (i / HEADS);
    if (h >= gc || g0 + h >= G) continue;
    float top = -INFINITY, sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int p = 0; p < kMaxSplit; ++p)
      if (p < split) top = fmaxf(top, ml[p * HEADS + h].x);
#pragma unroll
    for (int p = 0; p < kMaxSplit; ++p)
      if (p < split) {
        const float2 v = ml[p * HEADS + h];
        const float f = v.x == -INFINITY ? 0.f : ex2_fast(v.x - top);
        sum += f * v.y;
        x += f * merge[(p * own + d) * HEADS + h];
        y += f * merge[(p * own + d + 1) * HEADS + h];
      }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    *reinterpret_cast<uint32_t*>(a.out + (int64_t)b * a.out_stride + (int64_t)(kvh * G + g0 + h) * DH + rank * own + d) =
        bf16x2(x * inv, y * inv);
  }
}

template <int DH, int NB, bool SPLIT>
cudaError_t launch(const TokenAttnArgs& a, int gc, int hc, int split, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)split, (unsigned)(a.Hkv * hc), (unsigned)a.batch);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = Cfg<DH, NB>::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 1 : 0;
  CUtensorMap kmap = {}, vmap = {};
  if (a.cache_rows > 0) {  // without rows no tile is loaded
    const int DB = DH / 64;
    cudaError_t e = make_bf16_3d_map(&kmap, a.k, {64, (long)a.cache_rows, (long)a.Hkv * DB}, {(long)a.kv_stride, 64},
                                     {64, kKeys, DB});
    if (e == cudaSuccess)
      e = make_bf16_3d_map(&vmap, a.v, {64, (long)a.cache_rows, (long)a.Hkv * DB}, {(long)a.kv_stride, 64},
                           {64, kKeys, DB});
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, k_token_attn<DH, NB, SPLIT>, kmap, vmap, a, split, hc, gc);
}

template <int DH>
cudaError_t launch_dh(const TokenAttnArgs& a, int gc, int hc, int split, cudaStream_t s) {
  if (gc > 8) return split > 1 ? launch<DH, 2, true>(a, gc, hc, split, s) : launch<DH, 2, false>(a, gc, hc, 1, s);
  return split > 1 ? launch<DH, 1, true>(a, gc, hc, split, s) : launch<DH, 1, false>(a, gc, hc, 1, s);
}

template <int DH, int NB, bool SPLIT>
cudaError_t setup() {
  return cudaFuncSetAttribute(k_token_attn<DH, NB, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<DH, NB>::BYTES);
}

template <int DH>
cudaError_t setup_dh() {
  cudaError_t e = setup<DH, 1, false>();
  if (e == cudaSuccess) e = setup<DH, 2, false>();
  if (e == cudaSuccess) e = setup<DH, 1, true>();
  if (e == cudaSuccess) e = setup<DH, 2, true>();
  return e;
}

}  // namespace

cudaError_t launch_token_attention(const TokenAttnArgs& a, int dh, int sm_count, cudaStream_t s) {
  // heads of a group in chunks of at most 16
  const int G = a.Hq / a.Hkv, hc = (G + 15) / 16, gc = (G + hc - 1) / hc;
  const int64_t units = (int64_t)a.batch * a.Hkv * hc;
  if ((int64_t)a.Hkv * hc > 65535) return cudaErrorInvalidConfiguration;
  // Split a request's keys over more CTAs
  //  - while every cluster of the launch is resident at once (one CTA a SM at
  //    head_dim 256, two below) and a CTA keeps 256 keys, or a tile for every
  //    warp when there are no more CTAs than SMs: 12 requests of up to 2048 keys,
  //    8/1/256: 7.7 us split by 8, 24.2 unsplit; 96 requests of 100 keys: 6.6 us
  //    unsplit, 11.5 split by 2;
  //  - while a CTA keeps 2048 keys: the longest request of a ragged batch bounds
  //    its time (one of 16384 keys among 31 of 50, 32/8/128: 38 us split by 8,
  //    124 unsplit; 64 of 8k: 296 split by 4, 294 unsplit).
  const int64_t slots = (int64_t)sm_count * (dh == 256 ? 1 : 2);
  int split = 1;
  while (split < kMaxSplit) {
    const int64_t ctas = units * split * 2;
    const bool fits = (ctas <= sm_count && a.max_len > split * kWarps * kKeys) ||
                      (ctas <= slots && a.max_len >= split * 2 * 256);
    if (!fits && a.max_len < split * 2 * 2048) break;
    split *= 2;
  }
  if (dh == 64) return launch_dh<64>(a, gc, hc, split, s);
  if (dh == 128) return launch_dh<128>(a, gc, hc, split, s);
  return launch_dh<256>(a, gc, hc, split, s);
}

cudaError_t token_kernel_setup() {
  cudaError_t e = setup_dh<64>();
  if (e == cudaSuccess) e = setup_dh<128>();
  if (e == cudaSuccess) e = setup_dh<256>();
  return e;
}

}  // namespace ae
