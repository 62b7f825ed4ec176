// Attention of packed prompts on the tensor cores (ae_prompt_attention).
//
// The query heads of a KV group are folded into the rows of a tile: a tile is
// T = 128 / G consecutive tokens of a sequence times its G heads (row =
// token * G + head; T * G <= 128 rows used), so short prompts fill tiles and a
// causal diagonal covers few keys.  One CTA works on NQ tiles of one
// (sequence, KV head) and walks the keys in tiles of BK with an online softmax:
//   S = Q K^T       tcgen05, M = 128, N = BK, fp32 in tensor memory
//   P = 2^(c S - m) one thread per row; bf16 back over the S columns it read
//   O += P V        tcgen05, P as the TMEM A operand, O stays in tensor memory
// The exponent reference m is raised (and O, l rescaled) only when a row's
// maximum passes it by more than 2^8, so most tiles skip the rescale and P is
// at most 2^8; l sums the fp32 weights, P is rounded to bf16 because the tensor
// cores multiply bf16 (an error of at most 2^-8 of each term, as V's own).
// Roles: one warpgroup per tile does the softmax, one warp issues TMA loads
// into a ring of K and V tiles, one warp issues the MMAs.
//   head_dim 128: two tiles a CTA alternate, one's MMAs under the other's
//     softmax; a key tile (two query tiles) takes about 2770 clocks, of which
//     the MMAs 2048.  32768 tokens 32/8/128: 4.8 ms, 1820 TFLOP/s; bound by the
//     MMA rate, shared memory's bandwidth near it (operands and TMA writes take
//     2048 clocks a step too).
//     Where SMs would idle, one tile a CTA with two S buffers, as at 256: a key
//     tile then takes 1450 clocks (16/2/128: 1500 tokens 14.7 us against 22.3 with
//     two tiles a CTA, 4096 48.3 against 55.2 with one).
//   head_dim 256: O fills half of tensor memory; one tile, two S buffers, the
//     next Q K^T under this softmax; K and V in half tiles so that a ring of five
//     fits beside Q.  8192 tokens 8/1/256: 151 us, 1820 TFLOP/s.  (Key tiles of
//     64: 191 us, Q K^T of 64 columns is bound by reading Q from shared memory.)
//   head_dim 64: one tile a CTA and two CTAs a SM, each in the half of tensor
//     memory, so one's start, end and MMAs run under the other's softmax; key
//     tiles of 96, the largest of which two score buffers fit beside O, so the
//     next Q K^T runs under this softmax too.  No unit is full (issue 57% of the
//     cycles, exponentials 46%, tensor pipe 45%): the chain of a softmax warp
//     bounds it, two of which share a scheduler.  8192 tokens 12/4/64: 101 us,
//     1020 TFLOP/s.  (Key tiles of 128, one score buffer: 115 us, prompts of one
//     to 4097 tokens 40.6 against 34.7 us; 100 tokens, which that holds in one
//     tile, 14.6 against 15.0 us for 64 of them.  Two tiles sharing K and V in one
//     CTA: 117 us; four on keys of 64: 138 us.)
// What the MMAs need most is an issue thread that never waits: they are issued
// under elect.sync on warp-uniform operands (a plain lane test costs 75 clocks
// per MMA in register moves: 6.7 ms for the 32768 tokens), and both next slots
// are awaited before the weights.  Tried on earlier states of this kernel and
// slower, 8192 tokens 32/8/128 (340 us now): two threads a row (430 against 351
// us), P handed over in halves (493 against 461), persistent CTAs with static
// shares that fetch the next unit's tiles under this one's end (356 against 341;
// ragged batches, where starts and ends weigh most, were not tried).
// A unit's start and end cost about 8500 clocks (first loads and products 5000,
// output by TMA through the query tile 2400 at 32 bytes a clock); short prompts
// are bound by them.
// Keys that a row may not see get score -inf; V rows that no row may see (a
// sequence's end inside the tile, masked rows) are zeroed in shared memory,
// since 0 * NaN would reach every row.
// Few query rows over many keys leave SMs idle: the key tiles are then split
// over the CTAs of a cluster, which exchange fp32 partials through distributed
// shared memory (no workspace, one launch, sums in rank order).  SMs that are
// still idle take half of the value dims each (the scores twice, the rest once):
// the P V, the output and the merge of a CTA are halved.  16 tokens over 4080 keys
// 8/1/256: 12.3 us against 15.2 with whole rows; a prompt of 50: 7.3 against 7.5.
// (Not for pairs of tiles, which single ones replace before SMs idle: 8 prompts of
// 64 tokens 32/8/128 6.0 us in single tiles, 6.4 in pairs with halved dims.)
#include <math.h>

#include "ae_internal.h"
#include "ae_tc.cuh"

namespace ae {
namespace {

using namespace tc;

constexpr int kListTiles = 512;
constexpr float kRaise = 8.f;  // log2: raise the exponent reference past this

template <int DH, int NQ_>
struct Cfg {
  static constexpr int NQ = NQ_;                   // query tiles of a CTA
  static constexpr int SB = NQ == 1 ? 2 : 1;     // score buffers of a query tile
  static constexpr int CTAS = DH == 64 ? 2 : 1;    // resident a SM
  static constexpr int BK = DH == 64 ? 96 : 128;                   // keys of a tile
  static constexpr int DB = DH / 64;               // 64-dim blocks of a row
  static constexpr int LOG_DIMS = DH == 64 ? 6 : (DH == 128 ? 7 : 8);
  // a ring slot holds a K or V tile; at head_dim 256 half of one: all keys of half
  // the dims of K, all dims of half the keys of V
  static constexpr int PARTS = DH == 256 ? 2 : 1;
  static constexpr int DBK = DB / PARTS, BKV = BK / PARTS;
  static constexpr int SLOT = BK * DH * 2 / PARTS;
  static constexpr int NS = 5;                     // ring slots
  static constexpr int QBYTES = 128 * DH * 2;      // bytes of a query tile
  // threads: the softmax warpgroups, then one of which two warps work (loads,
  // MMAs).  It hands registers to the others where the launch's would not do:
  // 104 + 2 * 200 = 3 * 168 (NQ = 2), 96 + 160 = 2 * 128 (two CTAs a SM).
  static constexpr int THREADS = NQ * 128 + 128;
  static constexpr bool VS = DH > 64 && NQ == 1;   // the value dims may be halved
  static constexpr bool TRADE = NQ == 2 || CTAS == 2;
  static constexpr int REGS_AUX = NQ == 2 ? 104 : 96, REGS_MAX = NQ == 2 ? 200 : 160;
  static constexpr int W_LOAD = NQ * 4, W_MMA = NQ * 4 + 1;
  // shared memory, from a 1024-byte boundary
  static constexpr int RING = NQ * QBYTES;
  static constexpr int BARS = RING + NS * SLOT;
  static constexpr int ML = NQ * 128 * DH * 4;     // a split's partial: fp32 rows, then [NQ][128] (m, l)
  static constexpr int WT = ML + NQ * 128 * 8;     // [rows of this CTA][split] weights of the merge
  static constexpr int LIST = BARS + 256;          // key tiles with valid keys (masked calls): entries, then states
  static constexpr int BYTES = LIST + kListTiles * 3 + 1024;
  // a split launch of no more CTAs than SMs asks for more than half an SM's: two
  // CTAs of it would share SMs while others idle (16 tokens over 4080 keys 4/1/64)
  static constexpr int SPLIT_BYTES = BYTES > 120 * 1024 ? BYTES : 120 * 1024;
  // tensor memory columns: scores, then O
  static constexpr int O0 = NQ * SB * BK, COLS = O0 + NQ * DH <= 256 ? 256 : 512;
  static_assert(WT + NQ * 128 * 4 <= BARS, "fp32 partials fit over the tiles");
  static_assert(CTAS * (BYTES + 1024) <= 228 * 1024, "shared memory");
  static_assert(O0 + NQ * DH <= COLS && CTAS * COLS <= 512, "tensor memory");
};

struct Launch {
  int n_order;                       // sequences with work
  int G, Gc, hc, T;                  // heads of a group, of a tile; head chunks; tokens of a tile
  int per;                           // units of one token range: KV heads x head chunks
  uint32_t per_inv, gc_inv;          // ceil(2^32 / per), ceil(2^32 / Gc)
  int split;                         // CTAs of a cluster
  int vs;                            // 2: each half of the value dims is another CTA's (cluster's)
  int work_cu[AE_MAX_BATCH + 1];     // first work unit of the i-th sequence, longest first
  uint8_t order[AE_MAX_BATCH];
};

struct Bars {
  uint64_t q, full[8], empty[8], s[2], p[2], o[2], drain;
  uint32_t tmem;
  int abort;
  int listed[2];  // listed tiles of each query tile
};
static_assert(sizeof(Bars) <= 256, "");

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

#define AE_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), \
                    "=r"(r[o + 6]), "=r"(r[o + 7])
#define AE_U8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), "+r"(r[o + 5]), \
                    "+r"(r[o + 6]), "+r"(r[o + 7])
#define AE_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), \
                    "r"(r[o + 6]), "r"(r[o + 7])

// Start of a load of 32 lanes x 32 columns; the registers hold the values only
// after tmem_ld_wait() and landed().
__device__ __forceinline__ void tmem_ld32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : AE_R8(r, 0), AE_R8(r, 8), AE_R8(r, 16), AE_R8(r, 24)
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Orders uses of r behind the wait before it (the wait does not name the registers).
__device__ __forceinline__ void landed(uint32_t (&r)[32]) {
  asm volatile("" : AE_U8(r, 0), AE_U8(r, 8), AE_U8(r, 16), AE_U8(r, 24));
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      AE_I8(r, 0), AE_I8(r, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(
          taddr),
      AE_I8(r, 0), AE_I8(r, 8), AE_I8(r, 16), AE_I8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// mbar_wait of a whole warp: one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

// First n bits of the k-th word.
__device__ __forceinline__ uint32_t low_bits(int n, int k) {
  n -= 32 * k;
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// Valid keys of the tile at key0 of a sequence of n_keys keys (bit = key;
// mask: the sequence's mask bytes or nullptr).  Whole warp.
template <int BK>
__device__ __forceinline__ void tile_bits(const uint8_t* mask, int key0, int n_keys, uint32_t (&w)[BK / 32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < BK / 32; ++k) {
    if (mask != nullptr) {
      const int key = key0 + 32 * k + lane;
      w[k] = __ballot_sync(0xffffffffu, key < n_keys && mask[key] != 0);
    } else {
      w[k] = low_bits(n_keys - key0, k);
    }
  }
}

// A work unit: NQ tiles of one (sequence, KV head, chunk of its heads), and
// this CTA's range [lo, hi) of key tiles.
struct Unit {
  int tok0;        // first token of the first tile, within its sequence
  int n_new, n_keys, q_row0;
  int64_t kv_row0;
  int kvh, g0;     // KV head; first head of the tile within its group
};

// x / d for x >= 0; inv = ceil(2^32 / d) where x * d < 2^32 for every x (then
// the high word of the product is exact), else 0.
__device__ __forceinline__ int divide(int x, int d, uint32_t inv) {
  return d == 1 ? x : (inv != 0u ? (int)__umulhi((uint32_t)x, inv) : x / d);
}

template <int NQ>
__device__ __forceinline__ Unit find_unit(const PromptAttnArgs& a, const Launch& L, int u) {
  int i = 0;
  if (L.n_order > 1) {
#pragma unroll
    for (int step = 32; step > 0; step >>= 1)
      if (i + step < L.n_order && L.work_cu[i + step] <= u) i += step;
  }
  const int b = L.order[i];
  // counted from the sequence's last unit: its longest key ranges come first
  u = L.work_cu[i + 1] - 1 - u;
  Unit w;
  w.q_row0 = a.cu_q[b];
  w.n_new = a.cu_q[b + 1] - a.cu_q[b];
  w.n_keys = a.kv_len[b];
  w.kv_row0 = a.kv_row0[b];
  const int t = divide(u, L.per, L.per_inv), h = u - t * L.per;
  w.kvh = L.hc == 1 ? h : h / L.hc;
  w.g0 = (h - w.kvh * L.hc) * L.Gc;
  w.tok0 = t * L.T * NQ;
  return w;
}

// Rank r of P CTAs merges its share of the rows in use: 16-byte pieces of the
// partials, 16 in flight a thread, the first ones under the computation of the
// weights 2^(m_p - m) / l of every split.  Bound by remote shared memory (15 bytes
// a clock measured with all of them in flight), so rows that hold no query are
// left out: 16 tokens over 1016 keys 32/8/128 9.8 us, 12.4 with them.
template <int DH, int NQ, int P>
__device__ __forceinline__ void merge_rows(const PromptAttnArgs& a, const Launch& L, const Unit& w, uint8_t* smem,
                                           int rank, int half) {
  using C = Cfg<DH, NQ>;
  constexpr int UN = 16 / P;
  const int vs = C::VS ? L.vs : 1;
  const int shift = C::LOG_DIMS - 1 - vs, per = 1 << shift;  // pieces of a row
  const int rows0 = max(0, min(L.T, w.n_new - w.tok0)) * L.Gc;
  const int rows = rows0 + (C::NQ == 2 ? max(0, min(L.T, w.n_new - w.tok0 - L.T)) * L.Gc : 0);
  const int i_lo = rows * rank / P, share = rows * (rank + 1) / P - i_lo;
  auto tile_row = [&](int i) { return i_lo + i < rows0 ? i_lo + i : 128 + i_lo + i - rows0; };
  const uint32_t base = smem_u32(smem), ml = smem_u32(smem + C::ML);
  float* wt = reinterpret_cast<float*>(smem + C::WT);  // [share][P]
  uint32_t peer[P];
#pragma unroll
  for (int p = 0; p < P; ++p) peer[p] = mapa(base, p);
  float4 v[UN][P];
  auto load = [&](int i0) {
#pragma unroll
    for (int e = 0; e < UN; ++e) {
      const int i = i0 + e * C::THREADS, r = tile_row(i >> shift), q = i & (per - 1);
      if (i >= share << shift) break;
      const uint32_t off = r * (DH * 4) + ((q ^ (r & 7)) << 4);
#pragma unroll
      for (int p = 0; p < P; ++p) v[e][p] = ld_cluster_f4(peer[p] + off);
    }
  };
  load(threadIdx.x);
  for (int i = threadIdx.x; i < share; i += C::THREADS) {
    const int r = tile_row(i);
    float2 x[P];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = ld_cluster_f2(mapa(ml + r * 8, p));
#pragma unroll
    for (int p = 0; p < P; ++p) m = fmaxf(m, x[p].x);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      x[p].x = x[p].y > 0.f ? ex2_fast(x[p].x - m) : 0.f;
      l += x[p].x * x[p].y;
    }
#pragma unroll
    for (int p = 0; p < P; ++p) wt[i * P + p] = l > 0.f ? x[p].x / l : 0.f;
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < share << shift; i0 += UN * C::THREADS) {
    if (i0 != (int)threadIdx.x) load(i0);
#pragma unroll
    for (int e = 0; e < UN; ++e) {
      const int i = i0 + e * C::THREADS, r = tile_row(i >> shift), q = i & (per - 1);
      const int s = r >> 7, rr = r & 127;
      const int tok = divide(rr, L.Gc, L.gc_inv), g = w.g0 + rr - tok * L.Gc;
      if (i >= share << shift || g >= L.G) continue;
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const float f = wt[(i >> shift) * P + p];
        o.x += f * v[e][p].x;
        o.y += f * v[e][p].y;
        o.z += f * v[e][p].z;
        o.w += f * v[e][p].w;
      }
      *reinterpret_cast<uint2*>(a.out + (int64_t)(w.q_row0 + w.tok0 + s * L.T + tok) * a.out_stride +
                                (int64_t)(w.kvh * L.G + g) * DH + half * (DH / 2) + 4 * q) = make_uint2(bf16x2(o.x, o.y), bf16x2(o.z, o.w));
    }
  }
}

// MASKED: the call has a key mask.
template <int DH, int NQ, bool MASKED>
__global__ void __launch_bounds__(Cfg<DH, NQ>::THREADS, Cfg<DH, NQ>::CTAS)
    k_prompt_attn(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap, const __grid_constant__ CUtensorMap omap,
                  const __grid_constant__ PromptAttnArgs a,
                  const __grid_constant__ Launch L) {
  using C = Cfg<DH, NQ>;
  const int vs = C::VS ? L.vs : 1;
  constexpr int SB = C::SB, BK = C::BK, DB = C::DB, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars* B = reinterpret_cast<Bars*>(smem + C::BARS);
  volatile int* abort_flag = &B->abort;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const int rank = L.split > 1 ? (int)cluster_rank() : 0;
  if (warp == C::W_LOAD && lane == 0) {
    mbar_init(&B->q, 1);
    mbar_init(&B->drain, 1);
    for (int i = 0; i < 8; ++i) {
      mbar_init(&B->full[i], 1);
      mbar_init(&B->empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B->s[i], 1);
      mbar_init(&B->p[i], 4);
      mbar_init(&B->o[i], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
    prefetch_tensormap(&qmap);
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&omap);
  }
  if (warp == C::W_MMA) {
    tmem_alloc(&B->tmem, C::COLS);
    tmem_relinquish();
  }
  const int half = (int)(blockIdx.x / L.split) & (vs - 1);
  const Unit w = find_unit<NQ>(a, L, (int)(blockIdx.x / L.split) >> (vs - 1));
  const uint8_t* mask = MASKED ? a.key_mask + w.kv_row0 : nullptr;

  // key tiles of every query tile: up to its last token's last key
  int cnt[NQ], most = 0;
#pragma unroll
  for (int s = 0; s < NQ; ++s) {
    const int t0 = w.tok0 + s * L.T;
    const int last = min(t0 + L.T, w.n_new) - 1;
    const int keys = t0 >= w.n_new ? 0 : (a.causal ? w.n_keys - w.n_new + last + 1 : w.n_keys);
    cnt[s] = (keys + BK - 1) / BK;
    most = max(most, cnt[s]);
  }
  int lo = 0, hi = most;
  if (L.split > 1) {
    lo = (int)((int64_t)most * rank / L.split);
    hi = (int)((int64_t)most * (rank + 1) / L.split);
  }
  int n_tiles = 0;
#pragma unroll
  for (int s = 0; s < NQ; ++s) {
    cnt[s] = max(0, min(cnt[s], hi) - lo);
    n_tiles = max(n_tiles, cnt[s]);
  }

  const bool q_loaded = n_tiles > 0;
  if (warp == C::W_LOAD && lane == 0 && q_loaded) {  // under the look at the mask
    mbar_arrive_expect_tx(&B->q, (uint32_t)(NQ * DB * L.T * L.Gc * 128));
#pragma unroll
    for (int s = 0; s < NQ; ++s)
#pragma unroll
      for (int d = 0; d < DB; ++d)
        tma_load_3d_nohint(smem + s * C::QBYTES + d * (128 * 128), &qmap, &B->q, d * 64, w.kvh * L.G + w.g0,
                           w.q_row0 + w.tok0 + s * L.T);
  }

  // Masked calls: the tiles that hold a valid key, in order, with the top bit
  // set when some of their keys are masked; all other tiles are skipped.  (Key
  // ranges beyond the list's room look every tile's mask up instead.)
  uint16_t* list = reinterpret_cast<uint16_t*>(smem + C::LIST);
  const bool listed = MASKED && n_tiles <= kListTiles;
  if (listed) {
    uint8_t* state = smem + C::LIST + kListTiles * 2;  // 0 none, 1 some, 2 all keys valid
    for (int t = warp; t < n_tiles; t += C::THREADS / 32) {
      uint32_t bits[BK / 32], any = 0, all = 0xffffffffu;
      tile_bits<BK>(mask, (lo + t) * BK, w.n_keys, bits);
#pragma unroll
      for (int k = 0; k < BK / 32; ++k) {
        any |= bits[k];
        all &= bits[k];
      }
      if (lane == 0) state[t] = any == 0 ? 0 : (all == 0xffffffffu ? 2 : 1);
    }
    __syncthreads();
    if (warp == 0) {
      int n = 0, first = 0;  // listed tiles; those of the first query tile
      for (int t0 = 0; t0 < n_tiles; t0 += 32) {
        const int t = t0 + lane, st = t < n_tiles ? state[t] : 0;
        const uint32_t m = __ballot_sync(0xffffffffu, st != 0);
        if (st != 0) list[n + __popc(m & ((1u << lane) - 1u))] = (uint16_t)(t | (st == 1 ? 0x8000 : 0));
        n += __popc(m);
        first += __popc(m & low_bits(cnt[0] - t0, 0));
      }
      if (lane == 0) {
        B->listed[0] = first;
        if (NQ == 2) B->listed[1] = cnt[NQ - 1] >= cnt[0] ? n : 0;
      }
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < NQ; ++s) cnt[s] = B->listed[s];
    n_tiles = max(cnt[0], cnt[NQ - 1]);
  }
  // key tile (from lo) of the i-th step, and whether some of its keys are masked
  auto tile_at = [&](int i) { return listed ? list[i] & 0x7fff : i; };
  auto holes_at = [&](int i) { return listed ? (list[i] & 0x8000) != 0 : MASKED; };

  // The load warp starts the first copies before the CTA meets.  The ring holds
  // the tiles in the order the MMAs use them: K0 V0 K1 V1 .. (NQ = 2),
  // K0 K1 V0 K2 V1 .. (NQ = 1).
  int loaded = 0;
  auto load = [&]() {
    const int i = loaded / C::PARTS, h = loaded % C::PARTS;
    const bool is_v = SB == 1 ? (i & 1) : (i > 0 && ((i & 1) == 0 || i + 1 == 2 * n_tiles));
    const int t = SB == 1 ? i >> 1 : (is_v ? (i + 1 == 2 * n_tiles ? n_tiles - 1 : (i >> 1) - 1) : (i + 1) >> 1);
    const int slot = loaded % NS;
    mbar_arrive_expect_tx(&B->full[slot], is_v ? C::SLOT >> (vs - 1) : C::SLOT);
    tma_load_3d_nohint(smem + C::RING + slot * C::SLOT, is_v ? &vmap : &kmap, &B->full[slot], 0,
                       (int)(w.kv_row0 + (int64_t)(lo + tile_at(t)) * BK) + (is_v ? h * C::BKV : 0),
                       w.kvh * DB + (is_v ? half * (DB / 2) : h * C::DBK));
    ++loaded;
  };
  if (warp == C::W_LOAD && lane == 0 && n_tiles > 0) {
    while (loaded < C::PARTS) load();  // the first tile's K; the rest after the CTA has met
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B->tmem;

  if (warp >= C::W_LOAD) {
    if (C::TRADE) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_AUX));
  if (warp == C::W_LOAD) {
    // ---------------------------------------------------------------- loads
    if (lane == 0 && q_loaded) {
      while (loaded < 2 * C::PARTS * n_tiles &&
             (loaded < NS || mbar_wait(&B->empty[loaded % NS], (uint32_t)((loaded / NS) & 1) ^ 1u, abort_flag, a.status)))
        load();
      // every copy lands before the CTA's shared memory is released, also after a failure
      mbar_drain(&B->q, 0, a.status);
      for (int i = max(0, loaded - NS); i < loaded; ++i)
        mbar_drain(&B->full[i % NS], (uint32_t)(i / NS) & 1u, a.status);
    }
  } else if (warp == C::W_MMA) {
    // ---------------------------------------------------------------- MMAs
    constexpr uint32_t idesc_s = idesc_bf16(128, BK);
    const uint32_t idesc_o = vs == 2 ? idesc_bf16(128, DH / 2, true) : idesc_bf16(128, DH, true);
    int c = 0;  // ring slots consumed
    bool ok = n_tiles == 0 || warp_wait(&B->q, 0, abort_flag, a.status);
    auto wait_slot = [&](int i) { return warp_wait(&B->full[i % NS], (uint32_t)(i / NS) & 1u, abort_flag, a.status); };
    const uint64_t q_desc = sdesc_sw128(smem_u32(smem)), k_desc = sdesc_sw128(smem_u32(smem) + C::RING),
                   v_desc = sdesc_sw128_mn(smem_u32(smem) + C::RING, C::BKV * 128, 1024);
    // part h of S = Q K^T (of the dims) and of O += P V (of the keys)
    auto qk = [&](int s, int buf, int slot, int h) {
      const uint64_t ad = q_desc + (uint64_t)(s * C::QBYTES >> 4), bd = k_desc + (uint64_t)(slot * C::SLOT >> 4);
      if (elect_one()) {
#pragma unroll
        for (int d = 0; d < C::DBK; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_bf16(tmem + (uint32_t)(buf * BK), ad + (h * C::DBK + d) * (128 * 128 >> 4) + 2 * k,
                     bd + d * (BK * 128 >> 4) + 2 * k, idesc_s, (h > 0 || d > 0 || k > 0) ? 1u : 0u);
        if (h == C::PARTS - 1) mma_commit(&B->s[buf]);
      }
      __syncwarp();
    };
    auto pv = [&](int s, int buf, int slot, bool first, uint64_t* done, int h) {
      const uint64_t bd = v_desc + (uint64_t)(slot * C::SLOT >> 4);
      const uint32_t acc = first ? 0u : 1u;
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < C::BKV / 16; ++k)
          mma_bf16_ts(tmem + (uint32_t)(C::O0 + s * DH), tmem + (uint32_t)(buf * BK + 8 * (h * (C::BKV / 16) + k)),
                      bd + k * (2048 >> 4), idesc_o, (h > 0 || k > 0) ? 1u : acc);
        if (done != nullptr && h == C::PARTS - 1) mma_commit(done);
      }
      __syncwarp();
    };
    auto release = [&](int slot) {
      if (elect_one()) mma_commit(&B->empty[slot]);
      __syncwarp();
    };
    // zero the V rows of part h of tile i that no query may see
    auto clean_v = [&](int i, int slot, int h) {
      const int key0 = (lo + tile_at(i)) * BK + h * C::BKV;
      const bool holes = holes_at(i);
      if (!holes && key0 + C::BKV <= w.n_keys) return;
      uint32_t bits[C::BKV / 32];
      tile_bits<C::BKV>(holes ? mask : nullptr, key0, w.n_keys, bits);
      uint32_t all = 0xffffffffu;
#pragma unroll
      for (int k = 0; k < C::BKV / 32; ++k) all &= bits[k];
      if (all == 0xffffffffu) return;
      uint8_t* v = smem + C::RING + slot * C::SLOT;
#pragma unroll
      for (int k = 0; k < C::BKV / 32; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // 16-byte piece lane + 32 e of this word's 32 rows: row (lane + 32 e) / 8
          const int r = (lane >> 3) + 4 * e;
          if (!((bits[k] >> r) & 1u))
#pragma unroll
            for (int d = 0; d < DB; ++d)
              *reinterpret_cast<uint4*>(v + d * (C::BKV * 128) + (32 * k + r) * 128 + (lane & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
        }
      fence_proxy_async_smem();
      __syncwarp();
    };
    if (SB == 1) {
      if (n_tiles > 0 && ok && (ok = wait_slot(0))) {
#pragma unroll
        for (int s = 0; s < NQ; ++s)
          if (cnt[s] > 0) qk(s, s, 0, 0);
        release(0);
        c = 1;
      }
      for (int i = 0; i < n_tiles && ok; ++i) {
        // slot c: V of tile i, slot c + 1: K of tile i + 1
        if (!(ok = wait_slot(c))) break;
        clean_v(i, c % NS, 0);
        if (i + 1 < n_tiles && !(ok = wait_slot(c + 1))) break;
#pragma unroll
        for (int s = 0; s < NQ; ++s) {
          if (ok && i < cnt[s]) {
            if (!(ok = warp_wait(&B->p[s], (uint32_t)i & 1u, abort_flag, a.status))) break;
            tc_fence_after();
            pv(s, s, c % NS, i == 0, i + 1 == cnt[s] ? &B->o[s] : nullptr, 0);
            if (i + 1 < cnt[s]) qk(s, s, (c + 1) % NS, 0);
          }
        }
        if (!ok) break;
        release(c % NS);
        if (i + 1 < n_tiles) release((c + 1) % NS);
        c += 2;
      }
    } else {
#pragma unroll
      for (int h = 0; h < C::PARTS; ++h)
        if (n_tiles > 0 && ok && (ok = wait_slot(c))) {
          qk(0, 0, c % NS, h);
          release(c % NS);
          ++c;
        }
      for (int i = 0; i < n_tiles && ok; ++i) {
#pragma unroll
        for (int h = 0; h < C::PARTS; ++h)
          if (ok && i + 1 < n_tiles && (ok = wait_slot(c))) {
            qk(0, (i + 1) & 1, c % NS, h);
            release(c % NS);
            ++c;
          }
#pragma unroll
        for (int h = 0; h < C::PARTS; ++h) {
          if (!ok || !(ok = wait_slot(c))) break;
          clean_v(i, c % NS, h);
          if (h == 0) {
            if (!(ok = warp_wait(&B->p[i & 1], (uint32_t)(i >> 1) & 1u, abort_flag, a.status))) break;
            tc_fence_after();
          }
          pv(0, i & 1, c % NS, i == 0, &B->o[i & 1], h);
          release(c % NS);
          ++c;
        }
      }
    }
    if (!ok && lane == 0) {  // MMAs in flight must finish before tensor memory is freed
      mma_commit(&B->drain);
      mbar_drain(&B->drain, 0, a.status);
    }
    __syncwarp();
  }
  } else {
    // ---------------------------------------------------------------- softmax
    if (C::TRADE) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_MAX));
    const int s = warp >> 2;             // query tile of this warpgroup
    const int row = threadIdx.x & 127;   // its row, the TMEM lane
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const int tok = divide(row, L.Gc, L.gc_inv), g = w.g0 + row - tok * L.Gc;
    const int t0 = w.tok0 + s * L.T;
    const bool real = tok < L.T && t0 + tok < w.n_new && g < L.G;
    // keys this row sees; keys every row of the tile sees
    const int back = a.causal ? w.n_keys - w.n_new + 1 : 0;
    const int limit = !real ? 0 : (a.causal ? back + t0 + tok : w.n_keys);
    const int open = a.causal ? back + t0 : w.n_keys;
    const float c = a.scale * 1.4426950408889634f;  // scores in the log2 domain
    const uint32_t tm_o = tmem + lane_off + (uint32_t)(C::O0 + s * DH);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    const int n = s == 0 ? cnt[0] : cnt[NQ - 1];
    for (int i = 0; i < n; ++i) {
      const int buf = SB == 2 ? i & 1 : s;
      const uint32_t tm_s = tmem + lane_off + (uint32_t)(buf * BK);
      const int key0 = (lo + tile_at(i)) * BK;
      const bool holes = holes_at(i), partial = holes || key0 + BK > open;
      uint32_t bits[BK / 32];
      if (partial) {
        tile_bits<BK>(holes ? mask : nullptr, key0, w.n_keys, bits);
#pragma unroll
        for (int k = 0; k < BK / 32; ++k) bits[k] &= low_bits(limit - key0, k);
      }
      if (!warp_wait(&B->s[buf], (uint32_t)(SB == 2 ? i >> 1 : i) & 1u, abort_flag, a.status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sc[BK / 32][32];
      float mx[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) mx[e] = -INFINITY;
#pragma unroll
      for (int k = 0; k < BK / 32; ++k) tmem_ld32_start(tm_s + 32 * k, sc[k]);
      tmem_ld_wait();
#pragma unroll
      for (int k = 0; k < BK / 32; ++k) {
        landed(sc[k]);
        if (partial) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!((bits[k] >> j) & 1u)) sc[k][j] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int j = 0; j < 32; j += 2)
          mx[(j >> 1) & 7] = max3(mx[(j >> 1) & 7], __uint_as_float(sc[k][j]), __uint_as_float(sc[k][j + 1]));
      }
      const float top = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])),
                              fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * c;
      float factor = 1.f;
      if (top > m + kRaise) {  // -inf stays -inf while no key has been seen
        factor = ex2_fast(m - top);
        m = top;
      }
      if (i > 0 && __any_sync(0xffffffffu, factor != 1.f)) {
        // O holds tiles 0 .. i-1: with NQ = 2 their P V are done (S of this
        // tile was issued behind them), with NQ = 1 the last one may still run
        if (SB == 2 && !warp_wait(&B->o[(i - 1) & 1], (uint32_t)((i - 1) >> 1) & 1u, abort_flag, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        l *= factor;
#pragma unroll 1
        for (int d = 0; d < DH >> (vs - 1); d += 32) {
          uint32_t o[32];
          tmem_ld32_start(tm_o + d, o);
          tmem_ld_wait();
          landed(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * factor);
          tmem_st(tm_o + d, o);
        }
        tmem_st_wait();
      }
      const float base = m == -INFINITY ? 0.f : -m;
      const uint64_t c2 = pack2(c, c), b2 = pack2(base, base);
      uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < BK / 32; ++k) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float x, y;
          unpack2(fma2(pack2(__uint_as_float(sc[k][e]), __uint_as_float(sc[k][e + 1])), c2, b2), x, y);
          x = ex2_fast(x);
          y = ex2_fast(y);
          sum[(e >> 1) & 3] = add2(sum[(e >> 1) & 3], pack2(x, y));
          p[e >> 1] = bf16x2(x, y);
        }
        tmem_st(tm_s + 16 * k, p);  // over S columns read above
      }
      float x, y;
      unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), x, y);
      l += x + y;
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->p[buf]);
    }
    if (ok && n > 0)
      ok = SB == 2 ? warp_wait(&B->o[(n - 1) & 1], (uint32_t)((n - 1) >> 1) & 1u, abort_flag, a.status)
                   : warp_wait(&B->o[s], 0, abort_flag, a.status);
    // a masked tile without keys has waited for nothing yet, and its zeros go over
    // the query tile: the queries must have landed
    if (MASKED && n == 0 && q_loaded) ok = warp_wait(&B->q, 0, abort_flag, a.status);
    __syncwarp();
    tc_fence_after();
    if (L.split == 1) {
      // Rows through shared memory, over the query tile whose products are done
      // (its layout), then out by TMA; a tile cut short by the sequence's end (or
      // the group's) in runs of whole rows by its threads.
      const float inv = l > 0.f ? 1.f / l : 0.f;
      uint8_t* tile = smem + s * C::QBYTES;
      const bool whole = t0 + L.T <= w.n_new && w.g0 + L.Gc <= L.G;
#pragma unroll 1
      for (int d = 0; d < DB >> (vs - 1); ++d) {
        uint32_t o[2][32];
        if (n > 0) {
          tmem_ld32_start(tm_o + 64 * d, o[0]);
          tmem_ld32_start(tm_o + 64 * d + 32, o[1]);
          tmem_ld_wait();
          landed(o[0]);
          landed(o[1]);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          uint32_t v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = (8 * q + 2 * e) & 31;
            v[e] = l > 0.f ? bf16x2(__uint_as_float(o[q >> 2][k]) * inv, __uint_as_float(o[q >> 2][k + 1]) * inv) : 0u;
          }
          *reinterpret_cast<uint4*>(tile + d * (128 * 128) + sw128_offset(row, q)) = make_uint4(v[0], v[1], v[2], v[3]);
        }
        if (whole) {  // a block of 64 dims leaves while the next is staged
          fence_proxy_async_smem();
          if (s == 0) asm volatile("bar.sync 1, 128;" ::: "memory");
          else asm volatile("bar.sync 2, 128;" ::: "memory");
          if (row == 0 && ok) {
            tma_store_3d(&omap, tile + d * (128 * 128), half * (DH / 2) + d * 64, w.kvh * L.G + w.g0, w.q_row0 + t0);
            bulk_commit();
          }
        }
      }
      if (whole) {
        if (row == 0) bulk_wait_read_all();
      } else if (ok) {
        __syncwarp();  // a warp stores the 32 rows it wrote
        constexpr int CPR = DH / 8, RPI = 32 / CPR;  // pieces of a row; rows an instruction
        const int r0 = 32 * (warp & 3) + lane / CPR, ch = lane % CPR;
        bf16* out0 = a.out + (int64_t)(w.q_row0 + t0) * a.out_stride + (int64_t)(w.kvh * L.G + w.g0) * DH + half * (DH / 2) + 8 * ch;
        const int rows = min(32 * (warp & 3) + 32, min(L.T, w.n_new - t0) * L.Gc);
#pragma unroll 8
        for (int r = r0; r < rows; r += RPI) {
          const int rt = divide(r, L.Gc, L.gc_inv), rg = r - rt * L.Gc;
          if (w.g0 + rg < L.G && ch < CPR >> (vs - 1))
            *reinterpret_cast<uint4*>(out0 + rt * a.out_stride + rg * DH) =
                *reinterpret_cast<const uint4*>(tile + (ch >> 3) * (128 * 128) + sw128_offset(r, ch & 7));
        }
      }
    } else if (L.split > 1) {
      // this split's partial into shared memory, over the tiles: every TMA copy
      // and MMA of both warpgroups' tiles must have finished reading them
      if (NQ == 2) asm volatile("bar.sync 1, 256;" ::: "memory");
      reinterpret_cast<float2*>(smem + C::ML)[s * 128 + row] = ok ? make_float2(m, l) : make_float2(-INFINITY, 0.f);
      uint8_t* part = smem + (s * 128 + row) * (DH * 4);
#pragma unroll 1
      for (int d = 0; d < DH >> (vs - 1); d += 32) {
        uint32_t o[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) o[j] = 0u;
        if (n > 0 && ok) {
          tmem_ld32_start(tm_o + d, o);
          tmem_ld_wait();
          landed(o);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)  // 16-byte pieces XORed by row: conflict-free
          *reinterpret_cast<uint4*>(part + ((((d >> 2) + q) ^ (row & 7)) << 4)) =
              make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
  if (L.split > 1) {
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    // the unit found again: kept in registers it would spill in the loops above
    unsigned bx = blockIdx.x;
    asm volatile("" : "+r"(bx));
    const int half = (int)(bx / L.split) & (vs - 1);
    const Unit w = find_unit<NQ>(a, L, (int)(bx / L.split) >> (vs - 1));
    const int rank = (int)cluster_rank();
    if (L.split == 2) merge_rows<DH, NQ, 2>(a, L, w, smem, rank, half);
    else if (L.split == 4) merge_rows<DH, NQ, 4>(a, L, w, smem, rank, half);
    else merge_rows<DH, NQ, 8>(a, L, w, smem, rank, half);
    __syncthreads();
    cluster_arrive();  // no CTA leaves while a peer reads its partials
    cluster_wait();
  }
}

// The units of a call and their split; its cost in clocks, negative when there are
// too many units.  resident: clusters of 1, 2, 4 and 8 CTAs that the GPU holds at once.
template <int DH, int NQ>
double plan(const PromptAttnArgs& a, const int (&resident)[4], Launch& L, int& smem, int64_t& units) {
  using C = Cfg<DH, NQ>;
  L.G = a.Hq / a.Hkv;
  L.hc = (L.G + 127) / 128;
  L.Gc = (L.G + L.hc - 1) / L.hc;
  L.T = 128 / L.Gc;
  L.per = a.Hkv * L.hc;
  L.gc_inv = L.Gc > 1 ? (uint32_t)(((1ull << 32) + L.Gc - 1) / L.Gc) : 0;
  // sequences with queries, longest key ranges first
  int n = 0;
  for (int b = 0; b < a.batch; ++b)
    if (a.cu_q[b + 1] > a.cu_q[b]) {
      int i = n++;
      for (; i > 0 && a.kv_len[L.order[i - 1]] < a.kv_len[b]; --i) L.order[i] = L.order[i - 1];
      L.order[i] = (uint8_t)b;
    }
  L.n_order = n;
  units = 0;
  double steps = 0;  // key tiles of all units
  const int longest = (a.kv_len[L.order[0]] + C::BK - 1) / C::BK;  // of one unit
  for (int i = 0; i < n; ++i) {
    const int b = L.order[i], tok = a.cu_q[b + 1] - a.cu_q[b];
    L.work_cu[i] = (int)units;
    const int64_t mine = (int64_t)((tok + L.T * C::NQ - 1) / (L.T * C::NQ)) * a.Hkv * L.hc;
    steps += (double)mine * (a.causal ? a.kv_len[b] - 0.5 * tok : a.kv_len[b]) / C::BK + 0.5 * mine;
    units += mine;
    if (units > 0x7fffffff / 8) return -1;
  }
  L.work_cu[n] = (int)units;
  L.per_inv = L.per > 1 && units * L.per < ((int64_t)1 << 32) ? (uint32_t)(((1ull << 32) + L.per - 1) / L.per) : 0;
  // Split the keys of a unit over the CTAs of a cluster where that shortens the
  // launch: the longest unit, or all units over the SMs, whichever is more, in
  // clocks from measured costs of a key tile (alone; beside a second CTA of the
  // SM), of a unit's start and end, and of a merge (less where SMs are left to
  // halve the value dims).  Equal units run in whole rounds, those of a causal
  // prompt, longest first, fill the SMs but for an overhang.  At head_dim 64 the
  // split CTAs have a SM each while there are as many, else two share one.
  // Measured, chosen against other: 16 rows over 1016 keys 32/8/128 8.4 split by
  // 4, 14.6 unsplit; 400 tokens 10.8 unsplit, 13.7 split by 2; 8192 tokens 4/1/64
  // 45 split by 2, 54.5 unsplit, 12/4/64 101 unsplit, 128 split by 2.
  const double tile = DH == 64 ? 1150 : (DH == 128 && NQ == 1 ? 1450 : 2700), shared = 1560;
  const double ends = DH == 128 && NQ == 1 ? 7000 : 8500, overhang = 0.35;
  double best = 0;
  smem = C::BYTES;
  L.split = L.vs = 1;
  for (int e = 0; e < 4; ++e) {
    const int n = 1 << e, clusters = resident[e];
    if (clusters == 0 || longest < 2 * n - 1) continue;
    const bool pairs = C::CTAS == 2 && (n == 1 || units > clusters);
    const double ctas = (double)(clusters << e) * (pairs ? 2 : 1);  // at once
    const int vs = C::VS && units * n * 2 <= ctas ? 2 : 1;
    const double merge = n == 1 ? 0 : (DH > 64 ? 3000 + (3000 + 10000.0 / n) * (NQ * DH / 256.0) : (pairs ? 4000 + 1000 * n : 6000));
    const double own = (ends + merge) * (vs == 2 ? 0.6 : 1);
    const double chain = own + tile * ((longest + n - 1) / n);
    const double mean = own + (pairs ? shared : tile) * steps / ((double)units * n);
    double rounds = (double)units * n / ctas;
    if (!pairs) {
      const double even = fmax(0.0, fmin(1.0, 2 * mean / chain - 1));  // 1: equal units
      rounds = even * ceil(rounds) + (1 - even) * fmin(ceil(rounds), rounds + overhang);
    } else if (rounds > 1) {
      rounds += overhang;
    }
    const double all = rounds * mean;
    const double cost = chain > all ? chain : all;
    if (e == 0 || cost < best) {
      best = cost;
      L.split = n;
      L.vs = vs;
      smem = n > 1 && !pairs ? C::SPLIT_BYTES : C::BYTES;
    }
  }
  // over the queries themselves the halves would not start with the same queries
  if (a.out == a.q) L.vs = 1;
  return best;
}

template <int DH, int NQ>
cudaError_t run(const PromptAttnArgs& a, const Launch& L, int smem, int64_t units, cudaStream_t st) {
  using C = Cfg<DH, NQ>;
  CUtensorMap qmap, kmap, vmap, omap;
  cudaError_t e = make_bf16_3d_map(&qmap, a.q, {DH, a.Hq, a.cu_q[a.batch]}, {DH, (long)a.q_stride}, {64, L.Gc, L.T});
  if (e == cudaSuccess)
    e = make_bf16_3d_map(&omap, a.out, {DH, a.Hq, a.cu_q[a.batch]}, {DH, (long)a.out_stride}, {64, L.Gc, L.T});
  if (e == cudaSuccess)
    e = make_bf16_3d_map(&kmap, a.k, {64, (long)a.cache_rows, (long)a.Hkv * C::DB}, {(long)a.kv_stride, 64},
                         {64, C::BK, C::DBK});
  if (e == cudaSuccess)
    e = make_bf16_3d_map(&vmap, a.v, {64, (long)a.cache_rows, (long)a.Hkv * C::DB}, {(long)a.kv_stride, 64},
                         {64, C::BKV, C::DB / L.vs});
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * L.split * L.vs));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)L.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = L.split > 1 ? 1 : 0;
  return a.key_mask ? cudaLaunchKernelEx(&cfg, k_prompt_attn<DH, NQ, true>, qmap, kmap, vmap, omap, a, L)
                    : cudaLaunchKernelEx(&cfg, k_prompt_attn<DH, NQ, false>, qmap, kmap, vmap, omap, a, L);
}

template <int DH>
cudaError_t launch(const PromptAttnArgs& a, const int (&resident)[4], cudaStream_t st) {
  constexpr int NQ = DH == 128 ? 2 : 1;
  Launch L;
  int smem;
  int64_t units;
  const double cost = plan<DH, NQ>(a, resident, L, smem, units);
  if (cost < 0) return cudaErrorInvalidConfiguration;
  if (NQ == 2 && units <= 2 * resident[0]) {  // single tiles may fill the SMs better
    Launch L1;
    int smem1;
    int64_t units1;
    const double cost1 = plan<DH, 1>(a, resident, L1, smem1, units1);
    if (cost1 >= 0 && cost1 < cost) return run<DH, 1>(a, L1, smem1, units1, st);
  }
  return run<DH, NQ>(a, L, smem, units, st);
}

}  // namespace

cudaError_t launch_prompt_attention(const PromptAttnArgs& a, int dh, const int (&resident)[4], cudaStream_t s) {
  if (dh == 64) return launch<64>(a, resident, s);
  if (dh == 128) return launch<128>(a, resident, s);
  return launch<256>(a, resident, s);
}

template <int DH, int NQ>
static cudaError_t setup(int (&resident)[4]) {
  using C = Cfg<DH, NQ>;
  cudaError_t e = cudaSuccess;
  for (auto kern : {k_prompt_attn<DH, NQ, false>, k_prompt_attn<DH, NQ, true>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SPLIT_BYTES);
  for (int i = 0; i < 4 && e == cudaSuccess; ++i) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(8);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SPLIT_BYTES;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 1u << i;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&resident[i], k_prompt_attn<DH, NQ, false>, &cfg);
  }
  return e;
}

cudaError_t prompt_kernel_setup(int dh, int (&resident)[4]) {
  if (dh == 64) return setup<64, 1>(resident);
  if (dh == 256) return setup<256, 1>(resident);
  const cudaError_t e = setup<128, 1>(resident);  // a SM each in single tiles and in pairs: the same counts
  return e == cudaSuccess ? setup<128, 2>(resident) : e;
}

}  // namespace ae
