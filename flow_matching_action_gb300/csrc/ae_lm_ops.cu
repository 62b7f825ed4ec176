// Entry points of the language-model attention operators: argument checks and
// the launch arguments.  Everything a caller can get wrong on the host is
// refused here, before any CUDA call.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "ae_internal.h"

namespace {

ae_status fail(ae_ctx* c, ae_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  c->last_msg = buf;
  return st;
}

#define AE_TRY(expr)                 \
  do {                               \
    const ae_status s_ = (expr);     \
    if (s_ != AE_OK) return s_;      \
  } while (0)

// bf16 rows of `width` elements: 16-byte aligned base, stride a multiple of 8 and >= width.
ae_status check_rows(ae_ctx* c, const char* name, const void* p, int64_t stride, int64_t width) {
  if (p == nullptr) return fail(c, AE_ERR_INVALID_ARG, "%s is NULL", name);
  if ((uintptr_t)p % 16 != 0) return fail(c, AE_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  if (stride < width)
    return fail(c, AE_ERR_SHAPE, "%s: row stride %lld < row length %lld", name, (long long)stride, (long long)width);
  if (stride % 8 != 0)
    return fail(c, AE_ERR_INVALID_ARG, "%s: row stride %lld is not a multiple of 8", name, (long long)stride);
  // a TMA row stride has 40 bits
  if (stride > ((int64_t)1 << 38))
    return fail(c, AE_ERR_SHAPE, "%s: row stride %lld is too large", name, (long long)stride);
  return AE_OK;
}

// Written over its input, a row must land on itself (one row does, whatever the
// strides are): on another row it would replace what is still to be read.
ae_status check_in_place(ae_ctx* c, const char* out_name, const void* out, int64_t out_stride, const char* in_name,
                         const void* in, int64_t in_stride, int rows) {
  if (out == in && rows > 1 && out_stride != in_stride)
    return fail(c, AE_ERR_INVALID_ARG, "%s is %s but the row strides differ", out_name, in_name);
  return AE_OK;
}

// Row counts travel as 32-bit TMA coordinates.
ae_status check_cache_rows(ae_ctx* c, int64_t rows) {
  if (rows < 0 || rows > 0x7fffff00LL)
    return fail(c, AE_ERR_SHAPE, "cache_rows %lld outside 0..%lld", (long long)rows, 0x7fffff00LL);
  return AE_OK;
}

ae_status check_scale(ae_ctx* c, float scale) {
  if (!(scale >= 0.f) || isinf(scale)) return fail(c, AE_ERR_INVALID_ARG, "scale must be finite and >= 0");
  return AE_OK;
}

ae_status check_rotation(ae_ctx* c, int n_axes, const uint8_t* pair_axis, const double* pair_freq) {
  const int half = c->d.dh / 2;
  if (n_axes < 1 || n_axes > AE_MAX_AXES)
    return fail(c, AE_ERR_SHAPE, "n_axes %d outside 1..%d", n_axes, AE_MAX_AXES);
  if (pair_axis != nullptr)
    for (int j = 0; j < half; ++j)
      if (pair_axis[j] >= n_axes)
        return fail(c, AE_ERR_INVALID_ARG, "pair_axis[%d] = %d, n_axes is %d", j, pair_axis[j], n_axes);
  if (pair_freq != nullptr)
    for (int j = 0; j < half; ++j)
      if (!isfinite(pair_freq[j])) return fail(c, AE_ERR_INVALID_ARG, "pair_freq[%d] is not finite", j);
  return AE_OK;
}

void set_rotation(const ae_ctx* c, ae::RopeNormArgs* a, const uint8_t* pair_axis, const double* pair_freq) {
  a->turn_table = pair_freq ? nullptr : c->rope_turn;
  for (int j = 0; j < c->d.dh / 2; ++j) {
    a->axis[j] = pair_axis ? pair_axis[j] : 0;
    a->turn[j] = pair_freq ? ae::turn_fraction(pair_freq[j]) : 0;
  }
}

// Checks common to the operators.  `op` names the call.
ae_status check_context(ae_ctx* c, const void* args, const char* op) {
  if (args == nullptr) return fail(c, AE_ERR_INVALID_ARG, "%s: args is NULL", op);
  if (!c->fast) return fail(c, AE_ERR_UNSUPPORTED, "%s runs on bf16 contexts only", op);
  if (c->status_host && *(volatile int*)c->status_host)
    return fail(c, AE_ERR_DEVICE, "a device-side check failed earlier (code %d)", *c->status_host);
  return AE_OK;
}

// The last check: the first CUDA call.
ae_status check_device(ae_ctx* c) {
  int dev = -1;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(c, AE_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev != c->device)
    return fail(c, AE_ERR_INVALID_ARG, "device %d is current, the context lives on device %d", dev, c->device);
  return AE_OK;
}

ae_status launched(ae_ctx* c, cudaError_t e, const char* op) {
  if (e != cudaSuccess) return fail(c, AE_ERR_CUDA, "%s launch: %s", op, cudaGetErrorString(e));
  return AE_OK;
}

}  // namespace

namespace ae {

uint64_t turn_fraction(double radians) {
  // 1 / (2 pi) as the sum of two doubles: the product is good to 2^-63 of a turn for
  // every frequency up to 2^30 radians.  Of the magnitude, the sign last: dropping the
  // whole turns of a negative product near zero would round it (to 2^-54 of a turn).
  const double hi = 0x1.45f306dc9c883p-3, lo = -0x1.6b01ec5417056p-57;
  const double r = fabs(radians), turns = r * hi;
  const double frac = turns - floor(turns);  // exact, in [0, 1)
  double rest = fma(r, hi, -turns) + r * lo;
  rest -= rint(rest);
  if (rest >= 0.5) rest -= 1.0;
  const double top = floor(frac * 4294967296.0);
  const double low = (frac * 4294967296.0 - top) * 4294967296.0;
  const uint64_t t =
      ((uint64_t)top << 32) + (uint64_t)low + (uint64_t)(int64_t)(rest * 18446744073709551616.0);
  return radians < 0 ? 0 - t : t;
}

}  // namespace ae

extern "C" {

ae_status ae_qk_norm_rope(ae_ctx* c, const ae_qk_norm_rope_args* p) {
  if (c == nullptr) return AE_ERR_INVALID_ARG;
  const char* op = "ae_qk_norm_rope";
  AE_TRY(check_context(c, p, op));
  const ae::Dims& d = c->d;
  if (p->tokens < 0 || p->tokens > 0x7fff0000) return fail(c, AE_ERR_SHAPE, "tokens %d outside 0..%d", p->tokens, 0x7fff0000);
  if (!isfinite(p->norm_offset)) return fail(c, AE_ERR_INVALID_ARG, "norm_offset must be finite");
  AE_TRY(check_cache_rows(c, p->cache_rows));
  AE_TRY(check_rotation(c, p->n_axes, p->pair_axis, p->pair_freq));
  if (p->tokens == 0) return AE_OK;
  if (p->kv_rows == nullptr && p->tokens > p->cache_rows)
    return fail(c, AE_ERR_SHAPE, "%d tokens, %lld cache rows", p->tokens, (long long)p->cache_rows);
  AE_TRY(check_rows(c, "qkv", p->qkv, p->qkv_stride, d.qkvdim()));
  AE_TRY(check_rows(c, "q_out", p->q_out, p->q_stride, d.qdim()));
  if (p->cache_rows > 0) {  // without rows nothing is stored
    AE_TRY(check_rows(c, "k_cache", p->k_cache, p->kv_stride, d.kvdim()));
    AE_TRY(check_rows(c, "v_cache", p->v_cache, p->kv_stride, d.kvdim()));
  }
  AE_TRY(check_in_place(c, "q_out", p->q_out, p->q_stride, "qkv", p->qkv, p->qkv_stride, p->tokens));
  for (const void* w : {p->q_norm, p->k_norm})
    if ((uintptr_t)w % 16 != 0) return fail(c, AE_ERR_INVALID_ARG, "a norm weight is not 16-byte aligned");
  if (p->positions == nullptr) return fail(c, AE_ERR_INVALID_ARG, "positions is NULL");
  if ((uintptr_t)p->positions % 4 != 0 || (uintptr_t)p->kv_rows % 8 != 0)
    return fail(c, AE_ERR_INVALID_ARG, "positions / kv_rows is not aligned to its elements");
  AE_TRY(check_device(c));
  ae::RopeNormArgs a;
  a.tokens = p->tokens;
  a.n_axes = p->n_axes;
  a.Hq = d.Hq;
  a.Hkv = d.Hkv;
  a.qkv = (const ae::bf16*)p->qkv;
  a.qkv_stride = p->qkv_stride;
  a.q_norm = (const ae::bf16*)p->q_norm;
  a.k_norm = (const ae::bf16*)p->k_norm;
  a.norm_offset = p->norm_offset;
  a.eps = (float)d.eps;
  a.positions = p->positions;
  a.kv_rows = p->kv_rows;
  a.cache_rows = p->cache_rows;
  a.q_out = (ae::bf16*)p->q_out;
  a.q_stride = p->q_stride;
  a.k_cache = (ae::bf16*)p->k_cache;
  a.v_cache = (ae::bf16*)p->v_cache;
  a.kv_stride = p->kv_stride;
  a.status = c->status_dev;
  set_rotation(c, &a, p->pair_axis, p->pair_freq);
  return launched(c, ae::launch_qk_norm_rope(a, d.dh, c->sm_count, c->stream), op);
}

ae_status ae_prompt_attention(ae_ctx* c, const ae_prompt_attention_args* p) {
  if (c == nullptr) return AE_ERR_INVALID_ARG;
  const char* op = "ae_prompt_attention";
  AE_TRY(check_context(c, p, op));
  const ae::Dims& d = c->d;
  if (p->batch < 0 || p->batch > AE_MAX_BATCH)
    return fail(c, AE_ERR_SHAPE, "batch %d outside 0..%d", p->batch, AE_MAX_BATCH);
  AE_TRY(check_scale(c, p->scale));
  AE_TRY(check_cache_rows(c, p->cache_rows));
  if (p->batch == 0) return AE_OK;
  if (p->cu_q == nullptr) return fail(c, AE_ERR_INVALID_ARG, "cu_q is NULL");
  if ((p->kv_row0 == nullptr) != (p->kv_len == nullptr))
    return fail(c, AE_ERR_INVALID_ARG, "kv_row0 and kv_len come together");
  if (p->cu_q[0] != 0) return fail(c, AE_ERR_SHAPE, "cu_q[0] must be 0");
  ae::PromptAttnArgs a;
  for (int b = 0; b < p->batch; ++b) {
    const int64_t n = (int64_t)p->cu_q[b + 1] - p->cu_q[b];
    if (n < 0) return fail(c, AE_ERR_SHAPE, "cu_q decreases at sequence %d", b);
    const int64_t r0 = p->kv_row0 ? p->kv_row0[b] : p->cu_q[b];
    const int64_t m = p->kv_len ? p->kv_len[b] : n;
    if (m < n)
      return fail(c, AE_ERR_SHAPE, "sequence %d has %lld queries but %lld keys", b, (long long)n, (long long)m);
    // m - n keys without queries are never read, but a range is a range
    if (r0 < 0 || r0 > p->cache_rows || m > p->cache_rows - r0)
      return fail(c, AE_ERR_SHAPE, "sequence %d: cache rows %lld .. +%lld outside 0..%lld", b, (long long)r0,
                  (long long)m, (long long)p->cache_rows);
    a.cu_q[b] = p->cu_q[b];
    a.kv_row0[b] = r0;
    a.kv_len[b] = (int)m;
  }
  a.cu_q[p->batch] = p->cu_q[p->batch];
  const int total = p->cu_q[p->batch];
  if (total == 0) return AE_OK;
  if ((int64_t)total * (d.Hq / d.Hkv) > 0x7fffff00LL)
    return fail(c, AE_ERR_SHAPE, "%d query rows are too many", total);
  AE_TRY(check_rows(c, "q", p->q, p->q_stride, d.qdim()));
  AE_TRY(check_rows(c, "out", p->out, p->out_stride, d.qdim()));
  AE_TRY(check_in_place(c, "out", p->out, p->out_stride, "q", p->q, p->q_stride, total));
  AE_TRY(check_rows(c, "k", p->k, p->kv_stride, d.kvdim()));
  AE_TRY(check_rows(c, "v", p->v, p->kv_stride, d.kvdim()));
  AE_TRY(check_device(c));
  a.batch = p->batch;
  a.causal = p->causal != 0;
  a.Hq = d.Hq;
  a.Hkv = d.Hkv;
  a.cache_rows = p->cache_rows;
  a.q = (const ae::bf16*)p->q;
  a.k = (const ae::bf16*)p->k;
  a.v = (const ae::bf16*)p->v;
  a.q_stride = p->q_stride;
  a.kv_stride = p->kv_stride;
  a.out_stride = p->out_stride;
  a.key_mask = p->key_mask;
  a.scale = p->scale > 0.f ? p->scale : (float)(1.0 / sqrt((double)d.dh));
  a.out = (ae::bf16*)p->out;
  a.status = c->status_dev;
  return launched(c, ae::launch_prompt_attention(a, d.dh, c->prompt_resident, c->stream), op);
}

ae_status ae_token_attention(ae_ctx* c, const ae_token_attention_args* p) {
  if (c == nullptr) return AE_ERR_INVALID_ARG;
  const char* op = "ae_token_attention";
  AE_TRY(check_context(c, p, op));
  const ae::Dims& d = c->d;
  if (p->batch < 0 || p->batch > AE_MAX_TOKENS)
    return fail(c, AE_ERR_SHAPE, "batch %d outside 0..%d", p->batch, AE_MAX_TOKENS);
  if (p->max_len < 0) return fail(c, AE_ERR_SHAPE, "max_len %d < 0", p->max_len);
  AE_TRY(check_scale(c, p->scale));
  AE_TRY(check_cache_rows(c, p->cache_rows));
  if (p->batch == 0) return AE_OK;
  if (p->kv_row0 == nullptr || p->kv_len == nullptr)
    return fail(c, AE_ERR_INVALID_ARG, "kv_row0 / kv_len is NULL");
  if ((uintptr_t)p->kv_row0 % 8 != 0 || (uintptr_t)p->kv_len % 4 != 0)
    return fail(c, AE_ERR_INVALID_ARG, "kv_row0 / kv_len is not aligned to its elements");
  AE_TRY(check_rows(c, "q", p->q, p->q_stride, d.qdim()));
  AE_TRY(check_rows(c, "out", p->out, p->out_stride, d.qdim()));
  AE_TRY(check_in_place(c, "out", p->out, p->out_stride, "q", p->q, p->q_stride, p->batch));
  if (p->cache_rows > 0) {
    AE_TRY(check_rows(c, "k", p->k, p->kv_stride, d.kvdim()));
    AE_TRY(check_rows(c, "v", p->v, p->kv_stride, d.kvdim()));
  }
  AE_TRY(check_device(c));
  ae::TokenAttnArgs a;
  a.batch = p->batch;
  a.max_len = p->max_len;
  a.Hq = d.Hq;
  a.Hkv = d.Hkv;
  a.kv_row0 = p->kv_row0;
  a.kv_len = p->kv_len;
  a.cache_rows = p->cache_rows;
  a.q = (const ae::bf16*)p->q;
  a.k = (const ae::bf16*)p->k;
  a.v = (const ae::bf16*)p->v;
  a.q_stride = p->q_stride;
  a.kv_stride = p->kv_stride;
  a.out_stride = p->out_stride;
  a.key_mask = p->key_mask;
  a.scale = p->scale > 0.f ? p->scale : (float)(1.0 / sqrt((double)d.dh));
  a.out = (ae::bf16*)p->out;
  a.status = c->status_dev;
  return launched(c, ae::launch_token_attention(a, d.dh, c->sm_count, c->stream), op);
}

ae_status ae_prefill_prompts(ae_ctx* c, const ae_prefill_prompts_args* p) {
  if (c == nullptr) return AE_ERR_INVALID_ARG;
  const char* op = "ae_prefill_prompts";
  AE_TRY(check_context(c, p, op));
  const ae::Dims& d = c->d;
  if (p->batch < 0 || p->batch > AE_MAX_BATCH)
    return fail(c, AE_ERR_SHAPE, "batch %d outside 0..%d", p->batch, AE_MAX_BATCH);
  if (!isfinite(p->norm_offset)) return fail(c, AE_ERR_INVALID_ARG, "norm_offset must be finite");
  AE_TRY(check_rotation(c, p->n_axes, p->pair_axis, p->pair_freq));
  if (p->batch == 0) return AE_OK;
  if (p->cu_lens == nullptr) return fail(c, AE_ERR_INVALID_ARG, "cu_lens is NULL");
  if (p->cu_lens[0] != 0) return fail(c, AE_ERR_SHAPE, "cu_lens[0] must be 0");
  ae::PromptAttnArgs at = {};
  for (int b = 0; b < p->batch; ++b) {
    if (p->cu_lens[b + 1] < p->cu_lens[b]) return fail(c, AE_ERR_SHAPE, "cu_lens decreases at sequence %d", b);
    at.cu_q[b] = p->cu_lens[b];
    at.kv_row0[b] = p->cu_lens[b];
    at.kv_len[b] = p->cu_lens[b + 1] - p->cu_lens[b];
  }
  const int total = p->cu_lens[p->batch];
  at.cu_q[p->batch] = total;
  if (total > (int64_t)c->max_batch * d.H)
    return fail(c, AE_ERR_SHAPE, "%d tokens > max_batch * horizon = %lld", total, (long long)c->max_batch * d.H);
  if (total == 0) return AE_OK;
  AE_TRY(check_rows(c, "embeddings", p->embeddings, d.D, d.D));
  AE_TRY(check_rows(c, "out_k", p->out_k, d.kvdim(), d.kvdim()));
  AE_TRY(check_rows(c, "out_v", p->out_v, d.kvdim(), d.kvdim()));
  if (p->positions == nullptr) return fail(c, AE_ERR_INVALID_ARG, "positions is NULL");
  if ((uintptr_t)p->positions % 4 != 0)
    return fail(c, AE_ERR_INVALID_ARG, "positions is not aligned to its elements");
  for (const void* const* w : {p->q_norm, p->k_norm})
    if (w != nullptr)
      for (int l = 0; l < d.L; ++l)
        if (w[l] == nullptr || (uintptr_t)w[l] % 16 != 0)
          return fail(c, AE_ERR_INVALID_ARG, "norm weight of layer %d is NULL or not 16-byte aligned", l);
  AE_TRY(check_device(c));
  const ae::TimeTable* t = nullptr;
  AE_TRY(ae::ensure_time_table(c, 1, &t));  // constant conditioning: the modulation biases

  ae::RopeNormArgs r = {};
  r.tokens = total;
  r.n_axes = p->n_axes;
  r.Hq = at.Hq = d.Hq;
  r.Hkv = at.Hkv = d.Hkv;
  r.qkv = (const ae::bf16*)c->qkv;
  r.qkv_stride = d.qkvdim();
  r.norm_offset = p->norm_offset;
  r.eps = (float)d.eps;
  r.positions = p->positions;
  r.cache_rows = total;
  r.q_out = (ae::bf16*)c->qkv;  // in place
  r.q_stride = d.qkvdim();
  r.kv_stride = d.kvdim();
  r.status = at.status = c->status_dev;
  set_rotation(c, &r, p->pair_axis, p->pair_freq);
  at.batch = p->batch;
  at.causal = p->causal != 0;
  at.cache_rows = total;
  at.q = (const ae::bf16*)c->qkv;
  at.q_stride = d.qkvdim();
  at.kv_stride = d.kvdim();
  at.out = (ae::bf16*)c->o;
  at.out_stride = d.qdim();
  at.key_mask = p->token_mask;
  at.scale = (float)(1.0 / sqrt((double)d.dh));
  ae::PrefillOut po{(const ae::bf16*)p->embeddings, (ae::bf16*)p->out_k, (ae::bf16*)p->out_v};
  po.rope = &r;
  po.attn = &at;
  po.q_norm = p->q_norm;
  po.k_norm = p->k_norm;
  cudaError_t e = cudaSuccess;
  c->launches_sample = ae::launch_step_fast(c, *t, 0, nullptr, c->stream, &e, nullptr, &po);
  return launched(c, e, op);
}

}  // extern "C"
