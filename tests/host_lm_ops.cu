// Test helper: the entry points of the language-model operators over launches
// that only record what they are given, so that the calls they accept are tested
// on a machine without a GPU (and touch no GPU on one that has it).
#include <cuda_runtime.h>

static cudaError_t host_device(int* dev) {
  *dev = 0;
  return cudaSuccess;
}
#define cudaGetDevice host_device
#include "../flow_matching_action_gb300/csrc/ae_lm_ops.cu"
#undef cudaGetDevice

#include <string.h>

#define HOST_API extern "C" __attribute__((visibility("default")))

static ae::RopeNormArgs g_rope;
static ae::PromptAttnArgs g_prompt;
static ae::TokenAttnArgs g_token;
static int g_launches, g_clusters;

namespace ae {
cudaError_t launch_qk_norm_rope(const RopeNormArgs& a, int, int, cudaStream_t) {
  g_rope = a;
  ++g_launches;
  return cudaSuccess;
}
cudaError_t launch_prompt_attention(const PromptAttnArgs& a, int, const int (&resident)[4], cudaStream_t) {
  g_prompt = a;
  g_clusters = resident[0];
  ++g_launches;
  return cudaSuccess;
}
cudaError_t launch_token_attention(const TokenAttnArgs& a, int, int, cudaStream_t) {
  g_token = a;
  ++g_launches;
  return cudaSuccess;
}
ae_status ensure_time_table(ae_ctx*, int, const TimeTable**) { return AE_ERR_UNSUPPORTED; }
int launch_step_fast(ae_ctx*, const TimeTable&, int, float*, cudaStream_t, cudaError_t*, const AttnScratch*,
                     const PrefillOut*) {
  return 0;
}
}  // namespace ae

HOST_API void* host_context(int hq, int hkv, int dh) {
  ae_ctx* c = new ae_ctx();
  c->d = ae::Dims{1, 128, 128, hq, hkv, dh, 8, 1, 1e-6, 1e4, 4e-3, 4.0, AE_DTYPE_BF16, 0};
  c->fast = true;
  c->max_batch = 4;
  c->device = 0;
  return c;
}
HOST_API void host_context_free(void* c) { delete (ae_ctx*)c; }
HOST_API ae_status ae_last_error(const ae_ctx* c, char* buf, size_t n) {
  if (n > 0) {
    strncpy(buf, c ? c->last_msg.c_str() : "", n - 1);
    buf[n - 1] = 0;
  }
  return AE_OK;
}
HOST_API void host_set_clusters(void* c, int n) { ((ae_ctx*)c)->prompt_resident[0] = n; }
HOST_API int host_clusters() { return g_clusters; }
HOST_API int host_launches() { return g_launches; }
HOST_API const void* host_rope_rows(int64_t* q_stride, int64_t* qkv_stride) {
  *q_stride = g_rope.q_stride;
  *qkv_stride = g_rope.qkv_stride;
  return g_rope.q_out;
}
HOST_API uint64_t host_turn_fraction(double radians) { return ae::turn_fraction(radians); }
