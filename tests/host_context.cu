// Test helper: a context with head sizes and no GPU behind it, so that the
// host-side checks of the library's entry points run on a machine without one.
// Every call made on it must be refused before its first CUDA call.
#include "../flow_matching_action_gb300/csrc/ae_internal.h"

extern "C" __attribute__((visibility("default"))) void* host_context(int hq, int hkv, int dh, int bf16) {
  ae_ctx* c = new ae_ctx();
  c->d = ae::Dims{1, 128, 128, hq, hkv, dh, 8, 1, 1e-6, 1e4, 4e-3, 4.0, bf16 ? AE_DTYPE_BF16 : AE_DTYPE_F32, 0};
  c->fast = bf16 != 0;
  c->max_batch = 4;
  return c;
}

extern "C" __attribute__((visibility("default"))) void host_context_free(void* c) { delete (ae_ctx*)c; }
