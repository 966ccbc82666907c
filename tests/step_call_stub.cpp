// Stands in for the library under the module of the calls around the paged cache on a host without a GPU: each entry
// point counts its calls and returns the status that the test asked for.  Test infrastructure: built and driven by
// tests/test_step_host.py.
#include "keops_mi355x.h"

namespace {
int g_status = 0, g_calls = 0;
int answer() {
  ++g_calls;
  return g_status;
}
}  // namespace

extern "C" {
void stub_set(int status) {
  g_status = status;
  g_calls = 0;
}
int stub_calls() { return g_calls; }

int keops_rotary(const void *, int64_t, int32_t, int64_t, int32_t, int32_t, const int32_t *, const keops_rotary_t *, int32_t, void *,
                 int64_t, void *) {
  return answer();
}
int keops_cache_append_rotary(const keops_cache_t *, const void *, const void *, const void *, int64_t, int64_t, int64_t, int32_t, int32_t,
                              const int32_t *, int64_t, const int32_t *, const keops_rotary_t *, void *, int64_t, void *) {
  return answer();
}
int keops_cache_read(const keops_cache_t *, void *, void *, int64_t, int64_t, int32_t, const int32_t *, int64_t, void *) { return answer(); }
int keops_adjust_logits(const void *, int64_t, int32_t, int64_t, int32_t, const keops_logit_rules_t *, void *, int64_t, void *) {
  return answer();
}
}
