// Stands in for the library under the paged calls' module on a host without a GPU: each entry
// point counts its calls and returns the status that the test asked for.  Test infrastructure: built
// and driven by tests/test_paged_call_host.py.
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

int keops_cache_append(const keops_cache_t *, const void *, const void *, int64_t, int64_t, int32_t, const int32_t *, int64_t,
                       void *) {
  return answer();
}
int keops_paged_attention(const keops_cache_t *, const void *, int64_t, int32_t, int32_t, const int32_t *, int64_t, int32_t,
                          int32_t, float, int32_t, float, void *, float *, void *, int64_t, void *) {
  return answer();
}
int keops_cache_evict(const keops_cache_t *, const int32_t *, int64_t, int32_t, int32_t, int32_t, int32_t, int32_t *, int32_t *,
                      void *) {
  return answer();
}
int keops_verify_draft(const float *, const float *, const int32_t *, const int32_t *, const float *, const float *, int32_t,
                       int32_t, int32_t, int32_t *, int32_t *, void *, int64_t, void *) {
  return answer();
}
}
