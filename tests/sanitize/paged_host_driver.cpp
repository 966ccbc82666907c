// Drives the host side of the paged cache's C ABI (validation, launch plans, workspace sizes) in a
// sanitizer build, on a host without a GPU: every call fails validation or reaches the first HIP
// call, which fails without a device.  Addresses are stand-ins that validation never
// dereferences.  Test infrastructure: built and run by tests/test_sanitizers_paged.py.
#include <cstdint>
#include <cstdio>
#include <random>

#include <hip/hip_runtime_api.h>

#include "keops_mi355x.h"

int main() {
  int ndev = 0;
  if (hipGetDeviceCount(&ndev) == hipSuccess && ndev > 0) {
    std::printf("skipped: a GPU is visible\n");
    return 77;
  }
  std::mt19937_64 rng(1);
  const int64_t odd[] = {-1, 0, 1, 2, 7, 8, 16, 63, 64, 96, 128, 255, 256, 4096, 65535, 65536, 1 << 20, 1 << 30,
                         0x7fffffffLL, 0x80000000LL, (int64_t)1 << 40, (int64_t)1 << 62, INT64_MIN, INT64_MAX};
  const auto pick = [&] { return odd[rng() % (sizeof(odd) / sizeof(odd[0]))]; };
  const auto address = [&](unsigned k) { return rng() % 8 ? (void *)(uintptr_t)(((uint64_t)(k + 1) << 44) + (rng() % 4 ? 0 : rng() % 64)) : nullptr; };
  long counts[8] = {0};
  for (int i = 0; i < 400000; ++i) {
    keops_cache_t c{};
    const bool wild = rng() % 2;
    c.k_pages = address(0);
    c.v_pages = address(1);
    c.weights = rng() % 2 ? (float *)address(2) : nullptr;
    c.k_scale = (const float *)address(3);
    c.v_scale = (const float *)address(4);
    c.pages = wild ? pick() : 100;
    c.page_size = wild ? (int32_t)pick() : 16;
    c.heads = wild ? (int32_t)pick() : 4;
    c.dim = rng() % 3 ? 128 : (int32_t)pick();
    c.type = (int32_t)(rng() % 4);
    c.slot_stride = wild ? pick() : 512;
    c.page_stride = wild ? pick() : 512 * 16;
    c.head_stride = wild ? pick() : 128;
    c.page_table = (const int32_t *)address(5);
    c.table_stride = wild ? pick() : 8;
    c.table_width = wild ? (int32_t)pick() : 8;
    c.lens = (const int32_t *)address(6);
    c.seqs = wild ? (int32_t)pick() : 3;
    const int type = (int)(rng() % 3);
    int rc = 0;
    int64_t bytes = 0;
    switch (rng() % 5) {
      case 0:
        rc = keops_cache_append(rng() % 16 ? &c : nullptr, address(7), address(8), wild ? pick() : 512, wild ? pick() : 512, type,
                                (const int32_t *)address(9), wild ? pick() : 9, nullptr);
        break;
      case 1:
        rc = keops_paged_attention(rng() % 16 ? &c : nullptr, address(7), wild ? pick() : 1024, type, wild ? (int)pick() : 8,
                                   (const int32_t *)address(9), wild ? pick() : 9, wild ? (int)pick() : 3, wild ? (int)pick() : 100,
                                   rng() % 8 ? 0.1f : 0.0f / 0.0f, wild ? (int)pick() : 0, 0.0f, address(10), (float *)address(11),
                                   rng() % 2 ? address(12) : nullptr, pick(), nullptr);
        break;
      case 2:
        rc = keops_paged_attention_workspace(&c, type, wild ? (int)pick() : 8, wild ? pick() : 9, wild ? (int)pick() : 3,
                                             wild ? (int)pick() : 100, wild ? (int)pick() : 0, rng() % 16 ? &bytes : nullptr);
        break;
      case 3:
        rc = keops_cache_evict(rng() % 16 ? &c : nullptr, (const int32_t *)address(7), wild ? pick() : 8, wild ? (int)pick() : 8,
                               wild ? (int)pick() : 40, wild ? (int)pick() : 2, wild ? (int)pick() : 3, (int32_t *)address(10),
                               (int32_t *)address(11), nullptr);
        break;
      default: {
        const int S = wild ? (int)pick() : 3, K = wild ? (int)pick() : 2, V = wild ? (int)pick() : 100;
        rc = keops_verify_draft((const float *)address(0), (const float *)address(1), (const int32_t *)address(2),
                                (const int32_t *)address(3), (const float *)address(4), (const float *)address(5), S, K, V,
                                (int32_t *)address(6), (int32_t *)address(7), rng() % 2 ? address(8) : nullptr, pick(), nullptr);
        if (rc == KEOPS_OK || rc == KEOPS_ERR_HIP) rc = keops_verify_draft_workspace(S, K, V, rng() % 16 ? &bytes : nullptr);
      }
    }
    if (rc > 0 || rc < -5) {
      std::fprintf(stderr, "call %d returned %d\n", i, rc);
      return 1;
    }
    ++counts[-rc];
  }
  std::printf("ok: %ld no-ops, %ld invalid, %ld unsupported, %ld without memory, %ld up to the first HIP call, %ld short workspaces\n",
              counts[0], counts[1], counts[2], counts[3], counts[4], counts[5]);
  return counts[1] > 0 && counts[4] > 0 ? 0 : 1;
}
