// Drives the host side of the C ABI around the paged cache (rotary positions, the rotating append, reading, logits) in a
// sanitizer build, on a host without a GPU: every call fails validation or reaches the first HIP call, which fails
// without a device.  Addresses are stand-ins that validation never dereferences.  Test infrastructure: built and
// run by tests/test_sanitizers_step.py.
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
    const bool wild = rng() % 2;
    keops_cache_t c{};
    c.type = (int32_t)(rng() % 6) - (rng() % 16 == 0);
    c.k_pages = address(0);
    c.v_pages = address(1);
    c.weights = rng() % 2 ? (float *)address(2) : nullptr;
    c.k_powers = (uint8_t *)address(3);
    c.v_powers = (uint8_t *)address(4);
    c.pages = wild ? pick() : 100;
    c.page_size = wild ? (int32_t)pick() : 16;
    c.heads = wild ? (int32_t)pick() : 4;
    c.dim = rng() % 3 ? 128 : (int32_t)pick();
    c.slot_stride = wild ? pick() : 512;
    c.page_stride = wild ? pick() : 512 * 16;
    c.head_stride = wild ? pick() : 128;
    c.page_table = (const int32_t *)address(5);
    c.table_stride = wild ? pick() : 8;
    c.table_width = wild ? (int32_t)pick() : 8;
    c.lens = (const int32_t *)address(6);
    c.seqs = wild ? (int32_t)pick() : 3;
    keops_rotary_t r{(const double *)address(13), rng() % 8 ? 1.0 : 0.0 / 0.0, wild ? (int32_t)pick() : 32, (int32_t)(rng() % 2)};
    const int type = (int)(rng() % 4);
    const auto n = [&](int64_t plain) { return wild ? pick() : plain; };
    int rc = 0;
    switch (rng() % 6) {
      case 0:
        rc = keops_rotary(address(7), n(1024), type, n(9), (int32_t)n(8), (int32_t)n(128), (const int32_t *)address(8), rng() % 16 ? &r : nullptr,
                          0, address(rng() % 4 ? 9 : 7), n(1024), nullptr);
        break;
      case 1:
        rc = keops_cache_append_rotary(rng() % 16 ? &c : nullptr, address(7), address(8), address(9), n(1024), n(512), n(512), type, (int32_t)n(8),
                                       (const int32_t *)address(10), n(9), rng() % 2 ? (const int32_t *)address(11) : nullptr,
                                       rng() % 16 ? &r : nullptr, address(12), n(1024), nullptr);
        break;
      case 2:
        rc = keops_cache_read(rng() % 16 ? &c : nullptr, address(7), address(8), n(512), n(512), type, (const int32_t *)address(9), n(9), nullptr);
        break;
      case 3:
        rc = keops_cache_append(&c, address(7), address(8), n(512), n(512), type, (const int32_t *)address(9), n(9), nullptr);
        break;
      case 4: {
        int64_t bytes = 0;
        c.type = KEOPS_TYPE_E2M1;
        rc = keops_paged_attention_workspace(&c, type, (int32_t)n(8), n(9), (int32_t)n(3), (int32_t)n(100), (int32_t)n(0), &bytes);
        break;
      }
      default: {
        keops_logit_rules_t u{};
        u.starts = (const int32_t *)address(0);
        u.text = rng() % 2 ? (const int32_t *)address(1) : nullptr;
        u.text_stride = n(50);
        u.lens = (const int32_t *)address(2);
        u.repetition = rng() % 2 ? (const float *)address(3) : nullptr;
        u.bias_tokens = (const int32_t *)address(4);
        u.bias = (const float *)address(5);
        u.mask = rng() % 2 ? (const int32_t *)address(6) : nullptr;
        u.mask_stride = n(4);
        u.seqs = (int32_t)n(3);
        u.text_width = (int32_t)n(50);
        u.biases = (int32_t)n(6);
        rc = keops_adjust_logits(address(7), n(100), type, n(9), (int32_t)n(100), rng() % 16 ? &u : nullptr, address(rng() % 4 ? 8 : 7), n(100), nullptr);
      }
    }
    if (rc > 0 || rc < -5) {
      std::fprintf(stderr, "call %d returned %d\n", i, rc);
      return 1;
    }
    ++counts[-rc];
  }
  std::printf("ok: %ld no-ops, %ld invalid, %ld unsupported, %ld without memory, %ld up to the first HIP call\n", counts[0], counts[1],
              counts[2], counts[3], counts[4]);
  return counts[1] > 0 && counts[4] > 0 ? 0 : 1;
}
