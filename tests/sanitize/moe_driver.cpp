// moe_driver.cpp -- drives the expert layer's C ABI (host side) through valid
// and refused calls over many sizes, and its fixed-divisor division through
// edge values, in a sanitized build.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../fp4_quantization_amd/csrc/ufp4_moe.hpp"
#include "../../include/ufp4.h"

namespace ufp4 {
extern int g_moe_calls;
}

static void require(bool ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "moe driver: %s\n", what);
    abort();
  }
}

template <typename T>
static T* at(uintptr_t a) {
  return reinterpret_cast<T*>(a);
}

int main() {
  using namespace ufp4;
  uint64_t seed = 1;
  auto next = [&]() { return (uint32_t)((seed = seed * 6364136223846793005ull + 1442695040888963407ull) >> 33); };
  for (uint32_t i = 0; i < 20000; ++i) {
    const uint32_t d = i < 5000 ? i + 1 : (next() >> (next() % 30)) % 0x3FFFFFFFu + 1;
    const FastDiv f = fast_div(d);
    for (uint32_t n : {0u, d - 1, d, d + 1, 2 * d - 1, next() & 0x7FFFFFFFu, 0x7FFFFFFFu, 0x7FFFFFFFu / d * d, 0x7FFFFFFFu / d * d - 1})
      if (n < 0x80000000u) require(f.div(n) == n / d, "division");
  }
  const uintptr_t P = (uintptr_t)1 << 40;
  const int64_t sizes[] = {-1, 0, 1, 2, 31, 32, 33, 1000, 4096, (1 << 25) - 32, 1 << 25, (int64_t)1 << 28, (int64_t)1 << 40, INT64_MAX};
  ufp4_config cfg{};
  ufp4_qtensor q{at<uint8_t>(P), at<uint8_t>(P), at<float>(P)};
  int ok = 0, refused = 0;
  auto count = [&](int rc) {
    require(rc >= 0 && rc <= 4, "status");
    (rc == 0 ? ok : refused)++;
  };
  for (int64_t a : sizes)
    for (int64_t b : sizes)
      for (int32_t s : {-1, 0, 1, 8, 1024, 1025, INT32_MAX})
        for (int32_t e : {0, 1, 64, 1023, 1024, INT32_MAX}) {
          const int64_t rows = ufp4_expert_rows(a, s, e, 16);
          require(rows >= 0, "rows");
          count(ufp4_expert_sort(at<int32_t>(P), a, s, s, e, 16, b, at<int64_t>(P), at<int32_t>(P), at<int32_t>(P), nullptr));
          count(ufp4_expert_dispatch(at<uint16_t>(P), a, b, b, s, at<int32_t>(P), at<int32_t>(P), a, at<uint16_t>(P), b, nullptr));
          count(ufp4_expert_combine(at<void>(P), 0, a, b, b, at<int32_t>(P), nullptr, a, s, at<void>(P), 1, b, nullptr));
          count(ufp4_expert_combine_backward(at<void>(P), 0, a, b, b, s, at<void>(P), 1, a, b, at<int32_t>(P), at<int32_t>(P),
                                             nullptr, at<void>(P), b, at<float>(P), nullptr));
          count(ufp4_gemm_grouped_nt(&cfg, a, b, 64, q, q, 0, at<int64_t>(P), e, at<void>(P), 0, b, nullptr));
          count(ufp4_gemm_grouped_nt(&cfg, 64, 64, a, q, q, 1, at<int64_t>(P), e, at<void>(P), 0, 64, nullptr));
          count(ufp4_gemm_grouped_dw(&cfg, a, b, 64, q, q, at<int64_t>(P), e, at<void>(P), 1, nullptr));
          count(ufp4_gemm_grouped_dw(&cfg, 16, 16, a, q, q, at<int64_t>(P), e, at<void>(P), 1, nullptr));
        }
  for (int64_t a : sizes)
    for (int64_t b : sizes)
      for (int f : {-1, 0, 1, 2}) {
        count(ufp4_checkpoint_save(at<uint16_t>(P), a, b, b, f, at<uint8_t>(P), at<uint16_t>(P), nullptr));
        count(ufp4_checkpoint_load(at<uint8_t>(P), at<uint16_t>(P), a, b, f, at<void>(P), f, b, nullptr));
        const int64_t two = b > 0 && b < ((int64_t)1 << 50) ? 2 * b : b;
        count(ufp4_gated_act(at<uint16_t>(P), a, b, two, f, at<uint16_t>(P), b, 0, nullptr, nullptr, nullptr));
        count(ufp4_gated_act_backward(at<uint16_t>(P), b, at<uint8_t>(P), at<uint16_t>(P), 0, a, b, f, at<uint16_t>(P), two,
                                      nullptr, 0, nullptr));
      }
  require(ok > 100 && refused > 100 && g_moe_calls > 100, "coverage");
  printf("moe driver: %d accepted, %d refused, passed\n", ok, refused);
  return 0;
}
