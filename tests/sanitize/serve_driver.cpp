// serve_driver.cpp -- drives the decoding operators' C ABI (host side) through
// valid and refused calls over many sizes, in a sanitized build.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../fp4_quantization_amd/csrc/ufp4_serve.hpp"
#include "../../include/ufp4.h"

namespace ufp4 {
extern int g_serve_calls;
}

template <typename T>
static T* at(uintptr_t a) {
  return reinterpret_cast<T*>(a);
}

int main() {
  using namespace ufp4;
  const uintptr_t P = (uintptr_t)1 << 40;
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 2, 31, 32, 64, 1000, 4096, (1 << 21) - 1, (1 << 25) - 32, 1 << 25, (int64_t)1 << 28,
                           (int64_t)1 << 30, (int64_t)1 << 40, INT64_MAX};
  const int32_t small[] = {INT32_MIN, -1, 0, 1, 2, 32, 64, 256, 1024, 8192, 65535, 65536, 1 << 28, INT32_MAX};
  ufp4_config cfg{};
  ufp4_qtensor q{at<uint8_t>(P), at<uint8_t>(P), at<float>(P)};
  int ok = 0, refused = 0;
  auto count = [&](int rc) {
    if (rc < 0 || rc > 4) {
      fprintf(stderr, "serve driver: status %d\n", rc);
      abort();
    }
    (rc == 0 ? ok : refused)++;
  };
  for (int64_t a : sizes)
    for (int64_t b : sizes)
      for (int64_t c : sizes)
        for (int32_t mx : {0, 1}) {
          cfg.scaling = mx;
          const size_t n = ufp4_matvec_workspace(&cfg, a, b, c);
          count(ufp4_matvec(&cfg, at<void>(P), mx, a, c, c, q, b, at<void>(P), 1, b, at<void>(P), n, nullptr));
          if (n) count(ufp4_matvec(&cfg, at<void>(P), 0, a, c, c, q, b, at<void>(P), 0, b, at<void>(P), n - 1, nullptr));
        }
  cfg.scaling = 0;
  for (int64_t pages : sizes)
    for (int32_t page : small)
      for (int32_t heads : small)
        for (int32_t dim : {-32, 0, 32, 48, 96, 256, 288, INT32_MAX}) {
          const ufp4_cache c{at<uint8_t>(P), at<uint8_t>(P), at<uint8_t>(P), at<uint8_t>(P), nullptr, at<float>(P), pages, page, heads, dim};
          for (int64_t t : {(int64_t)0, (int64_t)5, (int64_t)1 << 28}) {
            const int64_t w = (int64_t)heads * dim;
            count(ufp4_cache_append(&cfg, &c, at<uint16_t>(P), w, at<uint16_t>(P), w, t, at<int64_t>(P), nullptr));
            count(ufp4_cache_read(&cfg, &c, at<int64_t>(P), t, 1, at<void>(P), w, nullptr, 0, 1, nullptr));
          }
        }
  const ufp4_cache c{at<uint8_t>(P), at<uint8_t>(P), at<uint8_t>(P), at<uint8_t>(P), nullptr, nullptr, 100, 64, 4, 96};
  for (int32_t heads : small)
    for (int32_t n : small)
      for (int32_t most : small)
        for (int64_t ld : sizes)
          for (int64_t rows : {(int64_t)-1, (int64_t)0, (int64_t)77, INT64_MAX}) {
            const size_t ws = ufp4_tree_attention_workspace(&c, heads, n, most);
            const int64_t w = (int64_t)heads * 96;
            count(ufp4_tree_attention(&cfg, &c, at<uint16_t>(P), w, heads, at<int64_t>(P), n, rows, most, at<int32_t>(P), at<int32_t>(P), ld,
                                      rows == 77 ? at<uint64_t>(P) : nullptr, 0.1f, at<uint16_t>(P), w, at<float>(P), at<void>(P), ws, nullptr));
          }
  if (ok < 100 || refused < 100 || g_serve_calls < 100) abort();
  printf("serve driver: %d accepted, %d refused, passed\n", ok, refused);
  return 0;
}
