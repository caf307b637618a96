// matvec_plan_driver.cpp -- walks the choice of a product's launch over tokens, N, K
// and parts, and checks what each kernel takes for granted.
#include <stdio.h>

#include <initializer_list>

#include "../../fp4_quantization_amd/csrc/ufp4_matvec_plan.hpp"

using namespace ufp4;

static int failed = 0;
static void require(bool ok, const char* what, int64_t T, int64_t N, int64_t K, int parts) {
  if (ok) return;
  if (++failed <= 20)
    fprintf(stderr, "%s: T %lld, N %lld, K %lld, %d parts\n", what, (long long)T, (long long)N, (long long)K, parts);
}

int main() {
  const int64_t Ts[] = {1, 2, 4, 5, 7, 16, 17, 20, 32, 33, 37, 48, 49, 64, 65, 130, 1000, 70000, (1 << 21) - 1};
  const int64_t Ns[] = {1, 15, 16, 17, 130, 1365, 2048, 4096, 4097, 14336, 16384, 65536, (1 << 25) - 1};
  const int64_t Ks[] = {0, 32, 96, 128, 512, 544, 2080, 4096, 4128, 8192, 16384, 65536, (1 << 25) - 32};
  bool seen[3][5] = {};
  for (int64_t T : Ts)
    for (int64_t N : Ns)
      for (int64_t K : Ks)
        for (int parts : {1, 2, 3}) {
          const MatvecPlan m = matvec_plan(T, N, K, parts);
          const int64_t chunks = (K + kMvChunk - 1) / kMvChunk, t16 = (T + 15) / 16;
          auto ok = [&](bool c, const char* what) { require(c, what, T, N, K, parts); };
          seen[m.x][m.nt] = true;
          ok(m.nt == 1 || m.nt == 2 || m.nt == 4, "tiles of tokens");
          ok(m.log_kw >= 0 && m.log_kw <= 3, "waves of a tile");
          ok(m.gx >= 1 && m.gx <= 512 && m.gy >= 1 && m.gy <= 65535, "grid");
          if (m.x == kXLds) {
            ok(T <= kLdsTokens && m.nt == 1 && m.gy == 1, "LDS: tokens");
            ok(chunks * kMvChunk * T * parts * 2 <= (int64_t)kLdsX, "LDS: bytes");
            continue;
          }
          // a call without values of K has no workspace: nothing may be read from it
          // but piece by piece of the chunks that there are
          ok(m.gy * m.nt >= t16, "all tokens");
          if (m.x == kXRegisters) {
            ok(chunks > 0, "registers: no chunk to read");
            ok(m.nt == 1 && parts == 1 && chunks <= (kSegment << m.log_kw), "registers: one segment");
          }
        }
  if (!seen[kXLds][1] || !seen[kXRegisters][1] || !seen[kXMemory][1] || !seen[kXMemory][2] || !seen[kXMemory][4]) {
    fprintf(stderr, "not every kernel was chosen\n");
    ++failed;
  }
  if (failed) return 1;
  printf("matvec plan driver: passed\n");
  return 0;
}
