// serve_stubs.cpp -- stand-ins for the decoding operators' kernel launchers, linked
// instead of the device code into a sanitized host build of their C ABI.  Each
// checks the parameter block the ABI prepared and returns success.
#include <stdio.h>
#include <stdlib.h>

#include "../../fp4_quantization_amd/csrc/ufp4_serve.hpp"

namespace ufp4 {

int g_serve_calls = 0;

static void require(bool ok, const char* what) {
  if (!ok) {
    fprintf(stderr, "serve stub: %s\n", what);
    abort();
  }
}

bool matvec_in_lds(int64_t tokens, int64_t K, int parts) { return tokens <= 4 && K * tokens * parts <= 49152; }
hipError_t launch_matvec(const MatvecParams& p, hipStream_t) {
  ++g_serve_calls;
  require(p.tokens > 0 && p.N > 0 && p.y && p.ldy >= p.N && p.ldx >= p.K && p.K % 32 == 0, "matvec");
  require(p.K == 0 || (p.x && p.codes && p.scales && (p.mx || p.ts)), "matvec operands");
  require(p.K == 0 || matvec_in_lds(p.tokens, p.K, p.mx ? 3 : 2) || (p.xp && p.shift), "matvec workspace");
  return hipSuccess;
}
static void view(const CacheView& c) {
  require(c.heads >= 1 && c.dim % 32 == 0 && c.dim <= 256 && c.page_tokens % 32 == 0 && c.pages >= 0, "cache");
  require(c.pages == 0 || (c.kc && c.ks && c.vc && c.vs), "cache arrays");
  for (uint32_t n : {0u, 31u, 32u, 65536u, 0x3FFFFFFFu}) require(c.page.div(n) == n / (uint32_t)c.page_tokens, "page division");
}
hipError_t launch_cache_append(const CacheParams& p, hipStream_t) {
  ++g_serve_calls;
  view(p.c);
  require(p.tokens > 0 && p.k && p.v && p.slots, "append");
  return hipSuccess;
}
hipError_t launch_cache_read(const CacheParams& p, hipStream_t) {
  ++g_serve_calls;
  view(p.c);
  require(p.tokens > 0 && p.slots && (p.k_out || p.v_out), "read");
  return hipSuccess;
}
int attend_rows(int32_t, int32_t group, int32_t max_draft) { return (int64_t)group * max_draft > 16 ? 32 : 16; }
int32_t attend_runs(int32_t, int32_t) { return 768; }
hipError_t launch_attend(const AttendParams& p, hipStream_t) {
  ++g_serve_calls;
  view(p.c);
  require(p.q && p.out && p.q_offsets && p.lengths && (p.ld_pages == 0 || p.table), "attend");
  require(p.row_tiles >= 1 && p.group >= 1 && p.split && p.ml && p.o && (uintptr_t)p.o % 16 == 0, "attend workspace");
  require(p.ld_pages * p.c.page_tokens <= (1 << 30) && p.sequences >= 1 && p.sequences <= 65535, "attend limits");
  return hipSuccess;
}

}  // namespace ufp4
