// Stand-ins for the launchers of the kernels for runs of tokens, for a host-only build of their ABI layer (qv_runs_abi.cpp)
// under AddressSanitizer and UndefinedBehaviorSanitizer.  Each stub counts its calls and reports a launch failure.
#include "qv_runs_internal.h"

static int g_launches = 0;

extern "C" int qv_stub_launches(void) { return g_launches; }
extern "C" void qv_stub_reset(void) { g_launches = 0; }

// Parts and workspace of a call, for checks of one against the other.
extern "C" int64_t qv_stub_parts(int64_t T, int64_t B, int64_t q_heads, int64_t heads, int64_t seen, int64_t room) {
  return qv::run_tiles(T, B, q_heads, heads, seen, room).parts;
}
extern "C" int64_t qv_stub_items(int64_t T, int64_t B, int64_t q_heads, int64_t heads) {
  return qv::run_tiles(T, B, q_heads, heads, 0).items;
}

namespace qv {

static hipError_t stub() {
  ++g_launches;
  return hipErrorInvalidValue;
}

hipError_t launch_page_tables(const TablesArgs&, hipStream_t) { return stub(); }
hipError_t launch_run_attention(const RunArgs&, hipStream_t) { return stub(); }

}  // namespace qv
