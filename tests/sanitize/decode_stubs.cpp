// Stand-ins for the launchers of the single-token kernels, for a host-only build of their ABI layer
// (qv_decode_abi.cpp) under AddressSanitizer and UndefinedBehaviorSanitizer.  Each stub counts its calls
// and reports a launch failure, so a test can tell whether a call got past the argument checks.
#include "qv_decode_internal.h"

static int g_launches = 0;

extern "C" int qv_stub_launches(void) { return g_launches; }
extern "C" void qv_stub_reset(void) { g_launches = 0; }

namespace qv {

static hipError_t stub() {
  ++g_launches;
  return hipErrorInvalidValue;
}

hipError_t launch_w4a16(const void*, bool, int64_t, int64_t, int64_t, bool, const float*, const uint8_t*, const float*,
                        int64_t, const float*, int64_t, bool, void*, bool, int64_t, float*, hipStream_t) {
  return stub();
}
hipError_t launch_kv_append(const AppendArgs&, hipStream_t) { return stub(); }
hipError_t launch_paged_attention(const AttentionArgs&, hipStream_t) { return stub(); }

}  // namespace qv
