// Attention of chunks over the 16-bit cache.
#include "q4_attn_tc.cuh"

namespace q4 {

size_t attend_tc_ws_bytes(int ctas) { return static_cast<size_t>(2) * ctas * Cfg<128>::kPiece * sizeof(float); }

cudaError_t launch_attend_tc(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a, bool bf16,
                             cudaStream_t st) {
    return s.d == 64 ? launch<Cfg<64>, false, 0>(s, b, c, a, bf16, st) : launch<Cfg<128>, false, 0>(s, b, c, a, bf16, st);
}

}  // namespace q4
