// Attention of few new tokens over the 16-bit cache.
#include "q4_attn_stream.cuh"

namespace q4 {

size_t attend_stream_ws_bytes(int ctas) { return static_cast<size_t>(2) * ctas * Cfg<128>::kPiece * sizeof(float); }

cudaError_t launch_attend_stream(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a,
                                 bool bf16, cudaStream_t st) {
    return s.d == 64 ? launch<Cfg<64>, false>(s, b, c, a, bf16, st) : launch<Cfg<128>, false>(s, b, c, a, bf16, st);
}

}  // namespace q4
