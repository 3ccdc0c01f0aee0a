// Attention of few new tokens over the 16-bit cache, through a window with
// first tokens that stay visible: key tiles between the two are left out of
// the items, so such a call costs what its visible tokens do.
#include "q4_attn_stream.cuh"

namespace q4 {

cudaError_t launch_attend_stream_sinks(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a,
                                       bool bf16, cudaStream_t st) {
    return s.d == 64 ? launch<Cfg<64>, true>(s, b, c, a, bf16, st) : launch<Cfg<128>, true>(s, b, c, a, bf16, st);
}

}  // namespace q4
