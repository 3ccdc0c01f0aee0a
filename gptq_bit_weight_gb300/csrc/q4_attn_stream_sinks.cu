// Attention of few new tokens over the 16-bit cache, through a window with
// first tokens that stay visible: key tiles between the two are left out of
// the items, so such a call costs what its visible tokens do: 32 requests of up
// to 65536 tokens at a window of 4096 and 4 first ones, 64 heads over 8 of 128: 93
// us, 5.8 TB/s of what is seen.
#include "q4_attn_stream.cuh"

namespace q4 {

cudaError_t launch_attend_stream_sinks(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a,
                                       bool bf16, cudaStream_t st) {
    return s.d == 64 ? launch<Cfg<64>, true>(s, b, c, a, bf16, st) : launch<Cfg<128>, true>(s, b, c, a, bf16, st);
}

}  // namespace q4
