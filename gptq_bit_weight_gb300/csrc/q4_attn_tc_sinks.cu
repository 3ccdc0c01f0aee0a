// Attention of chunks over the 16-bit cache, through a window with first tokens
// that stay visible: key tiles that no row of an item sees are left out of it.
// Two chunks of up to 1500 tokens at a window of 2048 and 100 first ones, 32 heads
// over 8 of 64: 67 us, bound as such chunks are without first tokens.
#include "q4_attn_tc.cuh"

namespace q4 {

cudaError_t launch_attend_tc_sinks(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a,
                                   bool bf16, cudaStream_t st) {
    return s.d == 64 ? launch<Cfg<64>, true, 0>(s, b, c, a, bf16, st) : launch<Cfg<128>, true, 0>(s, b, c, a, bf16, st);
}

}  // namespace q4
