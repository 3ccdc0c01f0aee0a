// Attention of chunks over the 4-bit cache, heads of 128: the warps that load and
// clean tiles of the 16-bit cache decode records into the same tiles.
#include "q4_attn_tc.cuh"

namespace q4 {

cudaError_t launch_attend_tc4_128(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                                 cudaStream_t st) {
    return c.group_log2 == 5 ? launch<Cfg<128, 5>, true, 5>(s, b, c, a, bf16, st) : launch<Cfg<128, 6>, true, 6>(s, b, c, a, bf16, st);
}

}  // namespace q4
