// Attention of few new tokens over the 4-bit cache: row tiles of 8 rows.
#include "q4_attn_stream4.cuh"

namespace q4 {
cudaError_t launch_attend_stream4_8(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a,
                                    bool bf16, cudaStream_t st) {
    return launch_rows<1, 3>(s, b, c, a, bf16, st);
}
}  // namespace q4
