// Device helpers shared by the adapter kernels.
#pragma once
#include "q4_serve.h"

namespace q4 {

template <bool BF>
__device__ __forceinline__ uint16_t to16(float x) {
    if constexpr (BF) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
    else return __half_as_ushort(__float2half_rn(x));
}
template <bool BF>
__device__ __forceinline__ float from16(uint16_t x) {
    if constexpr (BF) return __bfloat162float(__ushort_as_bfloat16(x));
    else return __half2float(__ushort_as_half(x));
}

// t goes into the second product as two 16-bit parts, hi = round(t) and
// lo = round(t - hi): together t to 2^-16 (bf16) or 2^-22 (fp16) of itself.
// fp16 has no range to spare: a row is scaled by a power of two that brings
// its largest value to [2^13, 2^14), which `split_scale` undoes at the end.
// NaN and infinity stay what they are.
__device__ __forceinline__ float split_scale_of(float top) {
    // exponent of top + 1 - 14, kept where both the scale and its inverse are normal
    const int e = static_cast<int>(__float_as_uint(top) >> 23 & 0xff) - 127 - 13;
    return __uint_as_float(static_cast<uint32_t>(min(max(e, -100), 100) + 127) << 23);
}
// The second part; none beside a first part that is infinite or NaN.
template <bool BF>
__device__ __forceinline__ uint16_t split_low(float x, uint16_t hi) {
    const float d = x - from16<BF>(hi);
    return isfinite(d) ? to16<BF>(d) : 0;
}

}  // namespace q4
