// Attention of a step's new tokens over the paged cache, with the running
// maximum m and sum l of the softmax: for each key j,
//     m' = max(m, s_j),  l = l 2^(m - m') + 2^(s_j - m'),  o = o 2^(m - m') + 2^(s_j - m') v_j,
// s_j = scale log2(e) q . k_j, and o / l at the end.
// One warp for each (token, query head).
#include <cstdint>

#include "q4_serve.h"

namespace q4 {
namespace {

template <bool BF, int D>
__global__ void __launch_bounds__(256) attend_kernel(AttnShape s, AttnBatch b, AttnCache c, AttendCall a) {
    constexpr int E = D / 64;                      // element pairs of a lane
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int t = static_cast<int>(w / s.hq), head = static_cast<int>(w % s.hq);
    if (t >= b.tokens) return;
    int before = 0;
    for (int i = lane; i < b.batch; i += 32) before += b.cu_q[i + 1] <= t;
    const int req = __reduce_add_sync(0xffffffffu, before);
    if (req >= b.batch || b.cu_q[req] > t) return;
    const Request r = load_request(b, req, s.page_log2);
    const int idx = r.kv - r.ql + (t - r.q0);
    int bad = r.bad ? kAttnBadBatch : 0;
    const float scale = a.scale * 1.4426950408889634f;
    const int64_t row = t * a.q_stride + head * D + 2 * lane;
    float2 q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = unpack2<BF>(*reinterpret_cast<const uint32_t *>(a.q + row + 64 * e));
        o[e] = make_float2(0.f, 0.f);
    }
    float m = -INFINITY, l = 0.f;
    const int j0 = a.window > 0 ? max(0, idx - a.window + 1) : 0;
    int64_t base = 0;
    for (int j = j0; j <= min(idx, r.kv - 1); ++j) {
        if (j == j0 || (j & (s.page - 1)) == 0) {
            int page = b.table[req * b.table_stride + (j >> s.page_log2)];
            if (page < 0 || page >= c.pages) {
                bad |= kAttnBadPage;
                page = 0;
            }
            base = page * c.page_stride + static_cast<int64_t>(head / s.group) * s.page * D + 2 * lane;
        }
        const int64_t at = base + static_cast<int64_t>(j & (s.page - 1)) * D;
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 k = unpack2<BF>(*reinterpret_cast<const uint32_t *>(c.k + at + 64 * e));
            dot = fmaf(q[e].x, k.x, fmaf(q[e].y, k.y, dot));
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
        dot *= scale;
        const float top = fmaxf(m, dot);
        const float keep = exp2f(m - (top == -INFINITY ? 0.f : top)), p = exp2f(dot - (top == -INFINITY ? 0.f : top));
        m = top;
        l = l * keep + p;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const float2 v = unpack2<BF>(*reinterpret_cast<const uint32_t *>(c.v + at + 64 * e));
            o[e].x = o[e].x * keep + p * v.x;
            o[e].y = o[e].y * keep + p * v.y;
        }
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    uint16_t *dst = a.out + t * a.out_stride + head * D + 2 * lane;
#pragma unroll
    for (int e = 0; e < E; ++e) *reinterpret_cast<uint32_t *>(dst + 64 * e) = pack2<BF>(o[e].x * inv, o[e].y * inv);
    if (bad && lane == 0) atomicOr(a.status, bad);
}

}  // namespace

cudaError_t launch_attend(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a, bool bf16,
                          cudaStream_t st) {
    const int64_t warps = static_cast<int64_t>(b.tokens) * s.hq;
    const unsigned grid = static_cast<unsigned>((warps + 7) / 8);
    auto go = [&](auto bf, auto d) { attend_kernel<decltype(bf)::value, decltype(d)::value><<<grid, 256, 0, st>>>(s, b, c, a); };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (s.d == 64) bf16 ? go(std::true_type{}, D64{}) : go(std::false_type{}, D64{});
    else bf16 ? go(std::true_type{}, D128{}) : go(std::false_type{}, D128{});
    return cudaGetLastError();
}

}  // namespace q4
