// Attention over either paged cache, with a window and first tokens that stay
// visible: the plainest form.  A CTA has one query row (new token and query
// head); its warps take the visible keys in turn, each with a running maximum,
// sum and output, in fp32, which are joined at the end.
#include <cstdint>

#include "q4_cache4.cuh"

namespace q4 {
namespace {

constexpr int kWarps = 4;

// Element pairs lane, lane + 32, .. of a head's row of keys or values.
template <bool BF, bool FOUR, int N>
__device__ __forceinline__ void load_row(const AttnShape &s, const AttnCache &c, const Cache4 &c4, int64_t page, int head,
                                         int slot, bool value, float2 (&x)[N]) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(head) * s.page + slot;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int pair = lane + 32 * i;
        if constexpr (FOUR) {
            const uint8_t *r = c4.kv + page * c4.page_stride + row * record_bytes(s.d, c4.group_log2);
            const uint32_t w = reinterpret_cast<const uint32_t *>(r + (value ? s.d / 2 : 0))[pair / 4];
            const uint32_t p = reinterpret_cast<const uint32_t *>(r + s.d + (value ? 4 * s.d >> c4.group_log2 : 0))[2 * pair >> c4.group_log2];
            const uint4 v = values_of<BF>(w, both_low(p), both_high(p));
            const uint32_t all[4] = {v.x, v.y, v.z, v.w};
            x[i] = unpack2<BF>((pair & 3) == 0 ? all[0] : (pair & 3) == 1 ? all[1] : (pair & 3) == 2 ? all[2] : all[3]);
        } else {
            const uint16_t *r = (value ? c.v : c.k) + page * c.page_stride + row * s.d;
            x[i] = unpack2<BF>(reinterpret_cast<const uint32_t *>(r)[pair]);
        }
    }
}

template <bool BF, bool FOUR, int D>
__global__ void __launch_bounds__(32 * kWarps)
    attend_any_kernel(AttnShape s, AttnBatch b, AttnCache c, Cache4 c4, AttendCall a) {
    constexpr int N = D / 64;
    __shared__ float s_o[kWarps][D], s_m[kWarps], s_l[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x, hq = blockIdx.y, head = hq / s.group, pages = FOUR ? c4.pages : c.pages;
    int before = 0;
    for (int i = lane; i < b.batch; i += 32) before += b.cu_q[i + 1] <= t;
    const int req = __reduce_add_sync(0xffffffffu, before);
    if (t == 0 && hq == 0)
        for (int i = threadIdx.x; i < b.batch; i += 32 * kWarps)
            if (load_request(b, i, s.page_log2).bad) atomicOr(a.status, kAttnBadBatch);
    if (req >= b.batch || b.cu_q[req] > t) return;
    const Request r = load_request(b, req, s.page_log2);
    const int i = r.kv - r.ql + (t - r.q0);              // the token's index
    const int first = a.window > 0 ? max(0, i - a.window + 1) : 0, sinks = min(a.sinks, first);
    float2 q[N], o[N];
    const uint32_t *qs = reinterpret_cast<const uint32_t *>(a.q + static_cast<int64_t>(t) * a.q_stride + hq * D);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        q[e] = unpack2<BF>(qs[lane + 32 * e]);
        o[e] = make_float2(0.f, 0.f);
    }
    const float scale = a.scale * 1.4426950408889634f;
    float m = -INFINITY, l = 0.f;
    const int n = i < 0 ? 0 : sinks + i + 1 - first;
    for (int u = warp; u < n; u += kWarps) {
        const int j = u < sinks ? u : first + u - sinks;
        int page = b.table[req * b.table_stride + (j >> s.page_log2)];
        if (page < 0 || page >= pages) {
            if (lane == 0) atomicOr(a.status, kAttnBadPage);
            page = 0;
        }
        float2 x[N];
        load_row<BF, FOUR, N>(s, c, c4, page, head, j & (s.page - 1), false, x);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) dot += q[e].x * x[e].x + q[e].y * x[e].y;
#pragma unroll
        for (int d = 16; d; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
        dot *= scale;
        const float top = fmaxf(m, dot), ref = top == -INFINITY ? 0.f : top, keep = exp2f(m - ref), p = exp2f(dot - ref);
        m = top;
        l = l * keep + p;
        load_row<BF, FOUR, N>(s, c, c4, page, head, j & (s.page - 1), true, x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
            o[e].x = o[e].x * keep + p * x[e].x;
            o[e].y = o[e].y * keep + p * x[e].y;
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
        s_o[warp][2 * (lane + 32 * e)] = o[e].x;
        s_o[warp][2 * (lane + 32 * e) + 1] = o[e].y;
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
    __syncthreads();
    if (threadIdx.x >= D / 2) return;
    float top = -INFINITY, sum = 0.f, x = 0.f, y = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
    for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(s_m[w] - (top == -INFINITY ? 0.f : top));
        if (f == 0.f) continue;
        sum += s_l[w] * f;
        x += s_o[w][2 * threadIdx.x] * f;
        y += s_o[w][2 * threadIdx.x + 1] * f;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    reinterpret_cast<uint32_t *>(a.out + static_cast<int64_t>(t) * a.out_stride + hq * D)[threadIdx.x] = pack2<BF>(x * inv, y * inv);
}

}  // namespace

cudaError_t launch_attend_any(const AttnShape &s, const AttnBatch &b, const AttnCache *c, const Cache4 *c4,
                              const AttendCall &a, bool bf16, cudaStream_t st) {
    auto kernel = c4 ? (s.d == 64 ? (bf16 ? attend_any_kernel<true, true, 64> : attend_any_kernel<false, true, 64>)
                                  : (bf16 ? attend_any_kernel<true, true, 128> : attend_any_kernel<false, true, 128>))
                     : (s.d == 64 ? (bf16 ? attend_any_kernel<true, false, 64> : attend_any_kernel<false, false, 64>)
                                  : (bf16 ? attend_any_kernel<true, false, 128> : attend_any_kernel<false, false, 128>));
    kernel<<<dim3(b.tokens, s.hq), 32 * kWarps, 0, st>>>(s, b, c ? *c : AttnCache{}, c4 ? *c4 : Cache4{}, a);
    return cudaGetLastError();
}

}  // namespace q4
