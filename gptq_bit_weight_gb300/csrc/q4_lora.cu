// Low-rank adapters of many requests beside a shared projection:
//     out[m] = y[m] + scale_a (x[m] . A_a^T) . B_a^T,   a = row_slot[m].
// Two launches: the sums t[m][r] = scale_a x[m] . A_a[r] in fp32, then the
// product with B and the sum with y, rounded once.
#include <cstdint>

#include "q4_serve.h"

namespace q4 {
namespace {

// Copies one adapter into its slot: A rows padded with zero rows to a rank
// that is a multiple of 16, B rows padded with zeros the same way.
__global__ void lora_set_kernel(uint16_t *a, uint16_t *b, LoraSlot *slot, const uint16_t *src_a,
                                const uint16_t *src_b, int K, int N, int rank, int r16, float scale) {
    const size_t na = static_cast<size_t>(r16) * K, nb = static_cast<size_t>(r16) * N;
    const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x;
    const size_t i0 = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    for (size_t i = i0; i < na; i += step) a[i] = i / K < static_cast<size_t>(rank) ? src_a[i] : 0;
    for (size_t i = i0; i < nb; i += step) {
        const size_t n = i / r16;
        const int r = static_cast<int>(i - n * r16);
        b[i] = r < rank ? src_b[n * rank + r] : 0;
    }
    if (i0 == 0) *slot = LoraSlot{rank, scale};
}

__device__ __forceinline__ int row_adapter(const LoraView &v, const LoraCall &c, int m, LoraSlot *s) {
    const int slot = c.row_slot[m];
    if (slot >= v.slots) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(v.status, kLoraBadSlot);
        return -1;
    }
    if (slot < 0) return -1;
    *s = v.slot[slot];
    return s->rank > 0 ? slot : -1;
}

// One warp for each (row, rank): a dot product over K.
template <bool BF>
__global__ void __launch_bounds__(256) lora_shrink_kernel(LoraView v, LoraCall c) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = blockIdx.y, r = blockIdx.x * 8 + warp;
    LoraSlot s;
    const int slot = row_adapter(v, c, m, &s);
    if (slot < 0 || r >= ceil16(s.rank)) return;
    const uint4 *x = reinterpret_cast<const uint4 *>(c.x + m * c.xs);
    const uint4 *a = reinterpret_cast<const uint4 *>(v.a + (static_cast<size_t>(slot) * v.rpad + r) * v.K);
    float acc = 0.f;
    for (int k = lane; k < v.K / 8; k += 32) {
        const uint4 p = x[k], q = a[k];
        const uint32_t pw[4] = {p.x, p.y, p.z, p.w}, qw[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 u = unpack2<BF>(pw[e]), w = unpack2<BF>(qw[e]);
            acc = fmaf(u.x, w.x, fmaf(u.y, w.y, acc));
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    if (lane == 0) v.t[static_cast<size_t>(m) * v.rpad + r] = acc * s.scale;
}

// One thread for each output column of a row.
template <bool BF>
__global__ void __launch_bounds__(256) lora_expand_kernel(LoraView v, LoraCall c) {
    const int m = blockIdx.y, n = 2 * (blockIdx.x * blockDim.x + threadIdx.x);
    LoraSlot s{0, 0.f};
    const int slot = row_adapter(v, c, m, &s);
    if (n >= v.N) return;
    const uint32_t y = *reinterpret_cast<const uint32_t *>(c.y + m * c.ys + n);
    float2 acc = make_float2(0.f, 0.f);
    if (slot >= 0) {
        const int r16 = ceil16(s.rank);
        const uint16_t *b = v.b + static_cast<size_t>(slot) * v.N * v.rpad + static_cast<size_t>(n) * r16;
        const float *t = v.t + static_cast<size_t>(m) * v.rpad;
        for (int r = 0; r < r16; r += 2) {
            const float2 p = unpack2<BF>(*reinterpret_cast<const uint32_t *>(b + r));
            const float2 q = unpack2<BF>(*reinterpret_cast<const uint32_t *>(b + r16 + r));
            acc.x = fmaf(t[r], p.x, fmaf(t[r + 1], p.y, acc.x));
            acc.y = fmaf(t[r], q.x, fmaf(t[r + 1], q.y, acc.y));
        }
    }
    const float2 yy = unpack2<BF>(y);
    *reinterpret_cast<uint32_t *>(c.out + m * c.os + n) = pack2<BF>(yy.x + acc.x, yy.y + acc.y);
}

}  // namespace

cudaError_t launch_lora_set(const LoraView &v, uint16_t *a, uint16_t *b, LoraSlot *slot, int s, const uint16_t *src_a,
                            const uint16_t *src_b, int rank, float scale, cudaStream_t st) {
    const int r16 = ceil16(rank);
    const size_t n = static_cast<size_t>(r16) * (v.K > v.N ? v.K : v.N);
    const int grid = static_cast<int>(n / 256 + 1 < 1216 ? n / 256 + 1 : 1216);
    lora_set_kernel<<<grid, 256, 0, st>>>(a + static_cast<size_t>(s) * v.rpad * v.K,
                                          b + static_cast<size_t>(s) * v.rpad * v.N, slot + s, src_a, src_b, v.K, v.N,
                                          rank, r16, scale);
    return cudaGetLastError();
}

cudaError_t launch_lora_add(const LoraView &v, const LoraCall &c, bool bf16, cudaStream_t st, int *launches) {
    for (int m0 = 0; m0 < c.M; m0 += 65535) {          // rows are the grid's y dimension
        LoraCall d = c;
        LoraView w = v;
        d.M = c.M - m0 < 65535 ? c.M - m0 : 65535;
        d.x += m0 * c.xs;
        d.y += m0 * c.ys;
        d.out += m0 * c.os;
        d.row_slot += m0;
        w.t += static_cast<size_t>(m0) * v.rpad;
        const dim3 gs(v.rpad / 8, d.M), ge((v.N + 511) / 512, d.M);
        if (bf16) {
            lora_shrink_kernel<true><<<gs, 256, 0, st>>>(w, d);
            lora_expand_kernel<true><<<ge, 256, 0, st>>>(w, d);
        } else {
            lora_shrink_kernel<false><<<gs, 256, 0, st>>>(w, d);
            lora_expand_kernel<false><<<ge, 256, 0, st>>>(w, d);
        }
        *launches += 2;
    }
    return cudaGetLastError();
}

}  // namespace q4
