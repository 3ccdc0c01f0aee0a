// Rotary positions and the append to the paged cache, in one pass over the
// fused projection's output: each (query or key) pair (a, b) becomes
// (a cos - b sin, b cos + a sin) in fp32, rounded once; values are copied.
// Bound by memory: every element is read once and written once.  Three prompts
// of 10423 tokens in all, 96 heads of 128: 85 us, 6.1 TB/s, 0.89 of the
// copy rate; 64 single tokens 4.2 us, a launch.  A work item has two 16-byte
// vectors, both halves of eight pairs, so that a pair never crosses threads;
// the cosines and sines come from a table (L2: all heads of a token share
// them), which is cheaper than their computation to the last bit.
#include <algorithm>
#include <cstdint>

#include "q4_serve.h"

namespace q4 {
namespace {

struct Freqs {
    double f[64];
};

// cos and sin of pos * f_i, the angle in fp64: at position 10^6 an fp32
// product would be off by 0.06 rad.
__global__ void rope_table_kernel(float2 *table, Freqs f, double scale, int half, int max_pos) {
    const size_t n = static_cast<size_t>(max_pos) * half, step = static_cast<size_t>(gridDim.x) * blockDim.x;
    for (size_t i = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
        const int pos = static_cast<int>(i / half), p = static_cast<int>(i - static_cast<size_t>(pos) * half);
        double s, c;
        sincos(pos * f.f[p], &s, &c);
        table[i] = make_float2(static_cast<float>(c * scale), static_cast<float>(s * scale));
    }
}

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;        // of one CTA: one warp looks each of them up

struct Token {
    int64_t dst;      // element offset of (page, head 0, token) in the cache; -1: no request or out of range
    int pos;          // rotary position
};

// Work item: 16 elements of one head of one token, as two 16-byte vectors:
// both halves of eight pairs (i, i + rot / 2), or eight interleaved pairs, or
// 16 elements past the rotated part.
template <bool BF>
__global__ void __launch_bounds__(kThreads)
    append_kernel(AttnShape s, AttnBatch b, AttnCache c, AppendCall a, int tokens_per_cta) {
    __shared__ Token tok[kMaxTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * tokens_per_cta, nt = min(tokens_per_cta, b.tokens - t0);
    if (warp < nt) {
        const int t = t0 + warp;
        int before = 0;                                  // requests that end at or before t
        for (int i = lane; i < b.batch; i += 32) before += b.cu_q[i + 1] <= t;
        const int req = __reduce_add_sync(0xffffffffu, before);
        if (lane == 0) {
            Token k{-1, 0};
            if (req < b.batch && b.cu_q[req] <= t) {
                const Request r = load_request(b, req, s.page_log2);
                const int idx = r.kv - r.ql + (t - r.q0);
                int bad = 0;
                // A length that had to be cut says nothing of where the token belongs: its index in the cut context
                // is another token's, and a table's padding may be another request's page.
                if (r.bad || idx < 0 || idx >= r.kv) {
                    bad = kAttnBadBatch;
                } else {
                    const int page = b.table[req * b.table_stride + (idx >> s.page_log2)];
                    k.pos = a.positions ? a.positions[t] : idx;
                    if (page < 0 || page >= c.pages) bad |= kAttnBadPage;
                    else if (a.rope && (k.pos < 0 || k.pos >= a.max_pos)) bad |= kAttnBadPosition;
                    else k.dst = page * c.page_stride + static_cast<int64_t>(idx & (s.page - 1)) * s.d;
                }
                if (bad) atomicOr(a.status, bad);
            }
            tok[warp] = k;
        }
    }
    __syncthreads();
    const int per_head = s.d / 16, heads = s.hq + 2 * s.hkv, per_token = heads * per_head;
    const int half = a.rot / 2, turned = a.rope ? a.rot / 16 : 0;
    for (int w = threadIdx.x; w < nt * per_token; w += kThreads) {
        const int ti = w / per_token, u = w - ti * per_token, head = u / per_head, item = u - head * per_head;
        const Token k = tok[ti];
        if (k.dst < 0) continue;
        const int64_t t = t0 + ti;
        const bool turn = item < turned && head < s.hq + s.hkv;
        int e0 = 16 * item, e1 = e0 + 8;                 // first elements of the two vectors
        if (turn && !a.interleaved) {
            e0 = 8 * item;
            e1 = e0 + half;
        }
        const uint16_t *src = a.qkv + t * a.qkv_stride + head * s.d;
        uint4 v0 = *reinterpret_cast<const uint4 *>(src + e0), v1 = *reinterpret_cast<const uint4 *>(src + e1);
        if (turn) {
            const float4 *cs = reinterpret_cast<const float4 *>(a.rope + static_cast<int64_t>(k.pos) * half + 8 * item);
            uint32_t *p = reinterpret_cast<uint32_t *>(&v0), *q = reinterpret_cast<uint32_t *>(&v1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {                // pairs 2e and 2e + 1 of the item's eight
                const float4 r = cs[e];                  // cos, sin, cos, sin
                if (a.interleaved) {
                    uint32_t *x = e < 2 ? p + 2 * e : q + 2 * (e - 2);
                    const float2 m = unpack2<BF>(x[0]), n = unpack2<BF>(x[1]);
                    x[0] = pack2<BF>(m.x * r.x - m.y * r.y, m.y * r.x + m.x * r.y);
                    x[1] = pack2<BF>(n.x * r.z - n.y * r.w, n.y * r.z + n.x * r.w);
                } else {
                    const float2 m = unpack2<BF>(p[e]), n = unpack2<BF>(q[e]);
                    p[e] = pack2<BF>(m.x * r.x - n.x * r.y, m.y * r.z - n.y * r.w);
                    q[e] = pack2<BF>(n.x * r.x + m.x * r.y, n.y * r.z + m.y * r.w);
                }
            }
        }
        uint16_t *dst;
        if (head < s.hq) {
            dst = a.q_out + t * a.q_stride + head * s.d;
        } else {
            const bool key = head < s.hq + s.hkv;
            const int h = head - s.hq - (key ? 0 : s.hkv);
            dst = (key ? c.k : c.v) + k.dst + static_cast<int64_t>(h) * s.page * s.d;
        }
        *reinterpret_cast<uint4 *>(dst + e0) = v0;
        *reinterpret_cast<uint4 *>(dst + e1) = v1;
    }
}

}  // namespace

cudaError_t launch_rope_table(float2 *table, const double *inv_freq, double length_scale, int half, int max_pos,
                              cudaStream_t st) {
    Freqs f{};
    for (int i = 0; i < half; ++i) f.f[i] = inv_freq[i];
    rope_table_kernel<<<608, 256, 0, st>>>(table, f, length_scale, half, max_pos);
    return cudaGetLastError();
}

cudaError_t launch_attn_append(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AppendCall &a,
                               bool bf16, cudaStream_t st) {
    // one token for each CTA until the GPU is full, then up to eight
    const int per = std::max(1, std::min(kMaxTokens, b.tokens / 1216));
    const int grid = (b.tokens + per - 1) / per;
    if (bf16) append_kernel<true><<<grid, kThreads, 0, st>>>(s, b, c, a, per);
    else append_kernel<false><<<grid, kThreads, 0, st>>>(s, b, c, a, per);
    return cudaGetLastError();
}

}  // namespace q4
