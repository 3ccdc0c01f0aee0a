// Rotary positions and the append to a paged cache held in 4 bits, and reading
// tokens back out of either cache as 16-bit values.
//
// Appending is one pass over the fused projection's output, as for the 16-bit
// cache (q4_attn_append.cu): queries are rotated and written; keys are rotated
// and rounded to 16 bits, then keys and values are quantised by groups of 32 or
// 64 elements: m = least, s = (greatest - m) / 15 rounded to 16 bits, c = round
// to even of (x - m) / s.
//   A code changes where (x - m) / s passes a half, so what goes in has to be the
//   same number wherever it is computed: the rotation carries the errors of its
//   two products and of their sum (Dekker's and Knuth's, by fma and two-sum), so
//   that its fp32 result is the exact one rounded once; the quotient is corrected
//   by its remainder, one exact fma (Markstein's); and a difference that fp32
//   cannot hold keeps its error.
//   That error says something only where the rounded difference is a half step
//   h s exactly: h s has at most 16 bits, so rounding to fp32 keeps the order of
//   x - m and h s otherwise.  fp32 loses bits of x - m if one of the two is below
//   2^-13 of the difference (2^-16 in bf16).  A tiny m is seen at once; where x
//   is tiny and x - m a half step, -m / s is within 2^-13 of a half.  Groups of
//   either sort go through code that compares with the error, and so does the
//   span's, which decides where a fifteenth of the rounded span is exact (prompts
//   84 -> 87 us).
// A work item has 16 elements of a head.  A key's pairs (i, i + rot / 2) come from
// two places, so the rotated elements go through shared memory, after which an
// item holds 16 neighbours and a group is 2 or 4 lanes.
// Three prompts of 9912 tokens, 96 heads of 128: 87 us, 4.4 TB/s, issue slots 58%
// busy, bound by the latency of a token's loads and what follows them (a code at a
// time, with its border looked at, 137); 64 single tokens of 80 heads 8 us with the
// launch.  Reading the prompts' tokens back: 37 us, 5.4 TB/s.
#include <algorithm>
#include <cstdint>

#include "q4_attn_rows.cuh"
#include "q4_cache4.cuh"

namespace q4 {
namespace {

constexpr int kThreads = 256;

// x y - u v, rounded once: the products' errors and the sum's are added back.
__device__ __forceinline__ float cross(float x, float y, float u, float v) {
    const float p = __fmul_rn(x, y), q = __fmul_rn(u, v);
    const float ep = __fmaf_rn(x, y, -p), eq = __fmaf_rn(u, v, -q);
    const float s = __fsub_rn(p, q), b = __fsub_rn(s, p);
    const float es = __fsub_rn(__fsub_rn(p, __fsub_rn(s, b)), __fadd_rn(q, b));
    const float r = __fadd_rn(s, __fadd_rn(es, __fsub_rn(ep, eq)));
    return fabsf(s) < INFINITY ? r : s;                  // of infinities there are no errors
}

template <bool BF>
__device__ __forceinline__ uint32_t min_2(uint32_t a, uint32_t b) {          // NaN if either is
    uint32_t d;
    if constexpr (BF) asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Two fp32 lanes in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// What the rounded difference d of x and y lacks, exactly (two-sum).
__device__ __forceinline__ float lost(float x, float y, float d) {
    const float b = __fsub_rn(d, x);
    return __fsub_rn(__fsub_rn(x, __fsub_rn(d, b)), __fadd_rn(y, b));
}
// x / 15, rounded once, for x >= 1e-30: the product with the rounded reciprocal, corrected by its remainder.
__device__ __forceinline__ float fifteenth(float x) {
    const float r = 1.f / 15.f, q = __fmul_rn(x, r);
    return __fmaf_rn(__fmaf_rn(-q, 15.f, x), r, q);
}

// Codes of sixteen 16-bit values, and s and m, of a group from lo to hi, whatever the differences lack in fp32.  Not
// inlined: few groups come here.
template <bool BF>
__device__ __noinline__ uint3 quantise_exactly(uint4 v0, uint4 v1, float lo, float hi) {
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    const float span = __fsub_rn(hi, lo), rest = lost(hi, lo, span);
    const bool small = span < 1e-30f;
    float part = small ? __fdiv_rn(span, 15.f) : fifteenth(span);
    // A fifteenth without remainder ends in three zeros or more, so one unit up or down passes no border of the type and
    // leaves one that it stands on, to the side of what the span lacks.
    if (rest != 0.f && __fmaf_rn(-part, 15.f, span) == 0.f) part = __int_as_float(__float_as_int(part) + (rest > 0.f ? 1 : -1));
    const uint32_t sm = pack2<BF>(part, lo);
    const float up = small ? 0x1p64f : 1.f, s = unpack2<BF>(sm).x * up, inv = s > 0.f ? __fdividef(1.f, s) : 0.f;  // in range
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const float2 f = unpack2<BF>(w[e >> 1]);
        const float x = e & 1 ? f.y : f.x, d0 = __fsub_rn(x, lo), d = d0 * up, k = fminf(floorf(d * inv), 15.f);
        const float past = __fmaf_rn(-(k + 0.5f), s, d) + lost(x, lo, d0) * up;     // of the half after k
        const int n = static_cast<int>(k);
        const int code = s > 0.f ? min(n + (past > 0.f || (past == 0.f && (n & 1))), 15) : 0;
        c[e >> 3] |= static_cast<uint32_t>(code) << (4 * ((e & 7) >> 1) + 16 * (e & 1));
    }
    return make_uint3(c[0], c[1], sm);
}

// Sixteen 16-bit values in two vectors -> their codes; s and m of the group (`lanes` lanes).
template <bool BF>
__device__ __forceinline__ uint2 quantise(const uint4 &v0, const uint4 &v1, int lanes, unsigned mask, uint32_t &sm) {
    const uint32_t w[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    uint32_t least = w[0], most = w[0] ^ 0x80008000u;                // of the negated values
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        least = min_2<BF>(least, w[i]);
        most = min_2<BF>(most, w[i] ^ 0x80008000u);
    }
    uint32_t ends = min_2<BF>(__byte_perm(least, most, 0x5410), __byte_perm(least, most, 0x7632));     // (least, -greatest)
    for (int o = 1; o < lanes; o <<= 1) ends = min_2<BF>(ends, __shfl_xor_sync(mask, ends, o));
    const float lo = unpack2<BF>(ends).x, hi = -unpack2<BF>(ends).y, span = __fsub_rn(hi, lo);
    if (!(span < INFINITY)) {
        const float nan = __int_as_float(0x7fffffff);
        sm = pack2<BF>(nan, nan);
        return make_uint2(0, 0);
    }
    sm = pack2<BF>(fifteenth(span), lo);
    const float step = unpack2<BF>(sm).x, by = __fdividef(1.f, step);
    constexpr float kRound = 12582912.f;
    // Whether fp32 may lack bits of a difference that matter: beside a tiny end (15 steps are the span but for the step's
    // rounding; a greatest element only bears on the step, whose borders bf16's spans miss), or where 0 is near a half
    // step.  A step of 0 makes `off` NaN.
    const float low = (BF ? 15.125f * 0x1p-16f : 15.125f * 0x1p-13f) * step;
    const float to0 = __fmaf_rn(-lo, by, -0.5f), off = __fsub_rn(to0, __fsub_rn(__fadd_rn(to0, kRound), kRound));
    const bool whole = span >= 1e-30f && (lo == 0.f || fabsf(lo) >= low) && (BF || hi == 0.f || fabsf(hi) >= low) &&
                       fabsf(off) > (BF ? 0x1p-12f : 0x1p-9f);
    // d / s to its last bit, the approximate quotient corrected by its remainder, so that a half is a half (in bf16 every
    // other warp has one); to the nearest by adding 1.5 2^23.  Four codes of a half word add up in fp32 as digits of base
    // 16.
    const uint64_t least2 = pair(-lo, -lo), by2 = pair(by, by), step2 = pair(-step, -step), round2 = pair(kRound, kRound);
    const uint64_t back2 = pair(-kRound, -kRound), base2 = pair(16.f, 16.f), whole2 = pair(8388608.f, 8388608.f);
    uint32_t c[2];
    float last = whole ? 0.f : 16.f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint64_t sum = 0;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const float2 f = unpack2<BF>(w[4 * h + i]);
            const uint64_t d = add2(pair(f.x, f.y), least2), near = fma2(d, by2, 0);
            const uint64_t q = add2(add2(fma2(fma2(near, step2, d), by2, near), round2), back2);
            const float2 k = unpair(q);
            last = max3(last, k.x, k.y);
            sum = fma2(sum, base2, q);
        }
        const float2 digits = unpair(add2(sum, whole2));
        c[h] = __byte_perm(__float_as_uint(digits.x), __float_as_uint(digits.y), 0x5410);
    }
    if (last <= 15.f) return make_uint2(c[0], c[1]);
    // also values past the last code (of a step that is a multiple of the type's least number), the smallest steps and none
    const uint3 r = quantise_exactly<BF>(v0, v1, lo, hi);
    sm = r.z;
    return make_uint2(r.x, r.y);
}

template <bool BF>
__global__ void __launch_bounds__(kThreads, 4)
    append4_kernel(AttnShape s, AttnBatch b, Cache4 c, AppendCall a, int tokens_per_cta) {
    __shared__ Token tok[kMaxTokens];
    __shared__ uint4 turned_rows[2 * kThreads];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * tokens_per_cta, nt = min(tokens_per_cta, b.tokens - t0);
    if (warp < nt) {
        const Token k = find_token(b, s, c.pages, t0 + warp, a.positions, a.rope ? a.max_pos : 0, a.status);
        if (lane == 0) tok[warp] = k;
    }
    __syncthreads();
    const int head_log2 = s.d == 64 ? 2 : 3, per_head = 1 << head_log2, per_token = (s.hq + 2 * s.hkv) << head_log2;
    const int half = a.rot / 2, turned = a.rope ? a.rot / 16 : 0;
    const int record = record_bytes(s.d, c.group_log2), group_lanes = 1 << (c.group_log2 - 4);
    const unsigned mask = ((1u << per_head) - 1) << (lane & ~(per_head - 1));                    // the head's lanes
    uint4 *row = turned_rows + 2 * (threadIdx.x & ~(per_head - 1));                              // the head's elements
    // a thread has the same place in every token
    for (int u = blockIdx.y * kThreads + threadIdx.x; u < per_token; u += gridDim.y * kThreads) {
        const int head = u >> head_log2, item = u & (per_head - 1);
        const bool query = head < s.hq, key = !query && head < s.hq + s.hkv;
        const bool turn = item < turned && (query || key);
        int e0 = 16 * item, e1 = e0 + 8;                 // first elements of the two vectors
        if (turn && !a.interleaved) {
            e0 = 8 * item;
            e1 = e0 + half;
        }
        const uint16_t *src = a.qkv + static_cast<int64_t>(t0) * a.qkv_stride + head * s.d;
        uint4 n0 = *reinterpret_cast<const uint4 *>(src + e0), n1 = *reinterpret_cast<const uint4 *>(src + e1);
        for (int ti = 0; ti < nt; ++ti) {
            const Token k = tok[ti];
            uint4 v0 = n0, v1 = n1;
            src += a.qkv_stride;
            if (ti + 1 < nt) {                           // the next token's, while this one's are worked on
                n0 = *reinterpret_cast<const uint4 *>(src + e0);
                n1 = *reinterpret_cast<const uint4 *>(src + e1);
            }
            if (k.page < 0) continue;
            const int64_t t = t0 + ti;
            if (turn) {
                const float4 *cs = reinterpret_cast<const float4 *>(a.rope + static_cast<int64_t>(k.pos) * half + 8 * item);
                uint32_t *p = reinterpret_cast<uint32_t *>(&v0), *q = reinterpret_cast<uint32_t *>(&v1);
                // queries are rounded once, whatever the last bit of the fp32 sum; keys go through a border
                auto rotate = [&](float x, float y, float co, float si) {
                    return key ? make_float2(cross(x, co, y, si), cross(y, co, -x, si)) : make_float2(x * co - y * si, y * co + x * si);
                };
#pragma unroll
                for (int e = 0; e < 4; ++e) {            // pairs 2e and 2e + 1 of the item's eight
                    const float4 r = cs[e];              // cos, sin, cos, sin
                    if (a.interleaved) {
                        uint32_t *x = e < 2 ? p + 2 * e : q + 2 * (e - 2);
                        const float2 m = unpack2<BF>(x[0]), n = unpack2<BF>(x[1]);
                        const float2 f = rotate(m.x, m.y, r.x, r.y), g = rotate(n.x, n.y, r.z, r.w);
                        x[0] = pack2<BF>(f.x, f.y);
                        x[1] = pack2<BF>(g.x, g.y);
                    } else {
                        const float2 m = unpack2<BF>(p[e]), n = unpack2<BF>(q[e]);
                        const float2 f = rotate(m.x, n.x, r.x, r.y), g = rotate(m.y, n.y, r.z, r.w);
                        p[e] = pack2<BF>(f.x, g.x);
                        q[e] = pack2<BF>(f.y, g.y);
                    }
                }
            }
            if (query) {
                uint16_t *dst = a.q_out + t * a.q_stride + head * s.d;
                *reinterpret_cast<uint4 *>(dst + e0) = v0;
                *reinterpret_cast<uint4 *>(dst + e1) = v1;
                continue;
            }
            if (key && turned && !a.interleaved) {       // to sixteen neighbours
                row[e0 / 8] = v0;
                row[e1 / 8] = v1;
                __syncwarp(mask);
                v0 = row[2 * item];
                v1 = row[2 * item + 1];
                __syncwarp(mask);
            }
            uint32_t sm;
            const uint2 codes = quantise<BF>(v0, v1, group_lanes, mask, sm);
            const int h = head - s.hq - (key ? 0 : s.hkv);
            uint8_t *dst = c.kv + k.page * c.page_stride + static_cast<int64_t>(h * s.page + k.slot) * record;
            *reinterpret_cast<uint2 *>(dst + (key ? 0 : s.d / 2) + 8 * item) = codes;
            if (item % group_lanes == 0)
                *reinterpret_cast<uint32_t *>(dst + s.d + (key ? 0 : 4 * s.d >> c.group_log2) + 4 * (item / group_lanes)) = sm;
        }
    }
}

struct ReadOut {
    uint16_t *k, *v;
    int64_t k_stride, v_stride;
    int *status;
};

// Work item: 16 elements of one head's key and value.
template <bool BF, bool FOUR>
__global__ void __launch_bounds__(kThreads)
    read_kernel(AttnShape s, AttnBatch b, AttnCache c, Cache4 c4, ReadOut o, int tokens_per_cta) {
    __shared__ Token tok[kMaxTokens];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = blockIdx.x * tokens_per_cta, nt = min(tokens_per_cta, b.tokens - t0);
    if (warp < nt) {
        const Token k = find_token(b, s, FOUR ? c4.pages : c.pages, t0 + warp, nullptr, 0, o.status);
        if (lane == 0) tok[warp] = k;
    }
    __syncthreads();
    const int per_head = s.d / 16, per_token = s.hkv * per_head;
    for (int w = threadIdx.x; w < nt * per_token; w += kThreads) {
        const int ti = w / per_token, u = w - ti * per_token, head = u / per_head, item = u - head * per_head;
        const Token k = tok[ti];
        if (k.page < 0) continue;
        const int64_t t = t0 + ti, slot = static_cast<int64_t>(head) * s.page + k.slot;
        uint4 out[4];
        if constexpr (FOUR) {
            const uint8_t *src = c4.kv + k.page * c4.page_stride + slot * record_bytes(s.d, c4.group_log2);
            const uint2 kc = *reinterpret_cast<const uint2 *>(src + 8 * item);
            const uint2 vc = *reinterpret_cast<const uint2 *>(src + s.d / 2 + 8 * item);
            const uint32_t *params = reinterpret_cast<const uint32_t *>(src + s.d);
            const int g = item >> (c4.group_log2 - 4);
            const uint32_t kp = params[g], vp = params[(s.d >> c4.group_log2) + g];
            out[0] = values_of<BF>(kc.x, both_low(kp), both_high(kp));
            out[1] = values_of<BF>(kc.y, both_low(kp), both_high(kp));
            out[2] = values_of<BF>(vc.x, both_low(vp), both_high(vp));
            out[3] = values_of<BF>(vc.y, both_low(vp), both_high(vp));
        } else {
            const int64_t at = k.page * c.page_stride + slot * s.d + 16 * item;
            out[0] = *reinterpret_cast<const uint4 *>(c.k + at);
            out[1] = *reinterpret_cast<const uint4 *>(c.k + at + 8);
            out[2] = *reinterpret_cast<const uint4 *>(c.v + at);
            out[3] = *reinterpret_cast<const uint4 *>(c.v + at + 8);
        }
        uint4 *kd = reinterpret_cast<uint4 *>(o.k + t * o.k_stride + head * s.d + 16 * item);
        uint4 *vd = reinterpret_cast<uint4 *>(o.v + t * o.v_stride + head * s.d + 16 * item);
        kd[0] = out[0];
        kd[1] = out[1];
        vd[0] = out[2];
        vd[1] = out[3];
    }
}

// Tokens of a CTA: one until the GPU is full, then up to `most`.
int tokens_each(int tokens, int most) { return std::max(1, std::min(most, tokens / 1216)); }

}  // namespace

cudaError_t launch_attn_append4(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AppendCall &a, bool bf16,
                                cudaStream_t st) {
    // few tokens: a CTA for every 256 items of each, so that none goes round its loop twice (64 tokens: 12.3 -> 8.3 us)
    const int per = tokens_each(b.tokens, 4), passes = ((s.hq + 2 * s.hkv) * (s.d / 16) + kThreads - 1) / kThreads;
    const dim3 grid((b.tokens + per - 1) / per, std::max(1, std::min(passes, 608 / b.tokens)));
    if (bf16) append4_kernel<true><<<grid, kThreads, 0, st>>>(s, b, c, a, per);
    else append4_kernel<false><<<grid, kThreads, 0, st>>>(s, b, c, a, per);
    return cudaGetLastError();
}

cudaError_t launch_attn_read(const AttnShape &s, const AttnBatch &b, const AttnCache *c, const Cache4 *c4, uint16_t *k,
                             int64_t k_stride, uint16_t *v, int64_t v_stride, bool bf16, int *status, cudaStream_t st) {
    const ReadOut o{k, v, k_stride, v_stride, status};
    const int per = tokens_each(b.tokens, kMaxTokens), grid = (b.tokens + per - 1) / per;
    auto kernel = !c4 ? read_kernel<false, false> : bf16 ? read_kernel<true, true> : read_kernel<false, true>;
    kernel<<<grid, kThreads, 0, st>>>(s, b, c ? *c : AttnCache{}, c4 ? *c4 : Cache4{}, o, per);
    return cudaGetLastError();
}

}  // namespace q4
