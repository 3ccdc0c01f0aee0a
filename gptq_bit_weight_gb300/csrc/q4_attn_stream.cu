// Attention of few new tokens over the paged cache: single tokens of a decode
// step, drafts of a few tokens.  The cache is streamed once through shared
// memory and the products run on mma.sync in tiles of 16 query rows (token x
// query head of the group): bound by reading the cache, not by the tensor
// cores.  64 requests of up to 8192 tokens, 64 heads over 8: 131 us, 6.2 TB/s;
// two of 131071 and about 100000: 103 us, 6.3 TB/s; one of 777, 32 heads: 11
// us, latency (lengths, page table, keys, the join of the pieces).
//
//   scores s = scale log2(e) q . k in fp32; running maximum m and sum l,
//   p = 2^(s - m) rounded to 16 bits for its product with v (l sums the
//   unrounded ones), o = sum p v in fp32; o / l rounded once.
//   One 16-bit part of p, as in the kernel for chunks, where a second would cost:
//   either kernel rounds alike.  The result's error against 64 bits is 1.04 to
//   1.08 times that of rounding the exact result (relative, bf16 1.7e-3, fp16
//   2.2e-4).
//
// One CTA per SM.  Warps 8 and 9 load key tiles of 128 tokens by TMA, keys and
// values, one box for each page and 64 columns, into a ring of half-stages
// (keys, values, keys, ..).  The other eight warps split each tile's tokens,
// 16 each, and keep maximum, sum and output of their own, so a tile needs no
// synchronization among them; they join at the end of an item.  Items cut by
// the shares join through the workspace: the CTA whose piece arrives last adds
// the pieces in order.
#include <cuda.h>

#include <algorithm>
#include <cstdint>

#include "q4_attn_tma.cuh"

namespace q4 {

namespace {

using namespace tc;

constexpr int kWarps = 8;                       // consumer warps
constexpr int kThreads = 32 * (kWarps + 2);     // and two loaders

constexpr int kRows = 16, kRowsLog2 = 4;        // rows of a row tile: one m16 MMA tile
constexpr int kKeys = kKt / kWarps;             // keys of a warp in a tile

template <int D_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr int kHalf = kKt * D * 2;   // bytes of a half-stage
    static constexpr int kQ = kRows * D * 2;    // query fragments, double-buffered
    static constexpr int kMerge = kWarps / 2 * (kRows * D * 4 + 4 * 32 * 4);
    static constexpr int kMisc = 1024;
    static constexpr int kRoom = 232448 - 1024 - 2 * kQ - kMerge - kMisc;
    static constexpr int kStages = kRoom / kHalf > 10 ? 10 : kRoom / kHalf;
    static constexpr int kSmem = kStages * kHalf + 2 * kQ + kMerge + kMisc + 1024;
    static constexpr int kPiece = kRows * (D + 2);   // floats of a piece in the workspace
};

struct Args {
    SchedParams p;
    AttnCache c;
    const uint16_t *q;
    uint16_t *out;
    int64_t q_stride, out_stride;
    float scale;                 // times log2(e)
    float *ws;                   // [2 * CTAs] pieces
    int *tickets;                // [CTAs], zero between calls
    int *status;
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint4 &a, uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }
// 2^x; 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The subtrahend of exponents under a running maximum that may still be -inf.
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }

template <bool BF, class C>
__global__ void __launch_bounds__(kThreads, 1)
    attend_stream_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, Args a) {
    constexpr int D = C::D, KS = D / 16, NT = D / 8, S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sb = smem_raw + (base - raw);
    uint4 *sq = reinterpret_cast<uint4 *>(sb + S * C::kHalf);                     // [2][KS][32]
    float4 *so = reinterpret_cast<float4 *>(sb + S * C::kHalf + 2 * C::kQ);       // [kWarps / 2][NT][32]
    float *sml = reinterpret_cast<float *>(so + kWarps / 2 * NT * 32);            // [kWarps / 2][4][32]
    uint8_t *misc = sb + S * C::kHalf + 2 * C::kQ + C::kMerge;
    const uint32_t bar0 = base + S * C::kHalf + 2 * C::kQ + C::kMerge;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    int *last_flag = reinterpret_cast<int *>(misc + 16 * S);
    SchedSmem &sched = *reinterpret_cast<SchedSmem *>(misc + 256);
    static_assert(16 * S + 4 <= 256 && 256 + sizeof(SchedSmem) <= C::kMisc, "misc region");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (const CUtensorMap *map : {&tmK, &tmV}) asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kWarps);
        }
        mbar_init_fence();
    }
    Item it;
    const Share sh = sched_share<kThreads>(a.p, sched, blockIdx.x, gridDim.x, a.status, it);
    if (sh.begin >= sh.end) return;

    if (warp >= kWarps) {
        // -------------------------------------------------- loaders: keys, values
        const bool values = warp > kWarps;
        int seq = values, bad = 0;
        bool alive = true;
        for (bool more = true; more && it.u < sh.end && alive; more = next_item(a.p, it)) {
            if (it.hi <= 0) continue;
            const int j0 = max(sh.begin - it.u, 0);
            const int j1 = min(sh.end - it.u, it.n);
            const PageWalk walk(a.p, it, a.c.pages);
            TilePages next = walk.tile(it, j0, bad);
            for (int j = j0; j < j1; ++j, seq += 2) {
                const TilePages t = next;
                if (j + 1 < j1) next = walk.tile(it, j + 1, bad);            // on its way while this one waits
                const int s = seq % S;
                if (seq >= S) alive = wait_all(alive, empty(s), ((seq / S) & 1) ^ 1);
                if (!alive) break;
                walk.copy<D>(t, base + s * C::kHalf, values ? &tmV : &tmK, full(s), it.head);
            }
        }
        if (bad) atomicOr(a.status, bad);
        if (!alive) {
            // a consumer stopped answering: let the copies in flight land before the CTA can exit
            if (lane == 0) atomicOr(a.status, kAttnTimeout);
            for (int i = seq - 2; i >= 0 && i > seq - 2 - S; i -= 2) wait_bounded(full(i % S), (i / S) & 1);
        }
        return;
    }

    // ------------------------------------------------------ consumers
    const int g = lane >> 2, t4 = lane & 3, group = a.p.group.d;
    bool alive = true;
    int seq = 0, buf = 0;
    for (bool more = true; more && it.u < sh.end; more = next_item(a.p, it), buf ^= 1) {
        const int j0 = max(sh.begin - it.u, 0);
        const int j1 = min(sh.end - it.u, it.n);
        const int r_first = it.tile * kRows, rows = it.ql * group - r_first;       // of this tile: min(rows, 16)
        // query rows, as MMA fragments
        uint4 *qf = sq + buf * (C::kQ / 16);
        for (int f = warp; f < KS; f += kWarps) {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = g + 8 * h;
                if (r < rows) {
                    const int rr = r_first + r, t = a.p.group(rr);
                    const uint16_t *src = a.q + static_cast<int64_t>(it.q0 + t) * a.q_stride +
                                          (it.head * group + rr - t * group) * D + f * 16 + 2 * t4;
                    w[h] = *reinterpret_cast<const uint32_t *>(src);
                    w[h + 2] = *reinterpret_cast<const uint32_t *>(src + 8);
                }
            }
            qf[f * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        bar_consumers();

        float o[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        int lim[2];                                                    // last key that a row sees
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) lim[h] = it.kv - it.ql + min(a.p.group(r_first + g + 8 * h), it.t1);
        const int lim_min = it.kv - it.ql + it.t0, lim_max = it.kv - it.ql + it.t1;
        if (it.hi > 0) {
            for (int j = j0; j < j1; ++j, seq += 2) {
                const int sk = seq % S, sv = (seq + 1) % S;
                const int key0 = ((it.first + j) << kKtLog2) + warp * kKeys;       // the warp's first key
                alive = wait_all(alive, full(sk), (seq / S) & 1);
                const uint32_t kb = base + sk * C::kHalf, vb = base + sv * C::kHalf;
                const bool some = key0 < it.hi && key0 + kKeys > it.lo;
                float s[2][4] = {};
                if (some) {
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        // keys 0-7 x d 0-7, keys 0-7 x d 8-15, keys 8-15 x d 0-7, keys 8-15 x d 8-15
                        const int row = warp * kKeys + (lane & 7) + (lane >> 4) * 8;
                        const int ch = 2 * (k & 3) + ((lane >> 3) & 1);
                        uint32_t b[4];
                        ldsm4(kb + (k >> 2) * (kKt * 128) + row * 128 + ((ch ^ (row & 7)) << 4), b);
                        const uint4 q = qf[k * 32 + lane];
                        mma16816<BF>(s[0], q, b[0], b[1]);
                        mma16816<BF>(s[1], q, b[2], b[3]);
                    }
                }
                const bool edge = key0 + kKeys - 1 > lim_min || (a.p.window > 0 && key0 <= lim_max - a.p.window);
                float top[2] = {-INFINITY, -INFINITY}, keep[2];
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float x = s[n][e] * a.scale;
                        if (edge) {
                            const int key = key0 + 8 * n + 2 * t4 + (e & 1), lm = lim[e >> 1];
                            if (key > lm || (a.p.window > 0 && key <= lm - a.p.window)) x = -INFINITY;
                        }
                        s[n][e] = x;
                        top[e >> 1] = fmaxf(top[e >> 1], x);
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                    top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
                    top[h] = fmaxf(top[h], m[h]);
                    keep[h] = ex2(m[h] - ref_of(top[h]));
                    m[h] = top[h];
                }
                if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        o[n][0] *= keep[0];
                        o[n][1] *= keep[0];
                        o[n][2] *= keep[1];
                        o[n][3] *= keep[1];
                    }
                    l[0] *= keep[0];
                    l[1] *= keep[1];
                }
                const float r0 = ref_of(m[0]), r1 = ref_of(m[1]);
                float p[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    p[n][0] = ex2(s[n][0] - r0);
                    p[n][1] = ex2(s[n][1] - r0);
                    p[n][2] = ex2(s[n][2] - r1);
                    p[n][3] = ex2(s[n][3] - r1);
                    l[0] += p[n][0] + p[n][1];
                    l[1] += p[n][2] + p[n][3];
                }
                const uint4 pf = make_uint4(pack2<BF>(p[0][0], p[0][1]), pack2<BF>(p[0][2], p[0][3]),
                                            pack2<BF>(p[1][0], p[1][1]), pack2<BF>(p[1][2], p[1][3]));
                alive = wait_all(alive, full(sv), ((seq + 1) / S) & 1);
                if (some) {
                    // slots past the visible keys hold anything: their values must not meet a weight of 0
                    const bool trim = key0 + kKeys > it.hi || key0 < it.lo;
                    uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                    if (trim) {
                        auto in = [&](int key) { return key >= it.lo && key < it.hi; };
                        const int k0 = key0 + 2 * t4;
                        keep0 = (in(k0) ? 0xffffu : 0u) | (in(k0 + 1) ? 0xffff0000u : 0u);
                        keep1 = (in(k0 + 8) ? 0xffffu : 0u) | (in(k0 + 9) ? 0xffff0000u : 0u);
                    }
#pragma unroll
                    for (int n2 = 0; n2 < NT / 2; ++n2) {
                        // keys 0-7 x d 0-7, keys 8-15 x d 0-7, keys 0-7 x d 8-15, keys 8-15 x d 8-15
                        const int row = warp * kKeys + (lane & 7) + ((lane >> 3) & 1) * 8;
                        const int ch = 2 * (n2 & 3) + (lane >> 4);
                        uint32_t b[4];
                        ldsm4t(vb + (n2 >> 2) * (kKt * 128) + row * 128 + ((ch ^ (row & 7)) << 4), b);
                        if (trim) {
                            b[0] &= keep0;
                            b[1] &= keep1;
                            b[2] &= keep0;
                            b[3] &= keep1;
                        }
                        mma16816<BF>(o[2 * n2], pf, b[0], b[1]);
                        mma16816<BF>(o[2 * n2 + 1], pf, b[2], b[3]);
                    }
                }
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(empty(sk));
                    mbar_arrive(empty(sv));
                }
            }
        }
        // ---------------------------------------- the warps' parts of the keys, joined in a fixed order
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
        }
        // (of a single short tile only the first warps have keys)
        const int held = j1 - j0 > 1 ? kWarps : min(kWarps, (max(it.hi - ((it.first + j0) << kKtLog2), 1) + kKeys - 1) / kKeys);
#pragma unroll 1
        for (int half = kWarps / 2; half; half >>= 1) {
            if (half >= held) continue;
            if (warp >= half && warp < 2 * half) {
                const int slot = warp - half;
#pragma unroll
                for (int n = 0; n < NT; ++n) so[(slot * NT + n) * 32 + lane] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
                float *ml = sml + slot * 128 + lane;
                ml[0] = m[0];
                ml[32] = m[1];
                ml[64] = l[0];
                ml[96] = l[1];
            }
            bar_consumers();
            if (warp < half) {
                const float *ml = sml + warp * 128 + lane;
                float mine[2], other[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float mo = ml[32 * h], top = fmaxf(m[h], mo), r = ref_of(top);
                    mine[h] = ex2(m[h] - r);
                    other[h] = ex2(mo - r);
                    m[h] = top;
                    l[h] = l[h] * mine[h] + ml[64 + 32 * h] * other[h];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float4 v = so[(warp * NT + n) * 32 + lane];
                    o[n][0] = o[n][0] * mine[0] + v.x * other[0];
                    o[n][1] = o[n][1] * mine[0] + v.y * other[0];
                    o[n][2] = o[n][2] * mine[1] + v.z * other[1];
                    o[n][3] = o[n][3] * mine[1] + v.w * other[1];
                }
            }
            bar_consumers();
        }
        // ---------------------------------------- output, or a piece for the workspace
        auto store = [&](int n, int h, float x, float y, float inv) {
            const int r = g + 8 * h;
            if (r >= rows) return;
            if (inv == 0.f) x = y = 0.f;                     // a row that sees nothing, beside whatever the values hold
            const int rr = r_first + r, t = a.p.group(rr);
            *reinterpret_cast<uint32_t *>(a.out + static_cast<int64_t>(it.q0 + t) * a.out_stride +
                                          (it.head * group + rr - t * group) * D + 8 * n + 2 * t4) =
                pack2<BF>(x * inv, y * inv);
        };
        auto inverse = [](float sum) { return sum == 0.f ? 0.f : 1.f / sum; };
        if (j0 == 0 && j1 == it.n) {
            if (warp == 0) {
                const float i0 = inverse(l[0]), i1 = inverse(l[1]);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    store(n, 0, o[n][0], o[n][1], i0);
                    store(n, 1, o[n][2], o[n][3], i1);
                }
            }
            continue;
        }
        // [NT][32] float4 fragments, then (m, l) of rows g and g + 8
        const int c0 = static_cast<uint32_t>(it.u) / sh.per, c1 = static_cast<uint32_t>(it.u + it.n - 1) / sh.per;
        auto piece = [&](int cta) {
            return reinterpret_cast<float4 *>(a.ws + static_cast<size_t>(2 * cta + (cta == c0)) * C::kPiece);
        };
        if (warp == 0) {
            float4 *w = piece(blockIdx.x);
#pragma unroll
            for (int n = 0; n < NT; ++n) __stcg(w + n * 32 + lane, make_float4(o[n][0], o[n][1], o[n][2], o[n][3]));
            if (t4 == 0) __stcg(w + NT * 32 + g, make_float4(m[0], m[1], l[0], l[1]));
        }
        bar_consumers();
        if (threadIdx.x == 0) {
            const int before = count_piece(a.tickets + c0);
            *last_flag = before == c1 - c0;
            if (before == c1 - c0) a.tickets[c0] = 0;
        }
        bar_consumers();
        if (!*reinterpret_cast<volatile int *>(last_flag)) continue;
        for (int n = 2 * warp; n < NT; n += 2 * kWarps) {
            float top0 = -INFINITY, top1 = -INFINITY;
            for (int c = c0; c <= c1; ++c) {
                const float4 v = __ldcg(piece(c) + NT * 32 + g);
                top0 = fmaxf(top0, v.x);
                top1 = fmaxf(top1, v.y);
            }
            const float r0 = ref_of(top0), r1 = ref_of(top1);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f), bcc = acc;
            float l0 = 0.f, l1 = 0.f;
#pragma unroll 2
            for (int c = c0; c <= c1; ++c) {
                const float4 *w = piece(c);
                const float4 v = __ldcg(w + NT * 32 + g), x = __ldcg(w + n * 32 + lane), y = __ldcg(w + (n + 1) * 32 + lane);
                const float f0 = ex2(v.x - r0), f1 = ex2(v.y - r1);
                l0 += v.z * f0;
                l1 += v.w * f1;
                acc.x += x.x * f0;
                acc.y += x.y * f0;
                acc.z += x.z * f1;
                acc.w += x.w * f1;
                bcc.x += y.x * f0;
                bcc.y += y.y * f0;
                bcc.z += y.z * f1;
                bcc.w += y.w * f1;
            }
            const float i0 = inverse(l0), i1 = inverse(l1);
            store(n, 0, acc.x, acc.y, i0);
            store(n, 1, acc.z, acc.w, i1);
            store(n + 1, 0, bcc.x, bcc.y, i0);
            store(n + 1, 1, bcc.z, bcc.w, i1);
        }
    }
    if (!alive && lane == 0) atomicOr(a.status, kAttnTimeout);
}

template <class C>
cudaError_t launch(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a, bool bf16,
                   cudaStream_t st) {
    CUtensorMap tk, tv;
    const uint32_t box = std::min(s.page, kKt);
    cudaError_t e = encode_pages(&tk, c.k, s, c, box);
    if (!e) e = encode_pages(&tv, c.v, s, c, box);
    if (e) return e;
    Args args{{b, s.hkv, s.page_log2, a.window, kKtLog2, FastDiv(s.group), kRowsLog2, FastDiv(1)},
              c, a.q, a.out, a.q_stride, a.out_stride, a.scale * 1.4426950408889634f, a.ws, a.tickets, a.status};
    auto kernel = bf16 ? attend_stream_kernel<true, C> : attend_stream_kernel<false, C>;
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem))) return e;
    kernel<<<a.ctas, kThreads, C::kSmem, st>>>(tk, tv, args);
    return cudaGetLastError();
}

}  // namespace

size_t attend_stream_ws_bytes(int ctas) { return static_cast<size_t>(2) * ctas * Cfg<128>::kPiece * sizeof(float); }

cudaError_t launch_attend_stream(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a,
                                 bool bf16, cudaStream_t st) {
    return s.d == 64 ? launch<Cfg<64>>(s, b, c, a, bf16, st) : launch<Cfg<128>>(s, b, c, a, bf16, st);
}

}  // namespace q4
