// Attention of few new tokens over the paged cache: single tokens of a decode
// step, drafts of a few tokens.  The cache is streamed once through shared
// memory and the products run on mma.sync: with at most 64 query rows for
// each key the call is bound by reading the cache, not by the tensor cores.
//
//   scores s = scale log2(e) q . k in fp32; running maximum m and sum l,
//   p = 2^(s - m) rounded to 16 bits for its product with v (l sums the
//   unrounded ones), o = sum p v in fp32; o / l rounded once.
//
// One CTA per SM.  Warps 8 and 9 load key tiles of 128 tokens by TMA, keys and
// values, one box for each page and 64 columns, into a ring of half-stages
// (keys, values, keys, ..).  The other eight warps split each tile's tokens (and, from 64 rows on,
// the rows) and keep maximum, sum and output of their own; they join at the
// end of an item.  Items cut by the shares join through the workspace: the
// CTA whose piece arrives last adds the pieces in order.
#include <cuda.h>

#include <algorithm>
#include <cstdint>

#include "q4_attn_tma.cuh"

namespace q4 {

namespace {

using namespace tc;

constexpr int kWarps = 8;                       // consumer warps
constexpr int kThreads = 32 * (kWarps + 2);     // and two loaders

template <int D_, int MT_, int WR_>
struct Cfg {
    static constexpr int D = D_;
    static constexpr int MT = MT_;              // m16 tiles of rows of a warp
    static constexpr int WR = WR_;              // warps along the rows
    static constexpr int WK = kWarps / WR;      // warps along the keys
    static constexpr int RT = 16 * MT * WR;     // rows of a row tile
    static constexpr int kRtLog2 = RT == 16 ? 4 : RT == 32 ? 5 : 6;
    static constexpr int KPW = kKt / WK;        // keys of a warp in a tile
    static constexpr int kHalf = kKt * D * 2;   // bytes of a half-stage
    static constexpr int kQ = RT * D * 2;       // query fragments, double-buffered
    static constexpr int kMerge = kWarps / 2 * MT * 16 * D * 4 + kWarps / 2 * MT * 4 * 32 * 4;
    static constexpr int kMisc = 1024;
    static constexpr int kRoom = 232448 - 1024 - 2 * kQ - kMerge - kMisc;
    static constexpr int kStages = kRoom / kHalf > 6 ? 6 : kRoom / kHalf;
    static constexpr int kSmem = kStages * kHalf + 2 * kQ + kMerge + kMisc + 1024;
    static constexpr int kPiece = RT * (D + 2);  // floats of a piece in the workspace
};

struct Args {
    SchedParams p;
    AttnCache c;
    const uint16_t *q;
    uint16_t *out;
    int64_t q_stride, out_stride;
    float scale;                 // times log2(e)
    int hq;
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
    constexpr int D = C::D, MT = C::MT, WR = C::WR, WK = C::WK, KS = D / 16, NT = D / 8, S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sb = smem_raw + (base - raw);
    uint4 *sq = reinterpret_cast<uint4 *>(sb + S * C::kHalf);                     // [2][MT * WR][KS][32]
    float4 *so = reinterpret_cast<float4 *>(sb + S * C::kHalf + 2 * C::kQ);       // [kWarps / 2][MT][NT][32]
    float *sml = reinterpret_cast<float *>(so + kWarps / 2 * MT * NT * 32);       // [kWarps / 2][MT][4][32]
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
    const int wr = warp % WR, wk = warp / WR, g = lane >> 2, t4 = lane & 3;
    const int group = a.p.group.d;
    bool alive = true;
    int seq = 0, buf = 0;
    for (bool more = true; more && it.u < sh.end; more = next_item(a.p, it), buf ^= 1) {
        const int j0 = max(sh.begin - it.u, 0);
        const int j1 = min(sh.end - it.u, it.n);
        const int rows = it.ql * group - it.tile * C::RT;             // of this tile: min(rows, RT)
        // query rows, as MMA fragments
        uint4 *qf = sq + buf * (C::kQ / 16);
        for (int f = warp; f < MT * WR * KS; f += kWarps) {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = f / KS * 16 + g + 8 * h;
                if (r < rows) {
                    const int rr = it.tile * C::RT + r, t = a.p.group(rr);
                    const uint16_t *src = a.q + static_cast<int64_t>(it.q0 + t) * a.q_stride +
                                          (it.head * group + rr - t * group) * D + f % KS * 16 + 2 * t4;
                    w[h] = *reinterpret_cast<const uint32_t *>(src);
                    w[h + 2] = *reinterpret_cast<const uint32_t *>(src + 8);
                }
            }
            qf[f * 32 + lane] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        bar_consumers();

        float o[MT][NT][4], m[MT][2], l[MT][2];
        int lim[MT][2];                                                // last key that a row sees
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int n = 0; n < NT; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                m[i][h] = -INFINITY;
                l[i][h] = 0.f;
                const int r = it.tile * C::RT + (wr * MT + i) * 16 + g + 8 * h;
                lim[i][h] = it.kv - it.ql + min(a.p.group(r), it.t1);
            }
        }
        const int lim_min = it.kv - it.ql + it.t0, lim_max = it.kv - it.ql + it.t1;
        if (it.hi > 0) {
            for (int j = j0; j < j1; ++j, seq += 2) {
                const int sk = seq % S, sv = (seq + 1) % S;
                const int key_w = ((it.first + j) << kKtLog2) + wk * C::KPW;    // the warp's first key
                alive = wait_all(alive, full(sk), (seq / S) & 1);
                const uint32_t kb = base + sk * C::kHalf, vb = base + sv * C::kHalf;
                uint4 pf[MT];
#pragma unroll
                for (int sub = 0; sub < C::KPW / 16; ++sub) {
                    const int key0 = key_w + 16 * sub;
                    const bool some = key0 < it.hi && key0 + 16 > it.lo;
                    float s[MT][2][4];
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int n = 0; n < 2; ++n) s[i][n][0] = s[i][n][1] = s[i][n][2] = s[i][n][3] = 0.f;
                    if (some) {
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            // keys 0-7 x d 0-7, keys 0-7 x d 8-15, keys 8-15 x d 0-7, keys 8-15 x d 8-15
                            const int row = wk * C::KPW + 16 * sub + (lane & 7) + (lane >> 4) * 8;
                            const int ch = 2 * (k & 3) + ((lane >> 3) & 1);
                            uint32_t b[4];
                            ldsm4(kb + (k >> 2) * (kKt * 128) + row * 128 + ((ch ^ (row & 7)) << 4), b);
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                const uint4 q = qf[((wr * MT + i) * KS + k) * 32 + lane];
                                mma16816<BF>(s[i][0], q, b[0], b[1]);
                                mma16816<BF>(s[i][1], q, b[2], b[3]);
                            }
                        }
                    }
                    const bool edge = key0 + 15 > lim_min || (a.p.window > 0 && key0 <= lim_max - a.p.window);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                float x = s[i][n][e] * a.scale;
                                if (edge) {
                                    const int key = key0 + 8 * n + 2 * t4 + (e & 1), lm = lim[i][e >> 1];
                                    if (key > lm || (a.p.window > 0 && key <= lm - a.p.window)) x = -INFINITY;
                                }
                                s[i][n][e] = x;
                                top[e >> 1] = fmaxf(top[e >> 1], x);
                            }
                        float keep[2];
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                            top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
                            top[h] = fmaxf(top[h], m[i][h]);
                            keep[h] = ex2(m[i][h] - ref_of(top[h]));
                            m[i][h] = top[h];
                        }
                        if (__any_sync(0xffffffffu, keep[0] != 1.f || keep[1] != 1.f)) {
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                o[i][n][0] *= keep[0];
                                o[i][n][1] *= keep[0];
                                o[i][n][2] *= keep[1];
                                o[i][n][3] *= keep[1];
                            }
                            l[i][0] *= keep[0];
                            l[i][1] *= keep[1];
                        }
                        const float r0 = ref_of(m[i][0]), r1 = ref_of(m[i][1]);
                        float p[2][4];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            p[n][0] = ex2(s[i][n][0] - r0);
                            p[n][1] = ex2(s[i][n][1] - r0);
                            p[n][2] = ex2(s[i][n][2] - r1);
                            p[n][3] = ex2(s[i][n][3] - r1);
                            l[i][0] += p[n][0] + p[n][1];
                            l[i][1] += p[n][2] + p[n][3];
                        }
                        pf[i] = make_uint4(pack2<BF>(p[0][0], p[0][1]), pack2<BF>(p[0][2], p[0][3]),
                                           pack2<BF>(p[1][0], p[1][1]), pack2<BF>(p[1][2], p[1][3]));
                    }
                    if (sub == C::KPW / 16 - 1) {          // the warp has read its keys
                        __syncwarp();
                        if (lane == 0) mbar_arrive(empty(sk));
                    }
                    if (sub == 0) alive = wait_all(alive, full(sv), ((seq + 1) / S) & 1);
                    if (some) {
                        // slots past the visible keys hold anything: their values must not meet a weight of 0
                        const bool trim = key0 + 16 > it.hi || key0 < it.lo;
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
                            const int row = wk * C::KPW + 16 * sub + (lane & 7) + ((lane >> 3) & 1) * 8;
                            const int ch = 2 * (n2 & 3) + (lane >> 4);
                            uint32_t b[4];
                            ldsm4t(vb + (n2 >> 2) * (kKt * 128) + row * 128 + ((ch ^ (row & 7)) << 4), b);
                            if (trim) {
                                b[0] &= keep0;
                                b[1] &= keep1;
                                b[2] &= keep0;
                                b[3] &= keep1;
                            }
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                mma16816<BF>(o[i][2 * n2], pf[i], b[0], b[1]);
                                mma16816<BF>(o[i][2 * n2 + 1], pf[i], b[2], b[3]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(sv));
            }
        }
        // ---------------------------------------- the warps' parts of the keys, joined in a fixed order
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 1);
                l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 2);
            }
        // (of a single short tile only the first warps have keys)
        const int held = j1 - j0 > 1 ? WK : min(WK, (max(it.hi - ((it.first + j0) << kKtLog2), 1) + C::KPW - 1) / C::KPW);
#pragma unroll 1
        for (int half = WK / 2; half; half >>= 1) {
            if (half >= held) continue;
            if (wk >= half && wk < 2 * half) {
                const int slot = (wk - half) * WR + wr;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        so[((slot * MT + i) * NT + n) * 32 + lane] =
                            make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]);
                    float *ml = sml + (slot * MT + i) * 128 + lane;
                    ml[0] = m[i][0];
                    ml[32] = m[i][1];
                    ml[64] = l[i][0];
                    ml[96] = l[i][1];
                }
            }
            bar_consumers();
            if (wk < half) {
                const int slot = wk * WR + wr;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const float *ml = sml + (slot * MT + i) * 128 + lane;
                    float mine[2], other[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float mo = ml[32 * h], top = fmaxf(m[i][h], mo), r = ref_of(top);
                        mine[h] = ex2(m[i][h] - r);
                        other[h] = ex2(mo - r);
                        m[i][h] = top;
                        l[i][h] = l[i][h] * mine[h] + ml[64 + 32 * h] * other[h];
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float4 v = so[((slot * MT + i) * NT + n) * 32 + lane];
                        o[i][n][0] = o[i][n][0] * mine[0] + v.x * other[0];
                        o[i][n][1] = o[i][n][1] * mine[0] + v.y * other[0];
                        o[i][n][2] = o[i][n][2] * mine[1] + v.z * other[1];
                        o[i][n][3] = o[i][n][3] * mine[1] + v.w * other[1];
                    }
                }
            }
            bar_consumers();
        }
        // ---------------------------------------- output, or a piece for the workspace
        auto store = [&](int i_global, int n, int h, float x, float y, float inv) {
            const int r = i_global * 16 + g + 8 * h;
            if (r >= rows || r >= C::RT) return;
            const int rr = it.tile * C::RT + r, t = a.p.group(rr);
            *reinterpret_cast<uint32_t *>(a.out + static_cast<int64_t>(it.q0 + t) * a.out_stride +
                                          (it.head * group + rr - t * group) * D + 8 * n + 2 * t4) =
                pack2<BF>(x * inv, y * inv);
        };
        auto inverse = [](float sum) { return sum == 0.f ? 0.f : 1.f / sum; };
        if (j0 == 0 && j1 == it.n) {
            if (wk == 0)
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const float i0 = inverse(l[i][0]), i1 = inverse(l[i][1]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        store(wr * MT + i, n, 0, o[i][n][0], o[i][n][1], i0);
                        store(wr * MT + i, n, 1, o[i][n][2], o[i][n][3], i1);
                    }
                }
            continue;
        }
        const int c0 = static_cast<uint32_t>(it.u) / sh.per, c1 = static_cast<uint32_t>(it.u + it.n - 1) / sh.per;
        auto piece = [&](int cta) { return a.ws + static_cast<size_t>(2 * cta + (cta == c0)) * C::kPiece; };
        if (wk == 0) {
            float *w = piece(blockIdx.x);
            float4 *wo = reinterpret_cast<float4 *>(w);
            float4 *wml = wo + C::RT * D / 4;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int ig = wr * MT + i;
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    __stcg(wo + (ig * NT + n) * 32 + lane, make_float4(o[i][n][0], o[i][n][1], o[i][n][2], o[i][n][3]));
                if (t4 == 0) __stcg(wml + ig * 8 + g, make_float4(m[i][0], m[i][1], l[i][0], l[i][1]));
            }
            __threadfence();
        }
        bar_consumers();
        if (threadIdx.x == 0) {
            __threadfence();
            const int before = atomicAdd(a.tickets + c0, 1);
            *last_flag = before == c1 - c0;
            if (before == c1 - c0) a.tickets[c0] = 0;
            __threadfence();
        }
        bar_consumers();
        if (!*reinterpret_cast<volatile int *>(last_flag)) continue;
        for (int f = warp; f < MT * WR * (NT / 2); f += kWarps) {
            const int ig = f / (NT / 2), n0 = f % (NT / 2) * 2;
            float top0 = -INFINITY, top1 = -INFINITY;
            for (int c = c0; c <= c1; ++c) {
                const float4 v = __ldcg(reinterpret_cast<const float4 *>(piece(c)) + C::RT * D / 4 + ig * 8 + g);
                top0 = fmaxf(top0, v.x);
                top1 = fmaxf(top1, v.y);
            }
            const float r0 = ref_of(top0), r1 = ref_of(top1);
            float acc[2][4] = {}, l0 = 0.f, l1 = 0.f;
#pragma unroll 2
            for (int c = c0; c <= c1; ++c) {
                const float4 *w = reinterpret_cast<const float4 *>(piece(c));
                const float4 v = __ldcg(w + C::RT * D / 4 + ig * 8 + g);
                const float4 x = __ldcg(w + (ig * NT + n0) * 32 + lane), y = __ldcg(w + (ig * NT + n0 + 1) * 32 + lane);
                const float f0 = ex2(v.x - r0), f1 = ex2(v.y - r1);
                l0 += v.z * f0;
                l1 += v.w * f1;
                acc[0][0] += x.x * f0;
                acc[0][1] += x.y * f0;
                acc[0][2] += x.z * f1;
                acc[0][3] += x.w * f1;
                acc[1][0] += y.x * f0;
                acc[1][1] += y.y * f0;
                acc[1][2] += y.z * f1;
                acc[1][3] += y.w * f1;
            }
            const float i0 = inverse(l0), i1 = inverse(l1);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                store(ig, n0 + e, 0, acc[e][0], acc[e][1], i0);
                store(ig, n0 + e, 1, acc[e][2], acc[e][3], i1);
            }
        }
    }
    if (!alive && lane == 0) atomicOr(a.status, kAttnTimeout);
}

template <class C>
cudaError_t launch(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a, bool bf16,
                   const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t st) {
    Args args{{b, s.hkv, s.page_log2, a.window, kKtLog2, FastDiv(s.group), C::kRtLog2, FastDiv(1)}, c, a.q, a.out, a.q_stride, a.out_stride,
              a.scale * 1.4426950408889634f, s.hq, a.ws, a.tickets, a.status};
    auto kernel = bf16 ? attend_stream_kernel<true, C> : attend_stream_kernel<false, C>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e) return e;
    kernel<<<a.ctas, kThreads, C::kSmem, st>>>(tk, tv, args);
    return cudaGetLastError();
}

}  // namespace

size_t attend_stream_ws_bytes(int ctas) { return static_cast<size_t>(2) * ctas * Cfg<128, 2, 2>::kPiece * sizeof(float); }

cudaError_t launch_attend_stream(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a,
                                 bool bf16, cudaStream_t st) {
    CUtensorMap tk, tv;
    const uint32_t box = std::min(s.page, kKt);
    cudaError_t e = encode_pages(&tk, c.k, s, c, box);
    if (!e) e = encode_pages(&tv, c.v, s, c, box);
    if (e) return e;
    // row tiles of 16, 32 or 64 rows: the smallest that holds a request's
    const int64_t rows = static_cast<int64_t>(a.max_q) * s.group;
    auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        if (rows <= 16) return launch<Cfg<D, 1, 1>>(s, b, c, a, bf16, tk, tv, st);
        if (rows <= 32) return launch<Cfg<D, 2, 1>>(s, b, c, a, bf16, tk, tv, st);
        return launch<Cfg<D, 2, 2>>(s, b, c, a, bf16, tk, tv, st);
    };
    return s.d == 64 ? go(std::integral_constant<int, 64>{}) : go(std::integral_constant<int, 128>{});
}

}  // namespace q4
