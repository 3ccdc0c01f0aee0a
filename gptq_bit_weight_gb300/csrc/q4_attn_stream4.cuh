// Attention of few new tokens over a paged cache held in 4 bits.  The cache is
// streamed once through shared memory as it lies (records of codes and
// parameters), decoded in registers and multiplied on mma.sync; a window with
// first tokens that stay visible only leaves tiles out.
//
//   scores s = scale log2(e) q . k in fp32; reference m and sum l of each row,
//   p = 2^(s - m) rounded to 16 bits for its product with v (l sums the
//   unrounded ones), o = sum p v in fp32; o / l rounded once.  m is raised only
//   when a score is more than 2^8 above it: any m gives the same result as long
//   as p fits 16 bits.
//
// Both products are turned round, keys (and the value's elements) as the rows
// of the MMA and the query rows as its columns: eight of them fill a tile,
// where the other way would take 16, and the operand that has to be decoded is
// the larger, A.  Its layout gives every thread whole runs of a record:
//   keys    thread (g, t) has rows g and g + 8 and along them a quarter of the
//           codes, one load; which elements an MMA multiplies is free as long as
//           the queries' fragment names the same
//   values  thread (g, t) has four tokens and of each the codes of one or two
//           words; halves of the words of two tokens joined give pairs of tokens
//           for one element, which is what A wants along the sum
//   weights the scores' fragment, transposed by movmatrix, is B
// One CTA has eight such warps, 16 tokens of a tile of 128 each, and a loader;
// records of a page and head are contiguous, one bulk copy.  Pieces of items
// meet as in the kernel for the 16-bit cache.
#pragma once
#include "q4_attn_tma.cuh"
#include "q4_cache4.cuh"

namespace q4 {

namespace {

using namespace tc;

constexpr int kWarps = 8;                       // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);     // and a loader
constexpr int kKeys = kKt / kWarps;             // tokens of a warp in a tile

template <int D_, int GL_, int NT_, int CTAS_>
struct Cfg {
    static constexpr int D = D_, GL = GL_, NT = NT_, kCtas = CTAS_;
    static constexpr int kRecord = record_bytes(D, GL);
    static constexpr int kRows = 8 * NT;                        // rows of a row tile
    static constexpr int MT = D / 16;                           // MMAs along the value's elements
    static constexpr int kStage = kKt * kRecord;
    static constexpr int kQ = NT == 1 ? 0 : NT * (D / 32) * 32 * 16;   // query fragments, double-buffered
    static constexpr int kMerge = kWarps / 2 * (NT * MT * 32 * 16 + NT * 4 * 16);
    static constexpr int kMisc = 1024;
    static constexpr int kRoom = 232448 / kCtas - 1024 - 128 - 2 * kQ - kMerge - kMisc;
    static constexpr int kStages = kRoom / kStage > 8 ? 8 : kRoom / kStage;
    static constexpr int kSmem = kStages * kStage + 2 * kQ + kMerge + kMisc + 128;
    static constexpr int kPiece = kRows * (D + 2);              // floats of a piece in the workspace
};

struct Args {
    SchedParamsT<true> p;
    Cache4 c;
    const uint16_t *q;
    uint16_t *out;
    int64_t q_stride, out_stride;
    float scale;                 // times log2(e)
    float *ws;                   // [2 * CTAs] pieces
    int *tickets;                // [CTAs], zero between calls
    int *status;
};

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ void bar_consumers() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }
// 2^x; 2^-inf = 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The subtrahend of exponents under a reference that may still be -inf.
__device__ __forceinline__ float ref_of(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float max_g(float v) {        // over the lanes of a column
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float sum_g(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// The token of row r of the eight in an MMA tile: an order in which the loads
// of neighbouring rows, a record apart, fall to different banks.
template <int RECORD>
__device__ __forceinline__ int token_of(int r) {
    if constexpr (RECORD == 160) return (r & 1) << 1 | (r >> 1 & 1) | (r & 4);
    else if constexpr (RECORD == 80) return (r & 3) << 1 | r >> 2;
    else return (r & 1) << 2 | r >> 1;
}

constexpr float kRescale = 8.f;                  // log2 of the growth that p may have

template <bool BF, class C>
__global__ void __launch_bounds__(kThreads, C::kCtas) attend_stream4_kernel(Args a) {
    constexpr int D = C::D, NT = C::NT, MT = C::MT, S = C::kStages, R = C::kRecord, GL = C::GL;
    constexpr int WORDS = D / 32;                // words of a key's codes in a thread
    constexpr int OCT = D / 64;                  // words of a value's codes
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 127u) & ~127u;
    uint8_t *sb = smem_raw + (base - raw);
    uint4 *sq = reinterpret_cast<uint4 *>(sb + S * C::kStage);                            // [2][NT][WORDS][32]
    float4 *so = reinterpret_cast<float4 *>(sb + S * C::kStage + 2 * C::kQ);              // [kWarps / 2][NT * MT][32]
    float4 *sml = so + kWarps / 2 * NT * MT * 32;                                         // [kWarps / 2][NT][4]
    uint8_t *misc = sb + S * C::kStage + 2 * C::kQ + C::kMerge;
    const uint32_t bar0 = base + S * C::kStage + 2 * C::kQ + C::kMerge;
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    int *last_flag = reinterpret_cast<int *>(misc + 16 * S);
    SchedSmem &sched = *reinterpret_cast<SchedSmem *>(misc + 256);
    static_assert(S >= 2 && 16 * S + 4 <= 256 && 256 + sizeof(SchedSmem) <= C::kMisc, "shared memory");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kWarps);
        }
        mbar_init_fence();
    }
    Item it;
    const Share sh = sched_share<kThreads>(a.p, sched, blockIdx.x, gridDim.x, a.status, it);
    if (sh.begin >= sh.end) return;

    if (warp == kWarps) {
        // -------------------------------------------------- loader
        int seq = 0, bad = 0;
        bool alive = true;
        for (bool more = true; more && it.u < sh.end && alive; more = next_item(a.p, it)) {
            if (it.hi <= 0) continue;
            const int j0 = max(sh.begin - it.u, 0), j1 = min(sh.end - it.u, it.n);
            const PageWalk walk(a.p, it, a.c.pages);
            const int boxes = kKt >> walk.box_log2, bytes = R << walk.box_log2;
            const uint8_t *head = a.c.kv + static_cast<int64_t>(it.head << a.p.page_log2) * R;
            TilePages next = walk.tile(a.p, it, j0, bad);
            for (int j = j0; j < j1; ++j, ++seq) {
                const TilePages t = next;
                if (j + 1 < j1) next = walk.tile(a.p, it, j + 1, bad);           // on its way while this one waits
                const int s = seq % S;
                if (seq >= S) alive = wait_all(alive, empty(s), ((seq / S) & 1) ^ 1);
                if (!alive) break;
                if (elect_one()) mbar_arrive_expect_tx(full(s), __popc(t.wanted) * bytes);
                __syncwarp();
                const uint32_t dst = base + s * C::kStage;
#pragma unroll 1
                for (int i = 0; i < boxes; ++i) {
                    const int page = __shfl_sync(0xffffffffu, t.page, i);
                    if ((t.wanted >> i & 1) && elect_one())
                        bulk_load(dst + i * bytes, head + page * a.c.page_stride + t.row * R, bytes, full(s));
                    __syncwarp();
                }
            }
        }
        if (bad) atomicOr(a.status, bad);
        if (!alive) {
            // a consumer stopped answering: let the copies in flight land before the CTA can exit
            if (lane == 0) atomicOr(a.status, kAttnTimeout);
            for (int i = seq - 1; i >= 0 && i > seq - 1 - S; --i) wait_bounded(full(i % S), (i / S) & 1);
        }
        return;
    }

    // ------------------------------------------------------ consumers
    const int g = lane >> 2, t4 = lane & 3, group = a.p.group.d;
    const int key_row = warp * kKeys + token_of<R>(g);                        // and 8 further on
    const int val_row0 = warp * kKeys + token_of<R>(2 * t4), val_row1 = warp * kKeys + token_of<R>(2 * t4 + 1);
    const uint8_t *k_at = sb + key_row * R, *va_at = sb + val_row0 * R, *vb_at = sb + val_row1 * R;
    constexpr int kParams = D, vParams = D + 4 * (D >> GL);
    const int k_codes = 4 * WORDS * t4, k_param = kParams + 4 * ((D / 4 * t4) >> GL);
    const int v_codes = D / 2 + 4 * OCT * g, v_param = vParams + 4 * ((8 * OCT * g) >> GL);
    bool alive = true;
    int seq = 0, buf = 0;
    for (bool more = true; more && it.u < sh.end; more = next_item(a.p, it), buf ^= 1) {
        const int j0 = max(sh.begin - it.u, 0), j1 = min(sh.end - it.u, it.n);
        const int r_first = it.tile * C::kRows, rows = it.ql * group - r_first;    // of this tile: min(rows, kRows)
        // queries: row 8 n + g, a quarter of its elements
        auto query = [&](int n, int w) {
            const int r = 8 * n + g;
            if (r >= rows) return make_uint4(0, 0, 0, 0);
            const int rr = r_first + r, t = a.p.group(rr);
            return *reinterpret_cast<const uint4 *>(a.q + static_cast<int64_t>(it.q0 + t) * a.q_stride +
                                                    (it.head * group + rr - t * group) * D + D / 4 * t4 + 8 * w);
        };
        uint4 qr[WORDS];
        uint4 *qf = sq + buf * (C::kQ / 16);
        if constexpr (NT == 1) {
#pragma unroll
            for (int w = 0; w < WORDS; ++w) qr[w] = query(0, w);
        } else {
            for (int f = warp; f < NT * WORDS; f += kWarps) qf[f * 32 + lane] = query(f / WORDS, f % WORDS);
            bar_consumers();
        }
        float o[NT][MT][4], m[NT][2], l[NT][2];
        int lim[NT][2];                                                // last key that a row sees
        const int own = it.kv - it.ql;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = -INFINITY;
                l[n][e] = 0.f;
                lim[n][e] = own + min(a.p.group(r_first + 8 * n + 2 * t4 + e), it.t1);
            }
        }
        const int lim_min = own + it.t0, lim_max = own + it.t1, window = a.p.window, sinks = a.p.sinks;
        if (it.hi > 0) {
            for (int j = j0; j < j1; ++j, ++seq) {
                const int st = seq % S;
                const int key0 = (key_tile(a.p, it, j) << kKtLog2) + warp * kKeys;     // the warp's first token
                alive = wait_all(alive, full(st), (seq / S) & 1);
                if (sees_some(a.p, it, key0, kKeys)) {
                    const int at = st * C::kStage;
                    float s[NT][4] = {};
                    {
                        const uint8_t *r0 = k_at + at, *r1 = r0 + 8 * R;
                        uint32_t w0[WORDS], w1[WORDS];
                        if constexpr (WORDS == 4) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(r0 + k_codes), y = *reinterpret_cast<const uint4 *>(r1 + k_codes);
                            w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
                            w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2 *>(r0 + k_codes), y = *reinterpret_cast<const uint2 *>(r1 + k_codes);
                            w0[0] = x.x, w0[1] = x.y;
                            w1[0] = y.x, w1[1] = y.y;
                        }
                        const uint32_t p0 = *reinterpret_cast<const uint32_t *>(r0 + k_param), p1 = *reinterpret_cast<const uint32_t *>(r1 + k_param);
                        const uint32_t s0 = both_low(p0), m0 = both_high(p0), s1 = both_low(p1), m1 = both_high(p1);
                        float s_odd[4] = {};                           // a second chain where there is one column tile
#pragma unroll
                        for (int w = 0; w < WORDS; ++w) {
                            const uint4 x = values_of<BF>(w0[w], s0, m0), y = values_of<BF>(w1[w], s1, m1);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                const uint4 q = NT == 1 ? qr[w] : qf[(n * WORDS + w) * 32 + lane];
                                mma16816<BF>(s[n], x.x, y.x, x.y, y.y, q.x, q.y);
                                mma16816<BF>(NT == 1 ? s_odd : s[n], x.z, y.z, x.w, y.w, q.z, q.w);
                            }
                        }
                        if constexpr (NT == 1)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[0][e] += s_odd[e];
                    }
                    // score e of a thread: token key_row (+ 8 from e = 2 on), row 8 n + 2 t4 + (e & 1)
                    const bool edge = key0 + kKeys - 1 > lim_min ||
                                      (window > 0 && key0 <= lim_max - window && key0 + kKeys > sinks);
                    const int key = key0 + key_row - warp * kKeys;
                    bool grows = false;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = s[n][e] * a.scale;
                            if (edge) {
                                const int kk = key + (e & 2) * 4, lm = lim[n][e & 1];
                                if (kk > lm || (window > 0 && kk <= lm - window && kk >= sinks)) x = -INFINITY;
                            }
                            s[n][e] = x;
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) grows |= fmaxf(s[n][e], s[n][e + 2]) > m[n][e] + kRescale;
                    }
                    if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            float keep[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const float top = fmaxf(m[n][e], max_g(fmaxf(s[n][e], s[n][e + 2])));
                                keep[e] = ex2(m[n][e] - ref_of(top));
                                m[n][e] = top;
                                l[n][e] *= keep[e];
                            }
#pragma unroll
                            for (int i = 0; i < MT; ++i) {
                                o[n][i][0] *= keep[0];
                                o[n][i][1] *= keep[1];
                                o[n][i][2] *= keep[0];
                                o[n][i][3] *= keep[1];
                            }
                        }
                    }
                    uint32_t pb[NT][2];
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float r0 = ref_of(m[n][0]), r1 = ref_of(m[n][1]);
                        const float p0 = ex2(s[n][0] - r0), p1 = ex2(s[n][1] - r1), p2 = ex2(s[n][2] - r0), p3 = ex2(s[n][3] - r1);
                        l[n][0] += p0 + p2;
                        l[n][1] += p1 + p3;
                        pb[n][0] = transpose8(pack2<BF>(p0, p1));
                        pb[n][1] = transpose8(pack2<BF>(p2, p3));
                    }
                    {
                        const uint8_t *ra = va_at + at, *rb = vb_at + at;
                        uint32_t wa[2][OCT], wb[2][OCT], sv[2], mv[2];          // tokens 2 t4 and 2 t4 + 1, and 8 further on
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if constexpr (OCT == 2) {
                                const uint2 x = *reinterpret_cast<const uint2 *>(ra + 8 * h * R + v_codes);
                                const uint2 y = *reinterpret_cast<const uint2 *>(rb + 8 * h * R + v_codes);
                                wa[h][0] = x.x, wa[h][1] = x.y;
                                wb[h][0] = y.x, wb[h][1] = y.y;
                            } else {
                                wa[h][0] = *reinterpret_cast<const uint32_t *>(ra + 8 * h * R + v_codes);
                                wb[h][0] = *reinterpret_cast<const uint32_t *>(rb + 8 * h * R + v_codes);
                            }
                            uint32_t pa = *reinterpret_cast<const uint32_t *>(ra + 8 * h * R + v_param);
                            uint32_t pc = *reinterpret_cast<const uint32_t *>(rb + 8 * h * R + v_param);
                            if (!sees_all(a.p, it, key0, kKeys)) {
                                // slots past the visible keys hold anything: their values must not meet a weight of 0
                                const int ka = key0 + val_row0 - warp * kKeys + 8 * h, kb = key0 + val_row1 - warp * kKeys + 8 * h;
                                if (!sees_some(a.p, it, ka, 1)) pa = 0;
                                if (!sees_some(a.p, it, kb, 1)) pc = 0;
                            }
                            sv[h] = __byte_perm(pa, pc, 0x5410);
                            mv[h] = __byte_perm(pa, pc, 0x7632);
                        }
#pragma unroll
                        for (int w = 0; w < OCT; ++w) {
                            uint32_t x[2][2][4];                               // [tokens][even, odd elements][4]
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                codes_of<BF>(__byte_perm(wa[h][w], wb[h][w], 0x5410), x[h][0]);
                                codes_of<BF>(__byte_perm(wa[h][w], wb[h][w], 0x7632), x[h][1]);
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t a0 = fma_2<BF>(x[0][0][i], sv[0], mv[0]), a1 = fma_2<BF>(x[0][1][i], sv[0], mv[0]);
                                const uint32_t a2 = fma_2<BF>(x[1][0][i], sv[1], mv[1]), a3 = fma_2<BF>(x[1][1][i], sv[1], mv[1]);
#pragma unroll
                                for (int n = 0; n < NT; ++n) mma16816<BF>(o[n][4 * w + i], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(st));
            }
        }
        // ---------------------------------------- the warps' parts of the keys, joined in a fixed order
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) l[n][e] = sum_g(l[n][e]);
        // (of a single short tile only the first warps have keys)
        const int held = j1 - j0 > 1 || it.hi <= 0
                             ? kWarps
                             : min(kWarps, (max(it.hi - (key_tile(a.p, it, j0) << kKtLog2), 1) + kKeys - 1) / kKeys);
#pragma unroll 1
        for (int half = kWarps / 2; half; half >>= 1) {
            if (half >= held) continue;
            if (warp >= half && warp < 2 * half) {
                const int slot = warp - half;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < MT; ++i)
                        so[(slot * NT * MT + n * MT + i) * 32 + lane] = make_float4(o[n][i][0], o[n][i][1], o[n][i][2], o[n][i][3]);
                    if (g == 0) sml[(slot * NT + n) * 4 + t4] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
                }
            }
            bar_consumers();
            if (warp < half) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float4 ml = sml[(warp * NT + n) * 4 + t4];
                    float mine[2], other[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mo = e ? ml.y : ml.x, top = fmaxf(m[n][e], mo), r = ref_of(top);
                        mine[e] = ex2(m[n][e] - r);
                        other[e] = ex2(mo - r);
                        m[n][e] = top;
                        l[n][e] = l[n][e] * mine[e] + (e ? ml.w : ml.z) * other[e];
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const float4 v = so[(warp * NT * MT + n * MT + i) * 32 + lane];
                        o[n][i][0] = o[n][i][0] * mine[0] + v.x * other[0];
                        o[n][i][1] = o[n][i][1] * mine[1] + v.y * other[1];
                        o[n][i][2] = o[n][i][2] * mine[0] + v.z * other[0];
                        o[n][i][3] = o[n][i][3] * mine[1] + v.w * other[1];
                    }
                }
            }
            bar_consumers();
        }
        // ---------------------------------------- output, or a piece for the workspace
        auto inverse = [](float sum) { return sum == 0.f ? 0.f : 1.f / sum; };
        // elements 2 i and 2 i + 1 of the thread's word w, of row 8 n + 2 t4 + e
        auto row_at = [&](int n, int e) -> uint16_t * {
            const int r = 8 * n + 2 * t4 + e;
            if (r >= rows) return nullptr;
            const int rr = r_first + r, t = a.p.group(rr);
            return a.out + static_cast<int64_t>(it.q0 + t) * a.out_stride + (it.head * group + rr - t * group) * D + 8 * OCT * g;
        };
        auto two = [](float x, float y, float inv) {
            if (inv == 0.f) x = y = 0.f;                     // a row that sees nothing, beside whatever the values hold
            return pack2<BF>(x * inv, y * inv);
        };
        if (j0 == 0 && j1 == it.n) {
            if (warp == 0) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        uint16_t *dst = row_at(n, e);
                        if (!dst) continue;
                        const float inv = inverse(l[n][e]);
#pragma unroll
                        for (int w = 0; w < OCT; ++w) {
                            float(*x)[4] = o[n] + 4 * w;
                            *reinterpret_cast<uint4 *>(dst + 8 * w) =
                                make_uint4(two(x[0][e], x[0][e + 2], inv), two(x[1][e], x[1][e + 2], inv),
                                           two(x[2][e], x[2][e + 2], inv), two(x[3][e], x[3][e + 2], inv));
                        }
                    }
            }
            continue;
        }
        // [NT][MT][32] float4 fragments, then [NT][4] (m, m, l, l) of a thread's two rows
        const int c0 = static_cast<uint32_t>(it.u) / sh.per, c1 = static_cast<uint32_t>(it.u + it.n - 1) / sh.per;
        auto piece = [&](int cta) {
            return reinterpret_cast<float4 *>(a.ws + static_cast<size_t>(2 * cta + (cta == c0)) * C::kPiece);
        };
        if (warp == 0) {
            float4 *w = piece(blockIdx.x);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    __stcg(w + (n * MT + i) * 32 + lane, make_float4(o[n][i][0], o[n][i][1], o[n][i][2], o[n][i][3]));
                if (g == 0) __stcg(w + NT * MT * 32 + 4 * n + t4, make_float4(m[n][0], m[n][1], l[n][0], l[n][1]));
            }
        }
        bar_consumers();
        if (threadIdx.x == 0) {
            const int before = count_piece(a.tickets + c0);
            *last_flag = before == c1 - c0;
            if (before == c1 - c0) a.tickets[c0] = 0;
        }
        bar_consumers();
        if (!*reinterpret_cast<volatile int *>(last_flag)) continue;
        for (int f = warp; f < NT * MT; f += kWarps) {
            const int n = f / MT, i = f - n * MT;
            float top0 = -INFINITY, top1 = -INFINITY;
            for (int c = c0; c <= c1; ++c) {
                const float4 v = __ldcg(piece(c) + NT * MT * 32 + 4 * n + t4);
                top0 = fmaxf(top0, v.x);
                top1 = fmaxf(top1, v.y);
            }
            const float r0 = ref_of(top0), r1 = ref_of(top1);
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float l0 = 0.f, l1 = 0.f;
#pragma unroll 4
            for (int c = c0; c <= c1; ++c) {
                const float4 *w = piece(c);
                const float4 v = __ldcg(w + NT * MT * 32 + 4 * n + t4), x = __ldcg(w + f * 32 + lane);
                const float f0 = ex2(v.x - r0), f1 = ex2(v.y - r1);
                l0 += v.z * f0;
                l1 += v.w * f1;
                acc.x += x.x * f0;
                acc.y += x.y * f1;
                acc.z += x.z * f0;
                acc.w += x.w * f1;
            }
            const float i0 = inverse(l0), i1 = inverse(l1);
            if (uint16_t *dst = row_at(n, 0)) *reinterpret_cast<uint32_t *>(dst + 2 * i) = two(acc.x, acc.z, i0);
            if (uint16_t *dst = row_at(n, 1)) *reinterpret_cast<uint32_t *>(dst + 2 * i) = two(acc.y, acc.w, i1);
        }
    }
    if (!alive && lane == 0) atomicOr(a.status, kAttnTimeout);
}

template <class C>
cudaError_t launch(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                   cudaStream_t st) {
    constexpr int rows_log2 = C::NT == 1 ? 3 : C::NT == 2 ? 4 : 5;
    Args args{{b, s.hkv, s.page_log2, a.window, kKtLog2, FastDiv(s.group), rows_log2, FastDiv(1), a.sinks},
              c, a.q, a.out, a.q_stride, a.out_stride, a.scale * 1.4426950408889634f, a.ws, a.tickets, a.status};
    auto kernel = bf16 ? attend_stream4_kernel<true, C> : attend_stream4_kernel<false, C>;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) return e;
    kernel<<<a.ctas * C::kCtas, kThreads, C::kSmem, st>>>(args);
    return cudaGetLastError();
}

// The kernel for row tiles of 8 NT rows.
template <int NT, int CTAS>
cudaError_t launch_rows(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                        cudaStream_t st) {
    if (s.d == 64)
        return c.group_log2 == 5 ? launch<Cfg<64, 5, NT, CTAS>>(s, b, c, a, bf16, st) : launch<Cfg<64, 6, NT, CTAS>>(s, b, c, a, bf16, st);
    return c.group_log2 == 5 ? launch<Cfg<128, 5, NT, CTAS>>(s, b, c, a, bf16, st) : launch<Cfg<128, 6, NT, CTAS>>(s, b, c, a, bf16, st);
}

}  // namespace

}  // namespace q4
