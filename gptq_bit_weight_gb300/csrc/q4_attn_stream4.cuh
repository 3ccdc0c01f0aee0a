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
// One CTA per SM has teams of four such warps, each with a loader and a share
// of the work for itself.  The loader goes through the team's items, hands over
// each with its query fragments, and fills the team's ring of key tiles of 128
// tokens (records of a page and head are contiguous, one bulk copy); a warp has
// 32 tokens of a tile, and the four meet at the end of an item.  Pieces of
// items meet as in the kernel for the 16-bit cache.
//   Three CTAs of one team each took as long as the slowest: some had finished
// after 29 us and others after 67.  Teams that shared the items of a CTA met
// too often: 88 us for 64 ragged requests.
#pragma once
#include <climits>

#include "q4_attn_tma.cuh"
#include "q4_cache4.cuh"

namespace q4 {

namespace {

using namespace tc;

constexpr int kWarps = 4;                       // of a team, and a loader
constexpr int kKeys = kKt / kWarps;             // tokens of a warp in a tile
constexpr int kBlocks = kKeys / 16;             // of 16 tokens, the rows of an MMA

template <int D_, int GL_, int NT_, int TEAMS_>
struct Cfg {
    static constexpr int D = D_, GL = GL_, NT = NT_, kTeams = TEAMS_;
    static constexpr int kThreads = 32 * (kWarps + 1) * kTeams;
    static constexpr int kRecord = record_bytes(D, GL);
    static constexpr int kRows = 8 * NT;                        // rows of a row tile
    static constexpr int MT = D / 16;                           // MMAs along the value's elements
    static constexpr int kStage = kKt * kRecord;
    static constexpr int kQ = NT * (D / 32) * 32 * 16;          // query fragments, double-buffered for each team
    static constexpr int kSlot = NT * MT * 32 * 16 + NT * 4 * 16;      // a warp's part: fragments, (m, m, l, l)
    static constexpr int kMisc = 1536;
    static constexpr int kFixed = kTeams * (2 * kQ + kWarps / 2 * kSlot) + kMisc + 128;
    static constexpr int kRoom = (232448 - 1024 - kFixed) / kStage;
    static constexpr int kStages = (kRoom > 9 ? 9 : kRoom) / kTeams * kTeams;    // a team has its own
    static constexpr int kSmem = kStages * kStage + kFixed;
    static constexpr int kPiece = kRows * (D + 2);              // floats of a piece in the workspace
};

// An item as a loader hands it to its team.
struct Handed {
    Item it;
    int more;                    // 0: there is none
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
__device__ __forceinline__ void bar_team(int team) {
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * kWarps) : "memory");
}
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
__global__ void __launch_bounds__(C::kThreads, 1) attend_stream4_kernel(Args a) {
    constexpr int D = C::D, NT = C::NT, MT = C::MT, S = C::kStages, T = C::kTeams, R = C::kRecord, GL = C::GL;
    constexpr int WORDS = D / 32;                // words of a key's codes in a thread
    constexpr int OCT = D / 64;                  // words of a value's codes
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 127u) & ~127u;
    uint8_t *sb = smem_raw + (base - raw);
    uint4 *sq = reinterpret_cast<uint4 *>(sb + S * C::kStage);                            // [T][2][NT][WORDS][32]
    uint8_t *slots = sb + S * C::kStage + 2 * T * C::kQ;                                  // [T][kWarps / 2]
    uint8_t *misc = slots + T * (kWarps / 2) * C::kSlot;
    const uint32_t bar0 = smem_u32(misc);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto handed = [&](int team, int buf) { return bar0 + 8u * (2 * S + 2 * team + buf); };
    auto taken = [&](int team, int buf) { return bar0 + 8u * (2 * S + 2 * T + 2 * team + buf); };
    int *flags = reinterpret_cast<int *>(misc + 8 * (2 * S + 4 * T));                     // [T]
    Handed *items = reinterpret_cast<Handed *>(misc + 320);                               // [T][2]
    TeamSchedSmem<T> &sched = *reinterpret_cast<TeamSchedSmem<T> *>(misc + 1024);
    static_assert((4 * NT * 16 + 32 * 4 * NT * 8) <= kWarps / 2 * C::kSlot && S >= 2 * T && S % T == 0 && 8 * (2 * S + 4 * T) + 4 * T <= 320 && 320 + 2 * T * sizeof(Handed) <= 1024 &&
                      1024 + sizeof(TeamSchedSmem<T>) <= C::kMisc,
                  "shared memory");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), kWarps);
        }
        for (int t = 0; t < T; ++t)
            for (int i = 0; i < 2; ++i) {
                mbar_init(handed(t, i), 1);
                mbar_init(taken(t, i), kWarps);
            }
        mbar_init_fence();
    }
    const int team = warp < T * kWarps ? warp / kWarps : warp - T * kWarps;
    Item it;
    const Share sh = team_share<C::kThreads, T>(a.p, sched, team, blockIdx.x, gridDim.x, a.status, it);
    if (sh.begin >= sh.end) return;
    constexpr int ST = S / T;                    // stages of a team
    const int first_stage = team * ST;

    if (warp >= T * kWarps) {
        // -------------------------------------------------- loaders
        int stage = 0, filled = 0, bad = 0;
        uint32_t phase = 0;
        bool alive = true;
        const int g = lane >> 2, t4 = lane & 3, group = a.p.group.d;
        bool more = true;
        for (int k = 0;; ++k) {
            // the item and its query fragments to the team: row 8 n + g, a quarter of its elements
            more = more && it.u < sh.end;
            const int buf = k & 1, r_first = it.tile * C::kRows, rows = more ? it.ql * group - r_first : 0;
            uint4 q[NT * WORDS];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = 8 * n + g, rr = r_first + r, t = a.p.group(rr);
                const uint16_t *src = a.q + static_cast<int64_t>(it.q0 + t) * a.q_stride + (it.head * group + rr - t * group) * D + D / 4 * t4;
#pragma unroll
                for (int w = 0; w < WORDS; ++w)
                    q[n * WORDS + w] = r < rows ? *reinterpret_cast<const uint4 *>(src + 8 * w) : make_uint4(0, 0, 0, 0);
            }
            if (k >= 2) alive = wait_all(alive, taken(team, buf), ((k >> 1) & 1) ^ 1);
            if (!alive) break;
#pragma unroll
            for (int f = 0; f < NT * WORDS; ++f) sq[((2 * team + buf) * NT * WORDS + f) * 32 + lane] = q[f];
            if (lane == 0) items[2 * team + buf] = Handed{it, more};
            __syncwarp();
            if (lane == 0) mbar_arrive(handed(team, buf));
            if (!more) break;
            const int j0 = max(sh.begin - it.u, 0), j1 = it.hi > 0 ? min(sh.end - it.u, it.n) : j0;
            const PageWalk walk(a.p, it, a.c.pages);
            const int boxes = kKt >> walk.box_log2, bytes = R << walk.box_log2;
            const uint8_t *head = a.c.kv + static_cast<int64_t>(it.head << a.p.page_log2) * R;
            // lane i has page i of a tile; the table is read a tile ahead, and looked at when the tile's turn comes
            auto entry = [&](int j) {
                const int key = (key_tile(a.p, it, j) << kKtLog2) + (lane << walk.box_log2);
                return lane < boxes && sees_some(a.p, it, key, 1 << walk.box_log2) ? __ldg(walk.table + (key >> walk.page_log2)) : INT_MIN;
            };
            int next = j0 < j1 ? entry(j0) : INT_MIN;
            for (int j = j0; j < j1; ++j) {
                int page = next;
                if (j + 1 < j1) next = entry(j + 1);
                if (filled >= ST) alive = wait_all(alive, empty(first_stage + stage), phase ^ 1);
                if (!alive) break;
                const unsigned wanted = __ballot_sync(0xffffffffu, page != INT_MIN);
                if (page != INT_MIN && (page < 0 || page >= a.c.pages)) {
                    bad = kAttnBadPage;
                    page = 0;
                }
                const int row = (key_tile(a.p, it, j) << kKtLog2) & ((1 << walk.page_log2) - 1) & ~((1 << walk.box_log2) - 1);
                const uint8_t *src = head + row * R;
                const uint32_t dst = base + (first_stage + stage) * C::kStage, bar = full(first_stage + stage);
                __syncwarp();
                if (elect_one()) mbar_arrive_expect_tx(bar, __popc(wanted) * bytes);
#pragma unroll 1
                for (int i0 = 0; i0 < boxes; i0 += 4) {
                    int pg[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) pg[i] = __shfl_sync(0xffffffffu, page, i0 + i);
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (wanted >> (i0 + i) & 1) bulk_load(dst + (i0 + i) * bytes, src + pg[i] * a.c.page_stride, bytes, bar);
                    }
                    __syncwarp();
                }
                ++filled;
                if (++stage == ST) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            if (!alive) break;
            more = next_item(a.p, it);
        }
        if (bad) atomicOr(a.status, bad);
        if (!alive) {
            // a consumer stopped answering: let the copies in flight land before the CTA can exit
            if (lane == 0) atomicOr(a.status, kAttnTimeout);
            for (int i = 0; i < min(filled, ST); ++i) {  // the newest first
                if (--stage < 0) {
                    stage = ST - 1;
                    phase ^= 1;
                }
                wait_bounded(full(first_stage + stage), phase);
            }
        }
        return;
    }

    // ------------------------------------------------------ consumers
    const int g = lane >> 2, t4 = lane & 3, group = a.p.group.d;
    const int member = warp % kWarps, key_first = member * kKeys;             // of the warp's tokens in a tile
    const int key_row = key_first + token_of<R>(g);                           // and 8 further on
    const int val_row0 = key_first + token_of<R>(2 * t4), val_row1 = key_first + token_of<R>(2 * t4 + 1);
    const int k_at = key_row * R, va_at = val_row0 * R, vb_at = val_row1 * R;
    constexpr int kParams = D, vParams = D + 4 * (D >> GL);
    const int k_codes = 4 * WORDS * t4, k_param = kParams + 4 * ((D / 4 * t4) >> GL);
    const int v_codes = D / 2 + 4 * OCT * g, v_param = vParams + 4 * ((8 * OCT * g) >> GL);
    bool alive = true;
    int stage = 0;
    uint32_t phase = 0;
    for (int k = 0;; ++k) {
        const int buf = k & 1;
        alive = wait_all(alive, handed(team, buf), (k >> 1) & 1);
        alive = bar_and(1 + team, 32 * kWarps, alive);           // a team stays together
        if (!alive || !items[2 * team + buf].more) break;
        it = items[2 * team + buf].it;
        const int j0 = max(sh.begin - it.u, 0), j1 = min(sh.end - it.u, it.n);
        const int r_first = it.tile * C::kRows, rows = it.ql * group - r_first;    // of this tile: min(rows, kRows)
        const uint4 *qf = sq + (2 * team + buf) * NT * WORDS * 32;
        uint4 qr[WORDS];
        if constexpr (NT == 1)
#pragma unroll
            for (int w = 0; w < WORDS; ++w) qr[w] = qf[w * 32 + lane];
        // m: greatest score so far; ref: what exponents are taken against, m as it was when it last moved, 0 for -inf
        float o[NT][MT][4], m[NT][2], ref[NT][2], l[NT][2];
        int lim[NT][2], lim_lo[NT][2];                                 // last key that a row sees; last one before its window
        bool fresh = true;                                             // some row has seen no key
        const int own = it.kv - it.ql, lim_min = own + it.t0, lim_max = own + it.t1, window = a.p.window, sinks = a.p.sinks;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[n][e] = -INFINITY;
                ref[n][e] = l[n][e] = 0.f;
                lim[n][e] = own + min(a.p.group(r_first + 8 * n + 2 * t4 + e), it.t1);
                lim_lo[n][e] = window > 0 ? lim[n][e] - window : -1;
            }
        }
        // The products of two tiles go together, a tile's values and the next one's keys: neither waits for the other.
        // Scores of a tile: token key_row (+ 8 from e = 2 on, + 16 b), row 8 n + 2 t4 + (e & 1).
        float s[kBlocks][NT][4];
        uint32_t pb[kBlocks][NT][2];
        auto keys = [&](const uint8_t *stage, int b) {
            const uint8_t *r0 = stage + k_at + 16 * b * R, *r1 = r0 + 8 * R;
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
#pragma unroll
            for (int n = 0; n < NT; ++n) s[b][n][0] = s[b][n][1] = s[b][n][2] = s[b][n][3] = 0.f;
#pragma unroll
            for (int w = 0; w < WORDS; ++w) {
                const uint4 x = values_of<BF>(w0[w], s0, m0), y = values_of<BF>(w1[w], s1, m1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 q = NT == 1 ? qr[w] : qf[(n * WORDS + w) * 32 + lane];
                    mma16816<BF>(s[b][n], x.x, y.x, x.y, y.y, q.x, q.y);
                    mma16816<BF>(s[b][n], x.z, y.z, x.w, y.w, q.z, q.w);
                }
            }
        };
        auto values = [&](const uint8_t *stage, int b) {
            const uint8_t *ra = stage + va_at + 16 * b * R, *rb = stage + vb_at + 16 * b * R;
            uint32_t wa[2][OCT], wb[2][OCT], sv[2], mv[2];              // tokens 2 t4 and 2 t4 + 1, and 8 further on
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
                const uint32_t pa = *reinterpret_cast<const uint32_t *>(ra + 8 * h * R + v_param);
                const uint32_t pc = *reinterpret_cast<const uint32_t *>(rb + 8 * h * R + v_param);
                sv[h] = __byte_perm(pa, pc, 0x5410);
                mv[h] = __byte_perm(pa, pc, 0x7632);
            }
#pragma unroll
            for (int w = 0; w < OCT; ++w) {
                uint32_t x[2][2][4];                                   // [tokens][even, odd elements][4]
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
                    for (int n = 0; n < NT; ++n) mma16816<BF>(o[n][4 * w + i], a0, a1, a2, a3, pb[b][n][0], pb[b][n][1]);
                }
            }
        };
        // Scores to weights.  edge: some token is hidden from some row (a few instructions beside the rest: a copy of the
        // code for such tiles ran cold, 5 us where a tile takes 1).
        auto weights = [&](uint8_t *stage, int key0, bool edge) {
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[b][n][e] *= a.scale;
            if (edge) {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = key0 + key_row - key_first + 16 * b + (e & 2) * 4;
                            if (key > lim[n][e & 1] || (key <= lim_lo[n][e & 1] && key >= sinks)) s[b][n][e] = -INFINITY;
                        }
                // slots past the visible tokens hold anything: their values must not meet a weight of 0
                if (!sees_some(a.p, it, key0 + lane, 1)) {
                    uint32_t *params = reinterpret_cast<uint32_t *>(stage + (key_first + lane) * R + vParams);
#pragma unroll
                    for (int i = 0; i < D >> GL; ++i) params[i] = 0;
                }
                fence_proxy_async();                     // before the next copy to the stage
                __syncwarp();
            }
            float top = -INFINITY;                       // the most that a score is above its row's reference
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = fmaxf(top, s[b][n][e] - ref[n][e & 1]);
            if (__any_sync(0xffffffffu, top > kRescale || fresh)) {
                fresh = false;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float keep[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float high = m[n][c];
#pragma unroll
                        for (int b = 0; b < kBlocks; ++b) high = fmaxf(high, fmaxf(s[b][n][c], s[b][n][c + 2]));
                        high = max_g(high);
                        ref[n][c] = ref_of(high);
                        keep[c] = ex2(m[n][c] - ref[n][c]);
                        m[n][c] = high;
                        l[n][c] *= keep[c];
                        fresh |= high == -INFINITY;
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
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) p[e] = ex2(s[b][n][e] - ref[n][e & 1]);
                    l[n][0] += p[0] + p[2];
                    l[n][1] += p[1] + p[3];
                    pb[b][n][0] = transpose8(pack2<BF>(p[0], p[1]));
                    pb[b][n][1] = transpose8(pack2<BF>(p[2], p[3]));
                }
        };
        const int tiles = it.hi > 0 ? j1 - j0 : 0;
        auto next_stage = [&] {
            if (++stage == ST) {
                stage = 0;
                phase ^= 1;
            }
        };
        if (tiles) {
            int at = first_stage + stage;
            alive = wait_all(alive, full(at), phase);
            next_stage();
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) keys(sb + at * C::kStage, b);
#pragma unroll 1
            for (int j = j0; j < j0 + tiles; ++j) {
                const int key_t = key_tile(a.p, it, j) << kKtLog2;
                // tiles without a hidden token: all but the last and those at the window's ends
                const bool edge = key_t + kKt - 1 > lim_min || (window > 0 && key_t <= lim_max - window && key_t + kKt > sinks);
                uint8_t *here = sb + at * C::kStage;
                weights(here, key_t + key_first, edge);
                const bool more_tiles = j + 1 < j0 + tiles;
                const int now = at;
                if (more_tiles) {                        // (past the last tile its own keys go through once more, for nothing)
                    at = first_stage + stage;
                    alive = wait_all(alive, full(at), phase);
                    next_stage();
                }
                const uint8_t *there = sb + at * C::kStage;
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    values(here, b);
                    keys(there, b);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(now));
            }
        }
        // ---------------------------------------- the warps' parts of the keys, added in a fixed order
        __syncwarp();
        if (lane == 0) mbar_arrive(taken(team, buf));
        {
            // members 2 and 3 to 0 and 1
            float4 *w = reinterpret_cast<float4 *>(slots + (team * (kWarps / 2) + member % (kWarps / 2)) * C::kSlot);
            auto put = [&] {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
#pragma unroll
                    for (int i = 0; i < MT; ++i) w[(n * MT + i) * 32 + lane] = make_float4(o[n][i][0], o[n][i][1], o[n][i][2], o[n][i][3]);
                    if (g == 0) w[NT * MT * 32 + 4 * n + t4] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
                }
            };
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) l[n][e] = sum_g(l[n][e]);
            if (member >= kWarps / 2) put();
            bar_team(team);
            if (member < kWarps / 2) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float4 ml = w[NT * MT * 32 + 4 * n + t4];
                    float own_f[2], other[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float mo = e ? ml.y : ml.x, top = fmaxf(m[n][e], mo), r = ref_of(top);
                        own_f[e] = ex2(m[n][e] - r);
                        other[e] = ex2(mo - r);
                        m[n][e] = top;
                        l[n][e] = l[n][e] * own_f[e] + (e ? ml.w : ml.z) * other[e];
                    }
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const float4 v = w[(n * MT + i) * 32 + lane];
                        o[n][i][0] = o[n][i][0] * own_f[0] + v.x * other[0];
                        o[n][i][1] = o[n][i][1] * own_f[1] + v.y * other[1];
                        o[n][i][2] = o[n][i][2] * own_f[0] + v.z * other[0];
                        o[n][i][3] = o[n][i][3] * own_f[1] + v.w * other[1];
                    }
                }
                __syncwarp();                            // the last fragment of (m, l) has been read
                put();
            }
        }
        bar_team(team);
        // every warp: fragments member, member + 4, .. of both slots
        constexpr int F = (NT * MT + kWarps - 1) / kWarps;
        float4 acc[F];
        float top[F][2], sum[F][2];
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int f = min(member + u * kWarps, NT * MT - 1), n = f / MT;
            const float4 *w0 = reinterpret_cast<const float4 *>(slots + team * (kWarps / 2) * C::kSlot);
            const float4 *w1 = reinterpret_cast<const float4 *>(slots + (team * (kWarps / 2) + 1) * C::kSlot);
            const float4 v0 = w0[NT * MT * 32 + 4 * n + t4], v1 = w1[NT * MT * 32 + 4 * n + t4];
            const float4 x0 = w0[f * 32 + lane], x1 = w1[f * 32 + lane];
            top[u][0] = fmaxf(v0.x, v1.x);
            top[u][1] = fmaxf(v0.y, v1.y);
            const float r0 = ref_of(top[u][0]), r1 = ref_of(top[u][1]);
            const float a0 = ex2(v0.x - r0), a1 = ex2(v0.y - r1), b0 = ex2(v1.x - r0), b1 = ex2(v1.y - r1);
            sum[u][0] = v0.z * a0 + v1.z * b0;
            sum[u][1] = v0.w * a1 + v1.w * b1;
            acc[u] = make_float4(x0.x * a0 + x1.x * b0, x0.y * a1 + x1.y * b1, x0.z * a0 + x1.z * b0, x0.w * a1 + x1.w * b1);
        }
        // ---------------------------------------- output, or a piece for the workspace
        auto inverse = [](float sum) { return sum == 0.f ? 0.f : 1.f / sum; };
        // the thread's elements of row 8 n + 2 t4 + e
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
        // elements 2 i and 2 i + 1 of the thread's words, of both its rows
        auto store = [&](int f, const float4 &x, float l0, float l1) {
            const int n = f / MT, i = f - n * MT;
            if (uint16_t *dst = row_at(n, 0)) *reinterpret_cast<uint32_t *>(dst + 2 * i) = two(x.x, x.z, inverse(l0));
            if (uint16_t *dst = row_at(n, 1)) *reinterpret_cast<uint32_t *>(dst + 2 * i) = two(x.y, x.w, inverse(l1));
        };
        if (j0 == 0 && j1 == it.n) {
#pragma unroll
            for (int u = 0; u < F; ++u)
                if (member + u * kWarps < NT * MT) store(member + u * kWarps, acc[u], sum[u][0], sum[u][1]);
            continue;
        }
        // [NT][MT][32] float4 fragments, then [NT][4] (m, m, l, l) of a thread's two rows
        const int c0 = static_cast<uint32_t>(it.u) / sh.per, c1 = static_cast<uint32_t>(it.u + it.n - 1) / sh.per;
        auto piece = [&](int cta) {
            return reinterpret_cast<float4 *>(a.ws + static_cast<size_t>(2 * cta + (cta == c0)) * C::kPiece);
        };
        float4 *own_piece = piece(blockIdx.x * T + team);
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int f = member + u * kWarps;
            if (f >= NT * MT) continue;
            __stcg(own_piece + f * 32 + lane, acc[u]);
            if (f % MT == 0 && g == 0) __stcg(own_piece + NT * MT * 32 + 4 * (f / MT) + t4, make_float4(top[u][0], top[u][1], sum[u][0], sum[u][1]));
        }
        bar_team(team);
        if (member == 0 && lane == 0) {
            const int before = count_piece(a.tickets + c0);
            flags[team] = before == c1 - c0;
            if (before == c1 - c0) a.tickets[c0] = 0;
        }
        bar_team(team);
        if (!*reinterpret_cast<volatile int *>(flags + team)) continue;
        // The pieces' weights first, all at once, then their fragments, eight pieces at a time; in the order of the CTAs.
        const int pieces = c1 - c0 + 1;
        float4 *factors = reinterpret_cast<float4 *>(slots + team * (kWarps / 2) * C::kSlot);     // [n][t4]: (m, m, l, l) of all
        float *lifts = reinterpret_cast<float *>(factors + 4 * NT);                             // [32 pieces][n][t4][2]
        if (warp == team * kWarps) {
            // lane: piece lane / 4 of eight, row pair t4
            for (int n = 0; n < NT; ++n) {
                float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll 4
                for (int c = g; c < pieces; c += 8) {
                    const float4 v = __ldcg(piece(c0 + c) + NT * MT * 32 + 4 * n + t4);
                    const float h0 = fmaxf(m0, v.x), h1 = fmaxf(m1, v.y);
                    l0 = l0 * ex2(m0 - ref_of(h0)) + v.z * ex2(v.x - ref_of(h0));
                    l1 = l1 * ex2(m1 - ref_of(h1)) + v.w * ex2(v.y - ref_of(h1));
                    m0 = h0;
                    m1 = h1;
                }
                const float t0 = max_g(m0), t1 = max_g(m1);
                l0 = sum_g(l0 * ex2(m0 - ref_of(t0)));
                l1 = sum_g(l1 * ex2(m1 - ref_of(t1)));
                if (g == 0) factors[4 * n + t4] = make_float4(t0, t1, l0, l1);
            }
        }
        bar_team(team);
#pragma unroll
        for (int u = 0; u < F; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int cc = 0; cc < pieces; cc += 32) {
            const int here = min(32, pieces - cc);
            for (int i = threadIdx.x % (32 * kWarps); i < here * 4 * NT; i += 32 * kWarps) {
                const int c = i / (4 * NT), row = i - c * 4 * NT;
                const float4 v = __ldcg(piece(c0 + cc + c) + NT * MT * 32 + row), all = factors[row];
                lifts[2 * i] = ex2(v.x - ref_of(all.x));
                lifts[2 * i + 1] = ex2(v.y - ref_of(all.y));
            }
            bar_team(team);
#pragma unroll
            for (int u = 0; u < F; ++u) {
                const int f = min(member + u * kWarps, NT * MT - 1), n = f / MT;
#pragma unroll 1
                for (int c = 0; c < here; c += 8) {
                    float4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = __ldcg(piece(c0 + cc + min(c + k, here - 1)) + f * 32 + lane);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (c + k >= here) continue;
                        const float2 w = *reinterpret_cast<const float2 *>(lifts + 2 * ((c + k) * 4 * NT + 4 * n + t4));
                        acc[u].x += x[k].x * w.x;
                        acc[u].y += x[k].y * w.y;
                        acc[u].z += x[k].z * w.x;
                        acc[u].w += x[k].w * w.y;
                    }
                }
            }
            bar_team(team);
        }
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int f = member + u * kWarps;
            if (f >= NT * MT) continue;
            const float4 all = factors[4 * (f / MT) + t4];
            store(f, acc[u], all.z, all.w);
        }
    }
    if (!alive && lane == 0) atomicOr(a.status, kAttnTimeout);
}

template <class C>
cudaError_t launch(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                   cudaStream_t st) {
    constexpr int rows_log2 = C::NT == 1 ? 3 : 4;
    Args args{{b, s.hkv, s.page_log2, a.window, kKtLog2, FastDiv(s.group), rows_log2, FastDiv(1), a.sinks},
              c, a.q, a.out, a.q_stride, a.out_stride, a.scale * 1.4426950408889634f, a.ws, a.tickets, a.status};
    auto kernel = bf16 ? attend_stream4_kernel<true, C> : attend_stream4_kernel<false, C>;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem)) return e;
    kernel<<<a.ctas, C::kThreads, C::kSmem, st>>>(args);
    return cudaGetLastError();
}

// The kernel for row tiles of 8 NT rows.
template <int NT, int TEAMS>
cudaError_t launch_rows(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                        cudaStream_t st) {
    if (s.d == 64)
        return c.group_log2 == 5 ? launch<Cfg<64, 5, NT, TEAMS>>(s, b, c, a, bf16, st) : launch<Cfg<64, 6, NT, TEAMS>>(s, b, c, a, bf16, st);
    return c.group_log2 == 5 ? launch<Cfg<128, 5, NT, TEAMS>>(s, b, c, a, bf16, st) : launch<Cfg<128, 6, NT, TEAMS>>(s, b, c, a, bf16, st);
}

}  // namespace

}  // namespace q4
