// Attention of few new tokens over a paged cache held in 4 bits.  The cache is
// streamed once through shared memory as it lies (records of codes and
// parameters), decoded in registers and multiplied on mma.sync; a window with
// first tokens that stay visible only leaves tiles out.
//
//   scores s = scale log2(e) q . k in fp32; reference m and sum l of each row,
//   p = 2^(s - m) rounded to 16 bits for its product with v (l sums the
//   unrounded ones), o = sum p v in fp32; o / l rounded once.  m is the greatest
//   score, in fp16 less weight_lift, and is raised only when a score is more than
//   2^8 above that: any m gives the same result as long as p fits 16 bits at both
//   ends.
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
// 64 requests of up to 8192 tokens, 64 heads over 8 of 128, groups of 32: 70.5
// us (the 16-bit cache: 132); two of 131071 and about 100000, groups of 64: 61
// (103); one of 777, 32 heads: 10 (latency, as there).  Reading the cache alone
// runs at 7.0 TB/s, the decoding and products on tiles that are there at 6.0;
// together 5.8 in the middle of a long call, and 20 us go to its ends: lengths,
// first tiles (3 us), the ends of items (1.5 each), the join.  Of a block of 16
// tokens' 361 instructions 208 decode, on two pipes of half rate; issue slots
// are 66% busy there.  Keys multiplied as codes, with step and least value
// applied to the groups' sums, took as long.
#include <climits>

#include "q4_attn_tma.cuh"
#include "q4_cache4.cuh"

namespace q4 {

namespace {

using namespace tc;

constexpr int kWarps = 4;                       // of a team, and a loader
constexpr int kKeys = kKt / kWarps;             // tokens of a warp in a tile
constexpr int kRows = 8, kRowsLog2 = 3;         // rows of a row tile: the columns of an MMA
constexpr int kBlocks = kKeys / 16;             // of 16 tokens, the rows of an MMA

template <int D_, int GL_>
struct Cfg {
    static constexpr int D = D_, GL = GL_, kTeams = 3;
    static constexpr int kThreads = 32 * (kWarps + 1) * kTeams;
    static constexpr int kRecord = record_bytes(D, GL);
    static constexpr int MT = D / 16;                           // MMAs along the value's elements
    static constexpr int kStage = kKt * kRecord;
    static constexpr int kQ = (D / 32) * 32 * 16;               // query fragments, double-buffered for each team
    static constexpr int kSlot = MT * 32 * 16 + 4 * 16;      // a warp's part: fragments, (m, m, l, l)
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

// What of an item falls to a share.  The first tile stands for two units: an item's end, and the way to the next one,
// take a team as long as a tile does.
struct Part {
    int j0, j1;                  // its key tiles
    bool whole;                  // the share has all units
    __device__ Part(const Item &it, const Share &sh) {
        const int r0 = max(sh.begin - it.u, 0), r1 = min(sh.end - it.u, it.n + 1);
        j0 = r0 == 0 ? 0 : max(r0 - 1, 1);
        j1 = it.hi > 0 ? max(r1 - 1, 1) : j0;
        whole = r0 == 0 && r1 == it.n + 1;
    }
};

struct Args {
    SchedParamsT<true, 1> p;
    Cache4 c;
    const uint16_t *q;
    uint16_t *out;
    int64_t q_stride, out_stride;
    float scale;                 // times log2(e)
    float *ws;                   // [2 * shares] pieces
    int *tickets;                // [shares], zero between calls
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
// With sums from 0.
template <bool BF>
__device__ __forceinline__ void mma16816_0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                           uint32_t b1) {
    if constexpr (BF)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
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

constexpr float kRescale = 8.f;                  // log2 of the growth that p may have

template <bool BF, class C>
__global__ void __launch_bounds__(C::kThreads, 1) attend_stream4_kernel(Args a) {
    constexpr int D = C::D, MT = C::MT, S = C::kStages, T = C::kTeams, R = C::kRecord, GL = C::GL;
    constexpr int WORDS = D / 32;                // words of a key's codes in a thread
    constexpr int OCT = D / 64;                  // words of a value's codes
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 127u) & ~127u;
    uint8_t *sb = smem_raw + (base - raw);
    uint4 *sq = reinterpret_cast<uint4 *>(sb + S * C::kStage);                            // [T][2][WORDS][32]
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
    static_assert(S >= 2 * T && S % T == 0, "stages");
    static_assert(4 * 16 + 32 * 4 * 8 <= kWarps / 2 * C::kSlot, "what the join keeps in the slots");
    static_assert(8 * (2 * S + 4 * T) + 4 * T <= 320 && 320 + 2 * T * sizeof(Handed) <= 1024 &&
                      1024 + sizeof(TeamSchedSmem<T>) <= C::kMisc,
                  "misc region");

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
            // the item and its query fragments to the team: row g, a quarter of its elements
            more = more && it.u < sh.end;
            const int buf = k & 1, rr = it.tile * kRows + g, t = a.p.group(rr);
            const bool row = more && rr < it.ql * group;
            const uint16_t *src = a.q + static_cast<int64_t>(it.q0 + t) * a.q_stride + (it.head * group + rr - t * group) * D + D / 4 * t4;
            uint4 q[WORDS];
#pragma unroll
            for (int w = 0; w < WORDS; ++w) q[w] = row ? *reinterpret_cast<const uint4 *>(src + 8 * w) : make_uint4(0, 0, 0, 0);
            const Part part(it, sh);
            const int j0 = part.j0, j1 = more ? part.j1 : j0;
            const PageWalk walk(a.p, it, a.c.pages);
            const int boxes = kKt >> walk.box_log2, bytes = R << walk.box_log2;
            const uint8_t *head = a.c.kv + static_cast<int64_t>(it.head << a.p.page_log2) * R;
            // lane i has page i of a tile; the table is read a tile ahead, and looked at when the tile's turn comes
            auto entry = [&](int j) {
                const int key = (key_tile(a.p, it, j) << kKtLog2) + (lane << walk.box_log2);
                return lane < boxes && sees_some(a.p, it, key, 1 << walk.box_log2) ? __ldg(walk.table + (key >> walk.page_log2)) : INT_MIN;
            };
            int next = j0 < j1 ? entry(j0) : INT_MIN;
            if (k >= 2) alive = wait_all(alive, taken(team, buf), ((k >> 1) & 1) ^ 1);
            if (!alive) break;
#pragma unroll
            for (int w = 0; w < WORDS; ++w) sq[((2 * team + buf) * WORDS + w) * 32 + lane] = q[w];
            if (lane == 0) items[2 * team + buf] = Handed{it, more};
            __syncwarp();
            if (lane == 0) mbar_arrive(handed(team, buf));
            if (!more) break;
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
        const Part part(it, sh);
        const int j0 = part.j0;
        const int r_first = it.tile * kRows, rows = it.ql * group - r_first;    // of this tile: min(rows, kRows)
        uint4 qr[WORDS];
#pragma unroll
        for (int w = 0; w < WORDS; ++w) qr[w] = sq[((2 * team + buf) * WORDS + w) * 32 + lane];
        // of the thread's two rows: what exponents are taken against, the sum of its tokens' weights, whether a token was seen
        float o[MT][4] = {}, ref[2] = {0.f, 0.f};
        uint64_t l2 = 0;
        bool unseen[2] = {true, true};
        const int own = it.kv - it.ql, lim_min = own + it.t0, lim_max = own + it.t1, window = a.p.window, sinks = a.p.sinks;
        int lim[2], lim_lo[2];                                         // last token that a row sees; last one before its window
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            lim[e] = own + min(a.p.group(r_first + 2 * t4 + e), it.t1);
            lim_lo[e] = window > 0 ? lim[e] - window : -1;
        }
        // tiles without a hidden token: neither the last ones, nor at the windows' ends, nor of the first tokens
        const int plain_hi = (max(lim_min + 1, 0) >> kKtLog2) - it.first;
        const int plain_lo = max(it.near, window > 0 && lim_max >= window ? ((lim_max - window) >> kKtLog2) + 1 - it.first : 0);
        // The products of two tiles go together, a tile's values and the next one's keys: neither waits for the other.
        // Scores of a tile: token key_row (+ 8 from e = 2 on, + 16 b), row 2 t4 + (e & 1).
        float s[kBlocks][4];
        uint32_t pb[kBlocks][2];
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
            for (int w = 0; w < WORDS; ++w) {
                const uint4 x = values_of<BF>(w0[w], s0, m0), y = values_of<BF>(w1[w], s1, m1);
                if (w == 0) mma16816_0<BF>(s[b], x.x, y.x, x.y, y.y, qr[w].x, qr[w].y);
                else mma16816<BF>(s[b], x.x, y.x, x.y, y.y, qr[w].x, qr[w].y);
                mma16816<BF>(s[b], x.z, y.z, x.w, y.w, qr[w].z, qr[w].w);
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
                    mma16816<BF>(o[4 * w + i], a0, a1, a2, a3, pb[b][0], pb[b][1]);
                }
            }
        };
        // Scores to weights.  edge: some token is hidden from some row (a few instructions beside the rest: a copy of the
        // code for such tiles ran cold, 5 us where a tile takes 1).
        auto weights = [&](uint8_t *stage, int key0, bool edge) {
            const uint64_t scale2 = pair(a.scale, a.scale), ref2 = pair(-ref[0], -ref[1]);
            float x[kBlocks][4];                         // exponents
#pragma unroll
            for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    const float2 v = unpair(fma2(pair(s[b][e], s[b][e + 1]), scale2, ref2));
                    x[b][e] = v.x;
                    x[b][e + 1] = v.y;
                }
            if (edge) {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + key_row - key_first + 16 * b + (e & 2) * 4;
                        if (key > lim[e & 1] || (key <= lim_lo[e & 1] && key >= sinks)) x[b][e] = -INFINITY;
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
            float top = -INFINITY;
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) top = max3(max3(top, x[b][0], x[b][1]), x[b][2], x[b][3]);
            if (__any_sync(0xffffffffu, top > kRescale + weight_lift<BF> || unseen[0] || unseen[1])) {
                float keep[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float high = -INFINITY;
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) high = max3(high, x[b][c], x[b][c + 2]);
                    high = max_g(high);
                    // to the greatest so far; a row's first token sets it, up or down
                    const float over = high - weight_lift<BF>, up = high == -INFINITY ? 0.f : unseen[c] ? over : fmaxf(over, 0.f);
                    keep[c] = unseen[c] ? 1.f : ex2(-up);
                    unseen[c] = unseen[c] && high == -INFINITY;
                    ref[c] += up;
#pragma unroll
                    for (int b = 0; b < kBlocks; ++b) {
                        x[b][c] -= up;
                        x[b][c + 2] -= up;
                    }
                }
                l2 = fma2(l2, pair(keep[0], keep[1]), 0);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    o[i][0] *= keep[0];
                    o[i][1] *= keep[1];
                    o[i][2] *= keep[0];
                    o[i][3] *= keep[1];
                }
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const float p0 = ex2(x[b][0]), p1 = ex2(x[b][1]), p2 = ex2(x[b][2]), p3 = ex2(x[b][3]);
                l2 = add2(l2, add2(pair(p0, p1), pair(p2, p3)));
                pb[b][0] = transpose8(pack2<BF>(p0, p1));
                pb[b][1] = transpose8(pack2<BF>(p2, p3));
            }
        };
        const int tiles = part.j1 - j0;
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
                uint8_t *here = sb + at * C::kStage;
                weights(here, (key_tile(a.p, it, j) << kKtLog2) + key_first, j < plain_lo || j >= plain_hi);
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
            // members 2 and 3 to 0 and 1; a row without a token has no reference
            const float2 sums = unpair(l2);
            float m[2], l[2] = {sum_g(sums.x), sum_g(sums.y)};
#pragma unroll
            for (int e = 0; e < 2; ++e) m[e] = l[e] == 0.f ? -INFINITY : ref[e];
            float4 *w = reinterpret_cast<float4 *>(slots + (team * (kWarps / 2) + member % (kWarps / 2)) * C::kSlot);
            auto put = [&] {
#pragma unroll
                for (int i = 0; i < MT; ++i) w[i * 32 + lane] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                if (g == 0) w[MT * 32 + t4] = make_float4(m[0], m[1], l[0], l[1]);
            };
            if (member >= kWarps / 2) put();
            bar_team(team);
            if (member < kWarps / 2) {
                const float4 ml = w[MT * 32 + t4];
                float own_f[2], other[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float mo = e ? ml.y : ml.x, top = fmaxf(m[e], mo), r = ref_of(top);
                    own_f[e] = ex2(m[e] - r);
                    other[e] = ex2(mo - r);
                    m[e] = top;
                    l[e] = l[e] * own_f[e] + (e ? ml.w : ml.z) * other[e];
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const float4 v = w[i * 32 + lane];
                    o[i][0] = o[i][0] * own_f[0] + v.x * other[0];
                    o[i][1] = o[i][1] * own_f[1] + v.y * other[1];
                    o[i][2] = o[i][2] * own_f[0] + v.z * other[0];
                    o[i][3] = o[i][3] * own_f[1] + v.w * other[1];
                }
                __syncwarp();                            // (m, l) have been read
                put();
            }
        }
        bar_team(team);
        // every warp: fragments member, member + 4, .. of both slots
        constexpr int F = MT / kWarps;
        float4 acc[F];
        float top[F][2], sum[F][2];
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int f = member + u * kWarps;
            const float4 *w0 = reinterpret_cast<const float4 *>(slots + team * (kWarps / 2) * C::kSlot);
            const float4 *w1 = reinterpret_cast<const float4 *>(slots + (team * (kWarps / 2) + 1) * C::kSlot);
            const float4 v0 = w0[MT * 32 + t4], v1 = w1[MT * 32 + t4];
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
        // the thread's elements of row 2 t4 + e
        auto row_at = [&](int e) -> uint16_t * {
            const int r = 2 * t4 + e;
            if (r >= rows) return nullptr;
            const int rr = r_first + r, t = a.p.group(rr);
            return a.out + static_cast<int64_t>(it.q0 + t) * a.out_stride + (it.head * group + rr - t * group) * D + 8 * OCT * g;
        };
        auto two = [](float x, float y, float inv) {
            if (inv == 0.f) x = y = 0.f;                     // a row that sees nothing, beside whatever the values hold
            return pack2<BF>(x * inv, y * inv);
        };
        // elements 2 i and 2 i + 1 of the thread's words, of both its rows
        auto store = [&](int i, const float4 &x, float l0, float l1) {
            if (uint16_t *dst = row_at(0)) *reinterpret_cast<uint32_t *>(dst + 2 * i) = two(x.x, x.z, inverse(l0));
            if (uint16_t *dst = row_at(1)) *reinterpret_cast<uint32_t *>(dst + 2 * i) = two(x.y, x.w, inverse(l1));
        };
        if (part.whole) {
#pragma unroll
            for (int u = 0; u < F; ++u) store(member + u * kWarps, acc[u], sum[u][0], sum[u][1]);
            continue;
        }
        // [MT][32] float4 fragments, then [4] (m, m, l, l) of a thread's two rows
        const int c0 = static_cast<uint32_t>(it.u) / sh.per, c1 = static_cast<uint32_t>(it.u + it.n) / sh.per;
        auto piece = [&](int cta) {
            return reinterpret_cast<float4 *>(a.ws + static_cast<size_t>(2 * cta + (cta == c0)) * C::kPiece);
        };
        float4 *own_piece = piece(blockIdx.x * T + team);
#pragma unroll
        for (int u = 0; u < F; ++u) {
            const int f = member + u * kWarps;
            __stcg(own_piece + f * 32 + lane, acc[u]);
            if (f == 0 && g == 0) __stcg(own_piece + MT * 32 + t4, make_float4(top[u][0], top[u][1], sum[u][0], sum[u][1]));
        }
        bar_team(team);
        if (member == 0 && lane == 0) {
            const int before = count_piece(a.tickets + c0);
            flags[team] = before == c1 - c0;
            if (before == c1 - c0) a.tickets[c0] = 0;
        }
        bar_team(team);
        if (!*reinterpret_cast<volatile int *>(flags + team)) continue;
        const int pieces = c1 - c0 + 1;
        if (pieces <= 8) {
            // all of them on their way at once
            float4 v[8], x[F][8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const float4 *w = piece(min(c0 + k, c1));
                v[k] = __ldcg(w + MT * 32 + t4);
#pragma unroll
                for (int u = 0; u < F; ++u) x[u][k] = __ldcg(w + (member + u * kWarps) * 32 + lane);
            }
            float t0 = -INFINITY, t1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {                // (a piece twice does no harm to a maximum)
                t0 = fmaxf(t0, v[k].x);
                t1 = fmaxf(t1, v[k].y);
            }
#pragma unroll
            for (int u = 0; u < F; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            const float r0 = ref_of(t0), r1 = ref_of(t1);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                if (k >= pieces) continue;
                const float f0 = ex2(v[k].x - r0), f1 = ex2(v[k].y - r1);
                l0 += v[k].z * f0;
                l1 += v[k].w * f1;
#pragma unroll
                for (int u = 0; u < F; ++u)
                    acc[u] = make_float4(acc[u].x + x[u][k].x * f0, acc[u].y + x[u][k].y * f1, acc[u].z + x[u][k].z * f0,
                                         acc[u].w + x[u][k].w * f1);
            }
#pragma unroll
            for (int u = 0; u < F; ++u) store(member + u * kWarps, acc[u], l0, l1);
            continue;
        }
        // The pieces' weights first, all at once, then their fragments, eight pieces at a time; in the order of the CTAs.
        float4 *factors = reinterpret_cast<float4 *>(slots + team * (kWarps / 2) * C::kSlot);     // [t4]: (m, m, l, l) of all
        float *lifts = reinterpret_cast<float *>(factors + 4);                                    // [32 pieces][t4][2]
        if (member == 0) {
            // lane: pieces g, g + 8, .., row pair t4
            float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
#pragma unroll 4
            for (int c = g; c < pieces; c += 8) {
                const float4 v = __ldcg(piece(c0 + c) + MT * 32 + t4);
                const float h0 = fmaxf(m0, v.x), h1 = fmaxf(m1, v.y);
                l0 = l0 * ex2(m0 - ref_of(h0)) + v.z * ex2(v.x - ref_of(h0));
                l1 = l1 * ex2(m1 - ref_of(h1)) + v.w * ex2(v.y - ref_of(h1));
                m0 = h0;
                m1 = h1;
            }
            const float t0 = max_g(m0), t1 = max_g(m1);
            l0 = sum_g(l0 * ex2(m0 - ref_of(t0)));
            l1 = sum_g(l1 * ex2(m1 - ref_of(t1)));
            if (g == 0) factors[t4] = make_float4(t0, t1, l0, l1);
        }
        bar_team(team);
#pragma unroll
        for (int u = 0; u < F; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int cc = 0; cc < pieces; cc += 32) {
            const int here = min(32, pieces - cc);
            if (const int i = threadIdx.x % (32 * kWarps); i < 4 * here) {
                const float4 v = __ldcg(piece(c0 + cc + (i >> 2)) + MT * 32 + (i & 3)), all = factors[i & 3];
                lifts[2 * i] = ex2(v.x - ref_of(all.x));
                lifts[2 * i + 1] = ex2(v.y - ref_of(all.y));
            }
            bar_team(team);
#pragma unroll
            for (int u = 0; u < F; ++u) {
                const int f = member + u * kWarps;
#pragma unroll 1
                for (int c = 0; c < here; c += 8) {
                    float4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = __ldcg(piece(c0 + cc + min(c + k, here - 1)) + f * 32 + lane);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (c + k >= here) continue;
                        const float2 w = *reinterpret_cast<const float2 *>(lifts + 2 * (4 * (c + k) + t4));
                        acc[u].x += x[k].x * w.x;
                        acc[u].y += x[k].y * w.y;
                        acc[u].z += x[k].z * w.x;
                        acc[u].w += x[k].w * w.y;
                    }
                }
            }
            bar_team(team);
        }
        const float4 all = factors[t4];
#pragma unroll
        for (int u = 0; u < F; ++u) store(member + u * kWarps, acc[u], all.z, all.w);
    }
    if (!alive && lane == 0) atomicOr(a.status, kAttnTimeout);
}

template <class C>
cudaError_t launch(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                   cudaStream_t st) {
    Args args{{b, s.hkv, s.page_log2, a.window, kKtLog2, FastDiv(s.group), kRowsLog2, FastDiv(1), a.sinks},
              c, a.q, a.out, a.q_stride, a.out_stride, a.scale * 1.4426950408889634f, a.ws, a.tickets, a.status};
    auto kernel = bf16 ? attend_stream4_kernel<true, C> : attend_stream4_kernel<false, C>;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), C::kSmem, a.allowed, kStream4 + (C::GL == 6))) return e;
    kernel<<<a.ctas, C::kThreads, C::kSmem, st>>>(args);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attend_stream4(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                                  cudaStream_t st) {
    if (s.d == 64) return c.group_log2 == 5 ? launch<Cfg<64, 5>>(s, b, c, a, bf16, st) : launch<Cfg<64, 6>>(s, b, c, a, bf16, st);
    return c.group_log2 == 5 ? launch<Cfg<128, 5>>(s, b, c, a, bf16, st) : launch<Cfg<128, 6>>(s, b, c, a, bf16, st);
}

}  // namespace q4
