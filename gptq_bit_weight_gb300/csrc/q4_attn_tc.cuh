// Attention of chunks of new tokens over the paged cache on the 5th-generation
// tensor cores (tcgen05), scores and outputs in tensor memory.
//
//   scores s = q . k (fp32); reference m and sum l of each row,
//   p = 2^(c (s - m)), c = scale log2(e), rounded to 16 bits for its product
//   with v (l sums the unrounded ones); o = sum p v in fp32; o / l rounded
//   once.  m is the maximum of the row's first key tile, and is raised to a
//   later tile's only when that is more than 2^8 away: any m gives the same
//   result as long as p fits 16 bits at both ends, so most tiles rescale no
//   output.  In fp16 p is 2^weight_lift of that.
//   The tensor cores take 16-bit operands: p in two parts would be half as much
//   again of the whole work.  In one, the result's error against 64 bits is 1.4
//   times that of rounding the exact result (relative, 512 tokens over 8192:
//   bf16 2.3e-3 and 1.7e-3; 384 over 4096, fp16: 2.8e-4 and 2.1e-4).
//
// One CTA per SM works on two tiles of up to 128 rows at a time (row = token x
// query head of the group, so the heads that share a key/value head share its
// tiles) against key tiles of 128 tokens:
//   warps 0-3, 4-7  softmax of the two row tiles: one thread for each row
//                   reads its scores (tcgen05.ld), writes p back over them
//                   as the A operand of the second product (tcgen05.st),
//                   rescales and, at the end, stores the output
//   warps 8, 11     load queries and keys, and values, by TMA (one box for
//                   each page and 64 columns) into a ring of half-stages
//   warp 9          one thread issues tcgen05.mma: while one row tile's
//                   softmax runs, the tensor cores work on the other's
//   warp 10         zeroes value rows outside the visible keys in the tiles
//                   at the edges: such slots hold anything, and 0 x NaN is NaN
// Two row tiles, because one alone leaves the tensor cores idle during its
// softmax; 184 registers for the softmax threads (a row of 128 scores each) and
// 136 for the others add up to the launch's 384 x 168.  The compiler keeps to
// 168 for all roles: the softmax's loop over key tiles spills (456 bytes of
// stores and 520 of loads; without the loop there are none), whatever the split
// leaves it; with 208 and 88 the other roles spill as well (604 and 648; 32
// requests of 4 tokens 58 us instead of 54.5).
// 4096 tokens over 16384, 64 heads over 8 of 128: 1120 us, 1.7 PFLOP/s, what the
// tensor cores sustain under the power limit; 512 over 8192: 98 us (1.36
// PFLOP/s: start, last wave and the join of the pieces); 384 together with 47
// single tokens of others: 111 us (a key tile is 1.8 us with two row tiles, 1.3
// with one).  Heads of 64, 4096 over 16384, 32 over 8: 463 us, bound by the
// softmax warps' own chain as it is compiled, spills among it (with columns of
// their own for the weights, so that the next scores never wait for the second
// product: 503).
// With first tokens that stay visible (SINKS), an item's key tiles are those of
// the first tokens and those of the window; a score's mask has the two ranges.
// Over a cache of 4 bits (FOUR) the launch has four more warps, 512 x 128
// registers: 256 x 184 + 256 x 72.  One warp loads records of half a tile by bulk
// copies, six decode blocks of 32 tokens into the tiles that the MMAs read
// (zeros for hidden tokens, so nothing is left to clean).  With two decoders it
// was 568 us for 1024 tokens over 16384, with four to six 411 (1.30 PFLOP/s; the
// 16-bit cache 340): two tiles fit beside the records and the queries, not two
// and a half, and the decoders' stores share the SM with the softmax.
// Every wait is bounded; a wait that runs out sets a status bit and its role
// goes on without waiting.
#pragma once
#include <cuda.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <type_traits>

#include "q4_attn_tma.cuh"
#include "q4_cache4.cuh"

namespace q4 {

namespace {

using namespace tc;

constexpr int kSoftmaxWarps = 8;
constexpr int kKeys = kSoftmaxWarps, kIssuer = kSoftmaxWarps + 1, kCleaner = kSoftmaxWarps + 2, kValues = kSoftmaxWarps + 3;
// Of the kernel for the 4-bit cache: the first of its decoders, which are all warps but the softmax's, the loader and the
// issuer.
constexpr int kDecoder = kSoftmaxWarps + 2, kDecoders = 6;
constexpr int threads_of(int four) { return 32 * (kSoftmaxWarps + (four ? 8 : 4)); }
constexpr uint32_t kTmemCols = 512;
constexpr float kRescale = 8.f;                  // log2 of the growth that p may have

// GL: 0 for the 16-bit cache, else log2 of the groups of a cache of 4 bits.
template <int D_, int GL_ = 0>
struct Cfg {
    static constexpr int D = D_, GL = GL_;
    static constexpr int kHalf = kKt * D * 2;    // bytes of a half-stage: keys or values of a tile
    static constexpr int kQ = 128 * D * 2;       // of one row tile's queries
    static constexpr int kMisc = 2048;
    static constexpr int kRecord = GL ? record_bytes(D, GL) : 0;
    static constexpr int kRaw = 64 * kRecord;    // the records of half a tile
    static constexpr int kRawStages = 3;
    static constexpr int kRoom = (232448 - 1024 - 2 * kQ - kRawStages * kRaw - kMisc) / kHalf;
    // what fits, 5 at D = 128; at D = 64 no more than 8 (12: 62.5 us for the window of 1024 instead of 59.4)
    static constexpr int kStages = kRoom > 8 ? 8 : kRoom;
    static constexpr int kSmem = 2 * kQ + kStages * kHalf + kRawStages * kRaw + kMisc + 1024;
    static constexpr int kPiece = 2 * 128 * (D + 2);   // floats of a piece in the workspace
};

template <bool SINKS, bool FOUR>
struct Args {
    SchedParamsT<SINKS> p;
    std::conditional_t<FOUR, Cache4, AttnCache> c;
    uint16_t *out;
    int64_t out_stride;
    float scale;                 // times log2(e), positive
    int tokens;                  // of a row tile: 128 / group
    float *ws;                   // [2 * CTAs] pieces
    int *tickets;                // [CTAs], zero between calls
    int *status;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int c1, int c2) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(
            dst),
        "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}
// D += A . B with A in tensor memory: row = lane, two 16-bit values of K in a column.
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
#define Q4_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
// 32 columns of the warp's lanes, without waiting for them.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : Q4_R8(r, 0), Q4_R8(r, 8), Q4_R8(r, 16), Q4_R8(r, 24)
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : Q4_R8(r, 0), Q4_R8(r, 8)
        : "r"(taddr)
        : "memory");
}
#undef Q4_R8
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
#define Q4_R8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        Q4_R8(r, 0), Q4_R8(r, 8)
        : "memory");
}
#undef Q4_R8
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two fp32 lanes in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y));
    return v;
}
__device__ __forceinline__ uint64_t pair_bits(uint32_t x, uint32_t y) {
    uint64_t v;
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(x), "r"(y));
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
__device__ __forceinline__ void bar_softmax() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// What of an item falls to this CTA, the same for every role.
struct Part {
    int j0, j1;              // its key tiles, counted from it.first
    bool two;                // the second row tile has rows
    __device__ Part(const Item &it, const Share &sh, int tokens)
        : j0(max(sh.begin - it.u, 0)),
          j1(min(sh.end - it.u, it.n)),
          two(it.t1 >= it.t0 + tokens) {}
};

// The values of 32 tokens, one of each lane, from their records to rows of a tile [D / 64][128][64], swizzled; zeros
// where `seen` is not set.  One copy of the code for all warps that decode: unrolled for a warp's blocks it was 17 KB
// beside the softmax's code and ran at 7 cycles an instruction (1024 tokens over 16384: 968 us).
template <bool BF, class C>
__device__ __forceinline__ void decode_rows(const uint8_t *record, bool value, bool seen, uint8_t *tile, int row) {
    constexpr int D = C::D, GL = C::GL;
    const uint8_t *codes = record + (value ? D / 2 : 0), *params = record + D + (value ? 4 * (D >> GL) : 0);
#pragma unroll
    for (int q = 0; q < D / 32; ++q) {                   // 32 elements, in one group
        uint32_t w[4];
        if constexpr (C::kRecord % 16 == 0) {
            const uint4 x = *reinterpret_cast<const uint4 *>(codes + 16 * q);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(codes + 16 * q), y = *reinterpret_cast<const uint2 *>(codes + 16 * q + 8);
            w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y;
        }
        uint32_t p = *reinterpret_cast<const uint32_t *>(params + 4 * (32 * q >> GL));
        if (!seen) p = 0;
        const uint32_t s2 = both_low(p), m2 = both_high(p);
        uint8_t *dst = tile + (q >> 1) * (kKt * 128) + row * 128;
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = values_of<BF>(w[i], s2, m2);
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4 *>(dst + (((4 * (q & 1) + i) ^ (row & 7)) << 4)) = v[i];
    }
}

// FOUR: 0 for the 16-bit cache, else log2 of the groups of a cache of 4 bits.
template <bool BF, class C, bool SINKS, int FOUR>
__global__ void __launch_bounds__(threads_of(FOUR), 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, Args<SINKS, FOUR != 0> a) {
    constexpr int D = C::D, S = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sb = smem_raw + (base - raw);
    const uint32_t ring = base + 2 * C::kQ, raws = ring + S * C::kHalf, bars = raws + C::kRawStages * C::kRaw;
    uint8_t *misc = sb + 2 * C::kQ + S * C::kHalf + C::kRawStages * C::kRaw;
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (S + s); };
    auto tail = [&](int s) { return bars + 8u * (2 * S + s); };
    const uint32_t q_full = bars + 8u * (3 * S), q_empty = q_full + 8, done = q_full + 16;
    auto s_full = [&](int i) { return q_full + 24 + 8u * i; };
    auto p_ready = [&](int i) { return q_full + 40 + 8u * i; };
    auto pv_done = [&](int i) { return q_full + 56 + 8u * i; };
    auto raw_full = [&](int s) { return q_full + 72 + 8u * s; };
    auto raw_empty = [&](int s) { return q_full + 72 + 8u * (C::kRawStages + s); };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 512);
    int *last_flags = reinterpret_cast<int *>(misc + 1016);             // of the first and the last item
    SchedSmem &sched = *reinterpret_cast<SchedSmem *>(misc + 520);
    float2 *s_ml = reinterpret_cast<float2 *>(misc + 1024);             // [128]: (m, l) of the second buffer
    static_assert(8 * (3 * S + 9 + 2 * C::kRawStages) <= 512 && 520 + sizeof(SchedSmem) <= 1016, "misc region");

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmQ) : "memory");
        if constexpr (!FOUR)
            for (const CUtensorMap *map : {&tmK, &tmV}) asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), FOUR ? 4 : 1);
            mbar_init(empty(s), 1);
            mbar_init(tail(s), 1);
        }
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(done, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full(i), 1);
            mbar_init(p_ready(i), 4);
            mbar_init(pv_done(i), 1);
        }
        for (int i = 0; FOUR && i < C::kRawStages; ++i) {
            mbar_init(raw_full(i), 1);
            mbar_init(raw_empty(i), 4);
        }
        mbar_init_fence();
    }
    if (warp == kIssuer) tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tc_fence_before();
    Item it;
    const Share sh = sched_share<threads_of(FOUR)>(a.p, sched, blockIdx.x, gridDim.x, a.status, it);   // synchronizes
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool alive = true;
    const bool work = sh.begin < sh.end;
    // 168 registers a thread at launch: 256 x 184 + 128 x 136 = 384 x 168; or 128: 256 x 184 + 256 x 72 = 512 x 128
    if (warp < kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        // ---------------------------------------------- softmax: a thread holds a row
        const int me = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lanes + 128 * me, tO = tmem + lanes + 256 + 128 * me;
        const float c = a.scale;
        [[maybe_unused]] const int sinks = SINKS ? a.p.sinks : 0;
        const int tok = a.p.group(row), head_in = row - tok * a.p.group.d;
        int uses = 0;
        for (bool more = work; more && it.u < sh.end; more = next_item(a.p, it)) {
            const Part part(it, sh, a.tokens);
            // With one row tile only, the two buffers take its key tiles in turn and are merged at the end.
            const bool turns = !part.two, joins = turns && part.j1 - part.j0 > 1;
            const bool active = me == 0 || !turns;
            const int ta = it.t0 + (turns ? 0 : me * a.tokens), t = ta + tok;    // the row tile's first token, the row's
            const bool mine = tok < a.tokens && t <= it.t1, valid = active && mine;
            const int lim = mine ? it.kv - it.ql + t : -1;             // last key that the row sees
            const int lim_lo = a.p.window > 0 ? lim - a.p.window : -1; // keys up to this one are out of the window
            float m = -INFINITY, l = 0.f, f0 = 1.f, f1 = 0.f;
            if (it.hi > 0 && (active || joins)) {
                // keys that every row of this row tile sees
                const int own = it.kv - it.ql, tb = min(ta + a.tokens - 1, it.t1);
                const int first_j = part.j0 + (turns ? me : 0), step = turns ? 2 : 1;
                const int all_hi = own + ta, all_lo = a.p.window > 0 ? own + tb - a.p.window : -1;
                for (int j = first_j; j < part.j1; j += step, ++uses) {
                    const int key_t = key_tile(a.p, it, j) << kKtLog2;
                    alive = wait_all(alive, s_full(me), uses & 1);
                    tc_fence_after();
                    uint32_t s[128];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(tS + 32 * q, s + 32 * q);
                    tmem_wait_ld();
                    if (key_t + kKt - 1 > all_hi || (key_t <= all_lo && !(SINKS && key_t + kKt <= sinks))) {
                        // visible keys of 32 as bits: those up to lim, without those up to lim_lo
                        auto upto = [](int n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int k0 = key_t + 32 * q - 1;
                            uint32_t out = upto(lim_lo - k0);
                            if constexpr (SINKS) out &= ~upto(sinks - 1 - k0);
                            const uint32_t seen = upto(lim - k0) & ~out;
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(seen >> e & 1)) s[32 * q + e] = 0xff800000u;
                        }
                    }
                    float top[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) top[e] = fmaxf(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]));
#pragma unroll
                    for (int e = 8; e < 128; e += 2)
                        top[e >> 1 & 3] = max3(top[e >> 1 & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
                    const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
                    const bool first = j == first_j;
                    const bool grows = first ? mx > m : (mx - m) * c > kRescale;
                    if (__any_sync(0xffffffffu, grows)) {
                        const float to = grows ? mx : m;
                        // from a row without any key so far, nothing is kept
                        const float f = grows ? ex2((m - to) * c) : 1.f;
                        l *= f;
                        m = to;
                        if (!first) {
                            alive = wait_all(alive, pv_done(me), (uses - 1) & 1);
                            tc_fence_after();
#pragma unroll
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t o[16];
                                tmem_ld16(tO + 16 * q, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st16(tO + 16 * q, o);
                            }
                        }
                    }
                    // (upwards in fp16, so that no weight is past 2^(kRescale + weight_lift), however large the scores)
                    const float ref = m == -INFINITY ? 0.f : BF ? m * c : __fmaf_ru(m, c, -weight_lift<BF>);
                    const uint64_t c2 = pair(c, c), ref2 = pair(-ref, -ref);
                    uint64_t sum[2] = {0, 0};
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t p[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 x = unpair(fma2(pair_bits(s[32 * h + 2 * e], s[32 * h + 2 * e + 1]), c2, ref2));
                            const float2 y = make_float2(ex2(x.x), ex2(x.y));
                            sum[e & 1] = add2(sum[e & 1], pair(y.x, y.y));
                            p[e] = pack2<BF>(y.x, y.y);
                        }
                        tmem_st16(tS + 16 * h, p);
                    }
                    const float2 total = unpair(add2(sum[0], sum[1]));
                    l += total.x + total.y;
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(p_ready(me));
                }
                alive = wait_all(alive, pv_done(me), (uses - 1) & 1);
                tc_fence_after();
                if (joins) {
                    if (me == 1) s_ml[row] = make_float2(m, l);
                    tc_fence_before();
                    bar_softmax();
                    tc_fence_after();
                    if (me == 0) {
                        const float2 v = s_ml[row];
                        const float top = fmaxf(m, v.x), ref = top == -INFINITY ? 0.f : top;
                        f0 = ex2((m - ref) * c);
                        f1 = ex2((v.x - ref) * c);
                        m = top;
                        l = l * f0 + v.y * f1;
                    }
                }
            }
            const bool rows_here = __any_sync(0xffffffffu, valid);     // in this warp
            auto outputs = [&](int q, float *o) {                      // 32 columns, of both buffers where they join
                tmem_ld32(tO + 32 * q, reinterpret_cast<uint32_t *>(o));
                if (joins) {
                    float y[32];
                    tmem_ld32(tO + 128 + 32 * q, reinterpret_cast<uint32_t *>(y));
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] = o[e] * f0 + y[e] * f1;
                } else {
                    tmem_wait_ld();
                }
            };
            auto end_item = [&] {
                tc_fence_before();
                if (joins) bar_softmax();                // the second buffer has been read
                tc_fence_after();
            };
            // ------------------------------------------ output, or a piece for the workspace
            uint16_t *dst = a.out + static_cast<int64_t>(it.q0 + t) * a.out_stride +
                            (it.head * static_cast<int>(a.p.group.d) + head_in) * D;
            auto store = [&](const float *o, float inv, int q) {       // 32 columns
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    *reinterpret_cast<uint4 *>(dst + 32 * q + 8 * v) =
                        make_uint4(pack2<BF>(o[8 * v] * inv, o[8 * v + 1] * inv), pack2<BF>(o[8 * v + 2] * inv, o[8 * v + 3] * inv),
                                   pack2<BF>(o[8 * v + 4] * inv, o[8 * v + 5] * inv),
                                   pack2<BF>(o[8 * v + 6] * inv, o[8 * v + 7] * inv));
            };
            if (part.j0 == 0 && part.j1 == it.n) {
                if (active && rows_here) {
                    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        float o[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                        if (it.hi > 0) outputs(q, o);
                        if (l == 0.f)                    // a row that sees nothing
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = 0.f;
                        if (valid) store(o, inv, q);
                    }
                }
                end_item();
                continue;
            }
            const int me_cta = blockIdx.x;
            const int c0 = static_cast<uint32_t>(it.u) / sh.per, c1 = static_cast<uint32_t>(it.u + it.n - 1) / sh.per;
            // of each row tile [D / 4][128] float4, then [2][128] (m, l)
            auto piece = [&](int cta) { return a.ws + static_cast<size_t>(2 * cta + (cta == c0)) * C::kPiece; };
            auto columns = [&](int cta, int q) {
                return reinterpret_cast<float4 *>(piece(cta)) + (me * (D / 4) + 8 * q) * 128 + row;
            };
            auto ml = [&](int cta) { return reinterpret_cast<float2 *>(piece(cta) + 2 * 128 * D) + me * 128 + row; };
            int *last_flag = last_flags + (it.u >= sh.begin);
            // A piece that finds all others there already need not be written.  But more than three pieces of few
            // rows are better added up by all threads, over rows and columns, out of memory (8 rows in 16 pieces:
            // 16 us for a call instead of 35).
            const bool few = c1 - c0 <= 2 || (it.t1 - it.t0 + 1) * static_cast<int>(a.p.group.d) > 64;
            bool last = false;
            if (few) {
                if (threadIdx.x == 0) {
                    *last_flag = pieces_counted(a.tickets + c0) == c1 - c0;
                }
                bar_softmax();
                last = *reinterpret_cast<volatile int *>(last_flag);
            }
            if (!last) {
                if (active && rows_here) {
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        float o[32];
                        outputs(q, o);
                        if (valid)                       // the other rows are not anybody's
#pragma unroll
                            for (int v = 0; v < 8; ++v)
                                __stcg(columns(me_cta, q) + v * 128, make_float4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]));
                    }
                    if (valid) __stcg(ml(me_cta), make_float2(m, l));
                }
                bar_softmax();
                if (threadIdx.x == 0) {
                    *last_flag = count_piece(a.tickets + c0) == c1 - c0;
                }
                bar_softmax();
                last = *reinterpret_cast<volatile int *>(last_flag);
            }
            if (last && !few) {
                if (threadIdx.x == 0) a.tickets[c0] = 0;
                const int group = a.p.group.d, rows = (it.t1 - it.t0 + 1) * group, full_tile = a.tokens * group;
#pragma unroll 1
                for (int e = threadIdx.x; e < rows * (D / 8); e += 256) {
                    const int r = e % rows, c8 = e / rows, tile = r >= full_tile, rt = r - tile * full_tile;
                    const int64_t at = static_cast<int64_t>(tile) * 128 * (D / 4) + 2 * c8 * 128 + rt;
                    auto of = [&](int k) { return __ldcg(reinterpret_cast<const float2 *>(piece(k) + 2 * 128 * D) + tile * 128 + rt); };
                    float top = -INFINITY, sum = 0.f, acc[8] = {};
#pragma unroll 4
                    for (int k = c0; k <= c1; ++k) top = fmaxf(top, of(k).x);
                    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 4
                    for (int k = c0; k <= c1; ++k) {
                        const float4 *w = reinterpret_cast<const float4 *>(piece(k)) + at;
                        const float4 x = __ldcg(w), y = __ldcg(w + 128);
                        const float2 v = of(k);
                        const float f = ex2((v.x - ref) * c);
                        sum += v.y * f;
                        acc[0] += x.x * f, acc[1] += x.y * f, acc[2] += x.z * f, acc[3] += x.w * f;
                        acc[4] += y.x * f, acc[5] += y.y * f, acc[6] += y.z * f, acc[7] += y.w * f;
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    const int token = a.p.group(r);
                    *reinterpret_cast<uint4 *>(a.out + static_cast<int64_t>(it.q0 + it.t0 + token) * a.out_stride +
                                               (it.head * group + r - token * group) * D + 8 * c8) =
                        make_uint4(pack2<BF>(acc[0] * inv, acc[1] * inv), pack2<BF>(acc[2] * inv, acc[3] * inv),
                                   pack2<BF>(acc[4] * inv, acc[5] * inv), pack2<BF>(acc[6] * inv, acc[7] * inv));
                }
            } else if (last) {
                // the pieces in the order of their CTAs, this one's from tensor memory
                if (threadIdx.x == 0) a.tickets[c0] = 0;
                if (active && rows_here) {
                    float top = m, sum = 0.f;
#pragma unroll 4
                    for (int k = c0; k <= c1; ++k)
                        if (k != me_cta && valid) top = fmaxf(top, __ldcg(ml(k)).x);
                    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll 4
                    for (int k = c0; k <= c1; ++k) {
                        const float2 v = k == me_cta || !valid ? make_float2(m, l) : __ldcg(ml(k));
                        sum += v.y * ex2((v.x - ref) * c);
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        float acc[32];
#pragma unroll
                        for (int e = 0; e < 32; ++e) acc[e] = 0.f;
#pragma unroll 1
                        for (int k = c0; k <= c1; ++k) {
                            float x[32], f;
                            if (k == me_cta) {
                                outputs(q, x);
                                f = ex2((m - ref) * c);
                            } else {
                                const float2 v = valid ? __ldcg(ml(k)) : make_float2(-INFINITY, 0.f);
#pragma unroll
                                for (int e = 0; e < 8; ++e) {
                                    const float4 y = valid ? __ldcg(columns(k, q) + e * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
                                    x[4 * e] = y.x, x[4 * e + 1] = y.y, x[4 * e + 2] = y.z, x[4 * e + 3] = y.w;
                                }
                                f = valid ? ex2((v.x - ref) * c) : 0.f;
                                __syncwarp();
                            }
#pragma unroll
                            for (int e = 0; e < 32; ++e) acc[e] += x[e] * f;
                        }
                        // a row that sees nothing, beside whatever the values hold (no such row is in an item of few
                        // rows that is cut: the last of them sees fewer keys than there are rows)
                        if (sum == 0.f)
#pragma unroll
                            for (int e = 0; e < 32; ++e) acc[e] = 0.f;
                        if (valid) store(acc, inv, q);
                    }
                }
            }
            end_item();
        }
    } else {
        if constexpr (FOUR) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 136;");
        if (!work) {
        } else if (!FOUR && (warp == kKeys || warp == kValues)) {
            if constexpr (!FOUR) {
            const bool values = warp == kValues;
            const int q_bytes = a.tokens * a.p.group.d * D * 2;
            int seq = values, items = 0, bad = 0;            // slots alternate between keys and values
            for (bool more = true; more && it.u < sh.end && alive; more = next_item(a.p, it)) {
                if (it.hi <= 0) continue;
                const Part part(it, sh, a.tokens);
                if (!values) {
                    if (items) alive = wait_all(alive, q_empty, (items - 1) & 1);
                    if (!alive) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(q_full, part.two ? 2 * q_bytes : q_bytes);
                        for (int i = 0; i < (part.two ? 2 : 1); ++i)
                            for (int h = 0; h < D / 64; ++h)
                                tma_load_3d(base + i * C::kQ + h * (128 * 128), &tmQ, q_full, 64 * h, it.head * a.p.group.d,
                                            it.q0 + it.t0 + i * a.tokens);
                    }
                    __syncwarp();
                    ++items;
                }
                const PageWalk walk(a.p, it, a.c.pages);
                TilePages next = walk.tile(a.p, it, part.j0, bad);
                for (int j = part.j0; j < part.j1; ++j, seq += 2) {
                    const TilePages t = next;
                    if (j + 1 < part.j1) next = walk.tile(a.p, it, j + 1, bad);       // on its way while this one waits
                    const int s = seq % S, key_t = key_tile(a.p, it, j) << kKtLog2;
                    if (seq >= S) alive = wait_all(alive, empty(s), ((seq / S) & 1) ^ 1);
                    if (!alive) break;
                    const bool edge = values && !sees_all(a.p, it, key_t, kKt);
                    walk.copy<D>(t, ring + s * C::kHalf, values ? &tmV : &tmK, edge ? tail(s) : full(s), it.head);
                }
            }
            if (bad) atomicOr(a.status, bad);
            if (!alive) {
                // let the copies in flight land before the CTA can exit
                if (items) wait_bounded(q_full, (items - 1) & 1);
                for (int i = seq - 2; i >= 0 && i > seq - 2 - S; i -= 2) {
                    wait_bounded(full(i % S), (i / S) & 1);
                    if (values) wait_bounded(tail(i % S), 0);
                }
            }
            }
        } else if (FOUR && warp != kIssuer) {
            if constexpr (FOUR) {
                // Records of half a tile come by bulk copies, issued by one warp.  A half has four blocks, two of 32 keys and
                // two of 32 values, which go to the decoders in turn.  (A decoder has a block in two of three halves, so it
                // sees the same two of the three raw stages at every turn of theirs.)
                constexpr int RS = C::kRawStages, R = C::kRecord;
                const int box_log2 = min(a.p.page_log2, 6), boxes = 64 >> box_log2, bytes = R << box_log2;
                static_assert(RS == 3 && kDecoders == 6, "who sees which stage");
                const int q_bytes = a.tokens * a.p.group.d * D * 2;
                int block = warp - kDecoder;                         // the decoder's next one
                int items = 0, bad = 0, half = 0, tile = 0;          // half tiles and tiles so far
                for (bool more = true; more && it.u < sh.end && alive; more = next_item(a.p, it)) {
                    if (it.hi <= 0) continue;
                    const Part part(it, sh, a.tokens);
                    const int halves = 2 * (part.j1 - part.j0);
                    auto first_key = [&](int h) { return (key_tile(a.p, it, part.j0 + (h >> 1)) << kKtLog2) + 64 * (h & 1); };
                    if (warp != kKeys) {
                        for (; block < 4 * (half + halves); block += kDecoders) {
                            const int h = (block >> 2) - half, st = (block >> 2) % RS;
                            const bool value = block & 2;
                            const int row = 32 * (block & 1) + lane, slot = 2 * (tile + (h >> 1)) + value;
                            alive = wait_all(alive, raw_full(st), ((block >> 2) / RS) & 1);
                            if (slot >= S) alive = wait_all(alive, empty(slot % S), ((slot / S) & 1) ^ 1);
                            if (!alive) break;
                            const uint8_t *raw = sb + 2 * C::kQ + S * C::kHalf + st * C::kRaw;
                            decode_rows<BF, C>(raw + row * R, value, sees_some(a.p, it, first_key(h) + row, 1),
                                               sb + 2 * C::kQ + slot % S * C::kHalf, 64 * (h & 1) + row);
                            fence_proxy_async();
                            __syncwarp();
                            if (lane == 0) {
                                mbar_arrive(raw_empty(st));
                                mbar_arrive(full(slot % S));
                            }
                        }
                        half += halves;
                        tile += halves >> 1;
                        continue;
                    }
                    const int32_t *table = a.p.b.table + it.b * a.p.b.table_stride;
                    const uint8_t *head = a.c.kv + static_cast<int64_t>(it.head << a.p.page_log2) * R;
                    // lane i has the page of box i; INT_MIN: no row sees it
                    auto entry = [&](int h) {
                        const int key = first_key(h) + (lane << box_log2);
                        return h < halves && lane < boxes && sees_some(a.p, it, key, 1 << box_log2) ? __ldg(table + (key >> a.p.page_log2)) : INT_MIN;
                    };
                    int next = entry(0);
                    if (items) alive = wait_all(alive, q_empty, (items - 1) & 1);
                    if (!alive) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(q_full, part.two ? 2 * q_bytes : q_bytes);
                        for (int i = 0; i < (part.two ? 2 : 1); ++i)
                            for (int h = 0; h < D / 64; ++h)
                                tma_load_3d(base + i * C::kQ + h * (128 * 128), &tmQ, q_full, 64 * h, it.head * a.p.group.d,
                                            it.q0 + it.t0 + i * a.tokens);
                    }
                    __syncwarp();
                    ++items;
                    for (int h = 0; h < halves; ++h, ++half) {
                        int page = next;
                        next = entry(h + 1);
                        const int st = half % RS;
                        if (half >= RS) alive = wait_all(alive, raw_empty(st), ((half / RS) & 1) ^ 1);
                        if (!alive) break;
                        const unsigned wanted = __ballot_sync(0xffffffffu, page != INT_MIN);
                        if (page != INT_MIN && (page < 0 || page >= a.c.pages)) {
                            bad = kAttnBadPage;
                            page = 0;
                        }
                        __syncwarp();
                        const int slot = first_key(h) & ((1 << a.p.page_log2) - 1) & ~((1 << box_log2) - 1);
                        const uint32_t dst = raws + st * C::kRaw, bar = raw_full(st);
                        const uint8_t *src = head + slot * R;
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
                    }
                }
                if (bad) atomicOr(a.status, bad);
                if (!alive && warp == kKeys) {
                    // let the copies in flight land before the CTA can exit
                    if (items) wait_bounded(q_full, (items - 1) & 1);
                    for (int i = half - 1; i >= 0 && i >= half - RS; --i) wait_bounded(raw_full(i % RS), (i / RS) & 1);
                }
            }
        } else if (warp == kIssuer) {
            if (elect_one()) {
                constexpr uint32_t fmt = BF ? (1u << 7) | (1u << 10) : 0u;         // A and B bf16
                constexpr uint32_t id_qk = idesc_f16(128, kKt, false) | fmt, id_pv = idesc_f16(128, D, true) | fmt;
                int tiles = 0, items = 0, uses[2] = {0, 0};
                auto wait = [&](uint32_t bar, int n) {
                    if (alive) alive = wait_bounded(bar, n & 1);
                    tc_fence_after();
                };
                auto qk = [&](int i, int tile, int seq) {            // scores buffer i = row tile's queries . keys
                    const uint32_t kb = ring + (seq % S) * C::kHalf;
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
                        umma_f16(tmem + 128 * i, smem_desc_sw128(base + tile * C::kQ + off, 16, 1024),
                                 smem_desc_sw128(kb + off, 16, 1024), id_qk, kk != 0);
                    }
                    umma_commit(s_full(i));
                };
                auto pv = [&](int i, int seq, bool first) {
                    const uint32_t vb = ring + (seq % S) * C::kHalf;
                    wait(p_ready(i), uses[i]++);
#pragma unroll
                    for (int kk = 0; kk < kKt / 16; ++kk)
                        umma_f16_ta(tmem + 256 + 128 * i, tmem + 128 * i + 8 * kk,
                                    smem_desc_sw128(vb + kk * 2048, kKt * 128, 1024), id_pv, !first || kk != 0);
                    umma_commit(pv_done(i));
                };
                for (bool more = true; more && it.u < sh.end; more = next_item(a.p, it)) {
                    if (it.hi <= 0) continue;
                    const Part part(it, sh, a.tokens);
                    // two row tiles: both against each key tile; one: its key tiles take the buffers in turn
                    const bool turns = !part.two;
                    const int n = part.j1 - part.j0, ahead = turns ? 2 : 1, each = turns ? 1 : 2;
                    wait(q_full, items++);
                    for (int j = 0; j < min(ahead, n); ++j) {
                        const int sk = 2 * (tiles + j);
                        wait(full(sk % S), sk / S);
                        for (int i = 0; i < each; ++i) qk(turns ? j : i, i, sk);
                        umma_commit(empty(sk % S));
                    }
                    if (n <= ahead) umma_commit(q_empty);
                    for (int j = 0; j < n; ++j, ++tiles) {
                        const int sv = 2 * tiles + 1, sk = 2 * (tiles + ahead);
                        const bool next = j + ahead < n;
                        wait(full(sv % S), sv / S);
                        for (int i = 0; i < each; ++i) {
                            const int buf = turns ? j & 1 : i;
                            pv(buf, sv, j < ahead);
                            if (i == each - 1) umma_commit(empty(sv % S));       // not after waiting for keys
                            if (!next) continue;
                            if (i == 0) wait(full(sk % S), sk / S);
                            qk(buf, i, sk);
                        }
                        if (next) umma_commit(empty(sk % S));
                        if (j + ahead + 1 == n) umma_commit(q_empty);
                    }
                }
                umma_commit(done);
                if (!wait_bounded(done, 0)) alive = false;
            }
        } else if (!FOUR && warp == kCleaner) {
            [[maybe_unused]] const int sinks = SINKS ? a.p.sinks : 0;
            int seq = 1;
            uint32_t turn = 0;                               // parity of each slot's tail barrier
            for (bool more = true; more && it.u < sh.end; more = next_item(a.p, it)) {
                if (it.hi <= 0) continue;
                const Part part(it, sh, a.tokens);
                for (int j = part.j0; j < part.j1; ++j, seq += 2) {
                    const int key_t = key_tile(a.p, it, j) << kKtLog2, s = seq % S;
                    if (sees_all(a.p, it, key_t, kKt)) continue;
                    alive = wait_all(alive, tail(s), (turn >> s) & 1);
                    turn ^= 1u << s;
                    uint8_t *v = sb + 2 * C::kQ + s * C::kHalf;
                    auto zero = [&](int r0, int r1) {
                        for (int i = r0 * 8 + lane; i < r1 * 8; i += 32)
#pragma unroll
                            for (int h = 0; h < D / 64; ++h)
                                *reinterpret_cast<uint4 *>(v + h * (kKt * 128) + i * 16) = make_uint4(0, 0, 0, 0);
                    };
                    zero(SINKS ? min(max(sinks - key_t, 0), kKt) : 0, min(max(it.lo - key_t, 0), kKt));
                    zero(max(min(it.hi - key_t, kKt), 0), kKt);
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full(s));
                }
            }
        }
    }
    if (!alive) atomicOr(a.status, kAttnTimeout);
    __syncthreads();
    if (warp == kIssuer) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

template <class C, bool SINKS, int FOUR, class Cache>
cudaError_t launch(const AttnShape &s, const AttnBatch &b, const Cache &c, const AttendCall &a, bool bf16,
                   cudaStream_t st) {
    CUtensorMap tq, tk{}, tv{};
    const int tokens = 128 / s.group;
    const uint32_t box = std::min(s.page, kKt);
    cudaError_t e = encode_queries(&tq, a.q, s, a.q_stride, b.tokens, tokens);
    if constexpr (!FOUR) {
        if (!e) e = encode_pages(&tk, c.k, s, c, box);
        if (!e) e = encode_pages(&tv, c.v, s, c, box);
    }
    if (e) return e;
    Args<SINKS, FOUR != 0> args{
        {b, s.hkv, s.page_log2, a.window, kKtLog2, FastDiv(s.group), -1, FastDiv(2 * tokens), a.sinks},
        c, a.out, a.out_stride, a.scale * 1.4426950408889634f, tokens, a.ws, a.tickets, a.status};
    auto kernel = bf16 ? attend_tc_kernel<true, C, SINKS, FOUR> : attend_tc_kernel<false, C, SINKS, FOUR>;
    if ((e = allow_smem(reinterpret_cast<const void *>(kernel), C::kSmem, a.allowed, FOUR ? kChunk4 + (FOUR == 6) : SINKS ? kChunkSinks : kChunk))) return e;
    kernel<<<a.ctas, threads_of(FOUR), C::kSmem, st>>>(tq, tk, tv, args);
    return cudaGetLastError();
}

}  // namespace

}  // namespace q4
