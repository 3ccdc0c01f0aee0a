// Low-rank adapters for many rows, on tcgen05 (prompts; few rows are in
// q4_lora.cu, which has the adapters' private layout).
//
// The call is bound by reading x and y and writing out: 2 M K + 4 M N bytes
// against 2 M r (K + N) flop, some 60 flop a byte at r = 64, a quarter of what
// the tensor cores would allow.  Both launches take tiles of 128 consecutive
// rows, as they lie in memory, so x, y and out move by TMA, each byte once.
// The rows of a tile may use several adapters: their ranks stand side by side
// as the columns of t, and t is zero where a row does not use the adapter.
// Prompts come in runs, so a tile has one or two; a tile of many costs a
// product each, and still one pass over x and y.
//
//   first   t[m][r] = scale x[m] . A[r]: x tiles by TMA, adapter tiles by
//           bulk copy, fp32 sums in tensor memory; K in parts over a cluster,
//           which adds them and leaves t as two 16-bit parts (high, low)
//   second  both parts of t are the A operand in tensor memory; B tiles by
//           bulk copy; the sums of 128 x 128 outputs in two tensor memory
//           buffers; y tiles are loaded, added to, rounded in place and
//           stored by TMA
//
// A tile whose adapters have more than kCap ranks in all (single tokens of many
// requests) takes passes over its output, each of which changes only the rows
// that use its adapters; where a tile can hold more than 512 ranks, such tiles
// are left to the kernels of few rows, which run behind over the tiles that the
// first launch marks (the second has copied their y to out by then).  Adapters
// with an infinity or NaN, which must not meet another row's zero, get passes
// of their own.
//
// 4099 rows of 6 runs, 8192 x 28672, rank 64, fp16: 112 us, 4.5 TB/s of the
// bytes that the call cannot do without (74 us at the copy rate): the first
// launch 15 of them (x is 67 MB), the second 1.43 us for a job of 128 x 128
// outputs on each SM.  There y and out move at 5.1 TB/s, and L2 serves 9.4 TB/s
// in all, B for each row tile among it; what that path could do at most is not
// measured.  The tensor cores are 5 % busy.  Sizes: 128 x 128 jobs in two tensor
// memory buffers keep loads, products and stores of three jobs in flight; four y
// stages and two B stages are what shared memory holds.  Every wait is bounded;
// one that runs out sets a status bit, and its role goes on without waiting.
#include <cuda.h>

#include <algorithm>
#include <cstdint>

#include "q4_attn_tma.cuh"
#include "q4_internal.cuh"
#include "q4_lora.cuh"
#include "q4_tc.cuh"

namespace q4 {

cudaError_t encode_2d(CUtensorMap *map, CUtensorMapDataType dt, const void *ptr, uint64_t inner, uint64_t outer,
                      uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle sw);

namespace {

using namespace tc;

constexpr int kTile = 128;           // rows of a tile, and columns in the second launch
constexpr int kCap = 176;            // ranks of a pass of the second launch: what two B tiles have room for
constexpr int kShrinkCap = 176;      // of the first

// The adapters of a tile's rows.
struct TileInfo {
    int n, passes, marked;
    int slot[kTile], rank[kTile];    // of each class; rank padded to 16
    int pass[kTile], off[kTile];     // its pass, and its first rank there
    int cls[kTile];                  // of each row; -1: none
    int s_slot[kTile], s_id[kTile];  // while it is built
    int leads[4];
};
// By the whole CTA (at least 128 threads).
__device__ void build_info(const LoraView &v, const LoraCall &c, int m0, int cap, bool solo, TileInfo &k) {
    const int i = threadIdx.x;
    int slot = -1;
    LoraSlot info{0, 0.f, 1};
    if (i < kTile) {
        if (m0 + i < c.M) {
            slot = c.row_slot[m0 + i];
            if (slot >= v.slots) {
                atomicOr(v.status, kLoraBadSlot);
                slot = -1;
            }
            if (slot >= 0) info = v.slot[slot];
            if (info.rank == 0) slot = -1;
        }
        k.s_slot[i] = slot;
    }
    __syncthreads();
    int lead = i;
    if (i < kTile) {
        if (slot >= 0)
#pragma unroll 16
            for (int j = kTile - 1; j >= 0; --j) lead = k.s_slot[j] == slot ? j : lead;
        const unsigned b = __ballot_sync(0xffffffffu, slot >= 0 && lead == i);
        if ((i & 31) == 0) k.leads[i >> 5] = b;
    }
    __syncthreads();
    if (i < kTile) {
        int id = -1;
        if (slot >= 0) {
            id = __popc(k.leads[lead >> 5] & ((1u << (lead & 31)) - 1));
            for (int w = 0; w < lead >> 5; ++w) id += __popc(k.leads[w]);
            if (lead == i) {
                k.slot[id] = slot;
                k.rank[id] = ceil16(info.rank);
                k.s_id[id] = info.finite;
            }
        }
        k.cls[i] = id;
    }
    __syncthreads();
    if (i == 0) {
        const int n = __popc(k.leads[0]) + __popc(k.leads[1]) + __popc(k.leads[2]) + __popc(k.leads[3]);
        int pass = 0, off = 0, ranks = 0;
        bool alone = false;
        for (int j = 0; j < n; ++j) {
            const bool own = solo && !k.s_id[j];
            if (off && (off + k.rank[j] > cap || own || alone)) {
                ++pass;
                off = 0;
            }
            alone = own;
            k.pass[j] = pass;
            k.off[j] = off;
            off += k.rank[j];
            ranks += k.rank[j];
        }
        k.marked = c.marks && ranks > kCap;              // left to the kernels of few rows
        k.n = k.marked ? 0 : n;
        k.passes = k.n ? pass + 1 : 0;
    }
    __syncthreads();
}

// K-major operand in shared memory without swizzle, as core matrices of 8
// rows x 16 bytes: `along` bytes to the next along K, `across` to the next 8 rows.
__device__ __forceinline__ uint64_t smem_desc_core(uint32_t saddr, uint32_t along, uint32_t across) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>((along >> 4) & 0x3FFFu) << 16 |
           static_cast<uint64_t>((across >> 4) & 0x3FFFu) << 32 | static_cast<uint64_t>(1) << 46;
}
__device__ __forceinline__ void umma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, uint32_t src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(map), "r"(src),
                 "r"(c0), "r"(c1)
                 : "memory");
}

// ------------------------------------------------------------ first launch
constexpr int kShrinkThreads = 192;  // warps 0-3 read the sums, 4 loads, 5 issues the MMAs
constexpr int kXBytes = kTile * 128, kABytes = kShrinkCap * 128, kShrinkStage = kXBytes + kABytes;
constexpr int kShrinkMaxStages = 5;
constexpr uint32_t kShrinkCols = 256;
constexpr int kShrinkMisc = 256 + static_cast<int>(sizeof(TileInfo)) + 1024;
// The sums of the tile's rows, [128][rpad + 4] fp32, lie behind the ring.
__host__ __device__ constexpr int sums_bytes(int rpad) { return kTile * (rpad + 4) * 4; }
__host__ __device__ constexpr int shrink_stages(int rpad) {
    const int n = (232448 - kShrinkMisc - sums_bytes(rpad)) / kShrinkStage;
    return n < kShrinkMaxStages ? n : kShrinkMaxStages;
}

// Grid: parts of K x row tiles, the parts of a tile in one cluster: each sums
// its share of the tile's rows over the parts, in their order, and splits
// scale times the sum into its two 16-bit parts.
// t16 [rows][2][rpad]: high and low parts; up [rows]: what they have been divided by.
template <bool BF>
__global__ void __launch_bounds__(kShrinkThreads, 1)
    shrink_tc_kernel(const __grid_constant__ CUtensorMap tmX, LoraView v, LoraCall c, uint16_t *t16, float *up,
                     int blocks_each, int parts, int S) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sb = smem_raw + (base - raw);
    float *sums = reinterpret_cast<float *>(sb + S * kShrinkStage);
    const int pitch = v.rpad + 4;
    uint8_t *misc = sb + S * kShrinkStage + sums_bytes(v.rpad);
    const uint32_t bars = base + S * kShrinkStage + sums_bytes(v.rpad);
    auto full = [&](int s) { return bars + 8u * s; };
    auto empty = [&](int s) { return bars + 8u * (kShrinkMaxStages + s); };
    const uint32_t d_full = bars + 16 * kShrinkMaxStages, d_empty = d_full + 8;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 16 * kShrinkMaxStages + 16);
    TileInfo &k = *reinterpret_cast<TileInfo *>(misc + 256);
    const int warp = threadIdx.x >> 5;
    const int part = blockIdx.x % parts, tile = blockIdx.x / parts, m0 = tile * kTile;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmX) : "memory");
        for (int s = 0; s < S; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(d_full, 1);
        mbar_init(d_empty, 128);
        mbar_init_fence();
    }
    if (warp == 5) tmem_alloc(smem_u32(tmem_slot), kShrinkCols);
    tc_fence_before();
    build_info(v, c, m0, kShrinkCap, false, k);                      // synchronizes
    tc_fence_after();
    if (c.marks && part == 0 && threadIdx.x == 0) c.marks[tile] = k.marked;
    const uint32_t tmem = *tmem_slot;
    const int kb0 = part * blocks_each, kb1 = min(kb0 + blocks_each, (v.K + 63) / 64);
    bool alive = true;
    if (warp == 4) {
        int seq = 0;
        for (int p = 0, c0 = 0; p < k.passes && alive; ++p) {
            int c1 = c0, ranks = 0;
            for (; c1 < k.n && k.pass[c1] == p; ++c1) ranks += k.rank[c1];
            for (int kb = kb0; kb < kb1; ++kb, ++seq) {
                const int s = seq % S;
                if (seq >= S) alive = wait_all(alive, empty(s), ((seq / S) & 1) ^ 1);
                if (!alive) break;
                const uint32_t st = base + s * kShrinkStage;
                if (elect_one()) {
                    mbar_arrive_expect_tx(full(s), kXBytes + ranks * 128);
                    tma_load_2d(st, &tmX, full(s), 64 * kb, m0);
#pragma unroll 1
                    for (int i = c0; i < c1; ++i)
                        bulk_load(st + kXBytes + k.off[i] * 128,
                                  v.a + static_cast<size_t>(k.slot[i]) * v.rpad * ceil64(v.K) +
                                      static_cast<size_t>(kb) * 64 * k.rank[i],
                                  k.rank[i] * 128, full(s));
                }
                __syncwarp();
            }
            c0 = c1;
        }
        if (!alive)
            for (int i = max(seq - S, 0); i < seq; ++i) wait_bounded(full(i % S), (i / S) & 1);
    } else if (warp == 5) {
        if (elect_one()) {
            int seq = 0;
            auto wait = [&](uint32_t bar, int n) {
                if (alive) alive = wait_bounded(bar, n & 1);
                tc_fence_after();
            };
            for (int p = 0, c0 = 0; p < k.passes; ++p) {
                int ranks = 0;
                for (; c0 < k.n && k.pass[c0] == p; ++c0) ranks += k.rank[c0];
                const uint32_t idesc = idesc_f16(128, 0, false) | static_cast<uint32_t>(ranks >> 3) << 17 |
                                       (BF ? (1u << 7) | (1u << 10) : 0u);
                if (p) wait(d_empty, p - 1);
                for (int kb = kb0; kb < kb1; ++kb, ++seq) {
                    const int s = seq % S;
                    wait(full(s), seq / S);
                    const uint32_t st = base + s * kShrinkStage;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_f16(tmem, smem_desc_sw128(st + 32 * kk, 16, 1024),
                                 smem_desc_core(st + kXBytes + 256 * kk, 128, 1024), idesc, kb != kb0 || kk != 0);
                    umma_commit(empty(s));
                }
                umma_commit(d_full);
            }
            // (every product has been read by the warps below before they end)
        }
    } else {
        const int row = threadIdx.x, mine = k.cls[row];
        float *dst = sums + row * pitch;
        for (int p = 0, c0 = 0; p < k.passes; ++p) {
            alive = wait_all(alive, d_full, p & 1);
            tc_fence_after();
            for (; c0 < k.n && k.pass[c0] == p; ++c0) {
                if (!__any_sync(0xffffffffu, mine == c0)) continue;
                for (int r = 0; r < k.rank[c0]; r += 16) {
                    uint32_t x[16];
                    tmem_ld_x16(tmem + (static_cast<uint32_t>(32 * warp) << 16) + k.off[c0] + r, x);
                    if (mine == c0)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *(reinterpret_cast<uint4 *>(dst + r) + e) = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                }
            }
            tc_fence_before();
            mbar_arrive(d_empty);
        }
    }
    if (!alive) atomicOr(v.status, kLoraTimeout);
    __syncthreads();
    if (warp == 5) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, kShrinkCols);
    }
    auto cluster_sync = [] {
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    };
    cluster_sync();
    // rows part, part + parts, ..: a warp holds a row, a lane two of each 64 ranks
    const int lane = threadIdx.x & 31;
    for (int row = part + parts * warp; row < kTile; row += parts * (kShrinkThreads / 32)) {
        const int mine = k.cls[row];
        if (mine < 0 || k.marked) continue;
        const int rank = k.rank[mine];
        const LoraSlot info = v.slot[k.slot[mine]];
        float2 x[3];                                     // kShrinkCap ranks
        float top = 0.f;
#pragma unroll
        for (int g = 0; g < 3; ++g) {
            x[g] = make_float2(0.f, 0.f);
            const int r = 64 * g + 2 * lane;
            if (r < rank) {
                const uint32_t at = smem_u32(sums + row * pitch + r);
#pragma unroll 4
                for (int q = 0; q < parts; ++q) {
                    uint32_t from;
                    float2 y;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(from) : "r"(at), "r"(q));
                    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(y.x), "=f"(y.y) : "r"(from) : "memory");
                    x[g].x += y.x;
                    x[g].y += y.y;
                }
                // a rank of the padding would be NaN in a row of x with an infinity
                x[g].x = r < info.rank ? x[g].x * info.scale : 0.f;
                x[g].y = r + 1 < info.rank ? x[g].y * info.scale : 0.f;
            }
            top = fmaxf(top, fmaxf(fabsf(x[g].x), fabsf(x[g].y)));
        }
        float by = 1.f;
        if constexpr (!BF) {
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            by = split_scale_of(top);
        }
        const float down = 1.f / by;                     // a power of two: exact
        uint16_t *dst = t16 + static_cast<size_t>(m0 + row) * 2 * v.rpad;
#pragma unroll
        for (int g = 0; g < 3; ++g) {
            const int r = 64 * g + 2 * lane;
            if (r >= rank) continue;
            const float y0 = x[g].x * down, y1 = x[g].y * down;
            const uint16_t h0 = to16<BF>(y0), h1 = to16<BF>(y1);
            *reinterpret_cast<uint32_t *>(dst + r) = h0 | static_cast<uint32_t>(h1) << 16;
            *reinterpret_cast<uint32_t *>(dst + v.rpad + r) =
                split_low<BF>(y0, h0) | static_cast<uint32_t>(split_low<BF>(y1, h1)) << 16;
        }
        if (lane == 0) up[m0 + row] = by;
    }
    cluster_sync();                                      // nobody leaves while its sums are read
}

// ----------------------------------------------------------- second launch
constexpr int kExpandThreads = 352;  // warps 0-3 and 4-7 turn by turn, 8 loads y, 9 issues the MMAs, 10 loads B
// An even number of y stages: each is then one set's, which waits for every use of it.  A set that saw only
// every other use could take the phase before for its own.
constexpr int kYStages = 4, kYBytes = kTile * kTile * 2;
static_assert(kYStages % 2 == 0, "a y stage belongs to one set of warps");
constexpr int kBStages = 2, kBBytes = kTile * kCap * 2;
constexpr int kExpandSmem = kYStages * kYBytes + kBStages * kBBytes + 256 + 512 + static_cast<int>(sizeof(TileInfo)) + 1024;
constexpr uint32_t kLow = 128;       // column of the low part of t
constexpr uint32_t kD = 256;         // of the sums, two buffers of 128

// A unit is 128 columns of a row tile; each CTA takes an equal run of units, row tile after row tile.
template <bool BF>
__global__ void __launch_bounds__(kExpandThreads, 1)
    expand_tc_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmO, LoraView v,
                     LoraCall c, const uint16_t *t16, const float *up_of) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    uint8_t *sb = smem_raw + (base - raw);
    const uint32_t bring = base + kYStages * kYBytes, bars = bring + kBStages * kBBytes;
    uint8_t *misc = sb + kYStages * kYBytes + kBStages * kBBytes;
    auto y_full = [&](int s) { return bars + 8u * s; };
    auto y_empty = [&](int s) { return bars + 32u + 8u * s; };
    auto b_full = [&](int s) { return bars + 64u + 8u * s; };
    auto b_empty = [&](int s) { return bars + 80u + 8u * s; };
    auto d_full = [&](int s) { return bars + 96u + 8u * s; };
    auto d_empty = [&](int s) { return bars + 112u + 8u * s; };
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(misc + 128);
    float *s_up = reinterpret_cast<float *>(misc + 256);
    TileInfo &k = *reinterpret_cast<TileInfo *>(misc + 768);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmY) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tmO) : "memory");
        for (int s = 0; s < kYStages; ++s) {
            mbar_init(y_full(s), 1);
            mbar_init(y_empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(b_full(s), 1);
            mbar_init(b_empty(s), 1);
            mbar_init(d_full(s), 1);
            mbar_init(d_empty(s), 128);
        }
        mbar_init_fence();
    }
    if (warp == 9) tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const int cols = (v.N + kTile - 1) / kTile, tiles = (c.M + kTile - 1) / kTile;
    const int64_t units = static_cast<int64_t>(tiles) * cols;
    int64_t u = units * blockIdx.x / gridDim.x;
    const int64_t u_end = units * (blockIdx.x + 1) / gridDim.x;
    bool alive = true, waited = false;
    int job = 0;                     // (unit, pass) jobs so far, the same in every role
    while (u < u_end) {
        const int tile = static_cast<int>(u / cols), n0 = static_cast<int>(u % cols), m0 = tile * kTile;
        const int n1 = static_cast<int>(min(static_cast<int64_t>(cols), n0 + (u_end - u)));
        u += n1 - n0;
        build_info(v, c, m0, kCap, true, k);
        // With one pass (or none) the tile's whole run is one stretch; with more, each (unit, pass) is.
        const bool single = k.passes <= 1;
        for (int stretch = 0; stretch < (single ? 1 : (n1 - n0) * k.passes); ++stretch) {
            const int p = single ? 0 : stretch % k.passes;
            const int a0 = single ? n0 : n0 + stretch / k.passes, a1 = single ? n1 : a0 + 1;
            int c0 = 0, c1, ranks = 0;
            while (c0 < k.n && k.pass[c0] < p) ++c0;
            for (c1 = c0; c1 < k.n && k.pass[c1] == p; ++c1) ranks += k.rank[c1];
            // -------------------------------- t of the pass into tensor memory: a thread holds a row
            if (warp < 4 && !waited) {                               // y and B need not wait for the first launch
                asm volatile("griddepcontrol.wait;" ::: "memory");
                waited = true;
            }
            if (warp < 4 && ranks) {
                const int row = threadIdx.x, mine = k.cls[row];
                const bool in = mine >= c0 && mine < c1;
                const uint16_t *src = t16 + static_cast<size_t>(m0 + row) * 2 * v.rpad;
                s_up[row] = in ? __ldcg(up_of + m0 + row) : 1.f;
                for (int i = c0; i < c1; ++i)
#pragma unroll 1
                    for (int r0 = 0; r0 < k.rank[i]; r0 += 64) {
                        uint4 h[4][2], l[4][2];          // 64 ranks, all on their way together; zero in other rows
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                h[q][e] = l[q][e] = make_uint4(0, 0, 0, 0);
                                if (mine == i && r0 + 16 * q < k.rank[i]) {
                                    h[q][e] = __ldcg(reinterpret_cast<const uint4 *>(src + r0 + 16 * q) + e);
                                    l[q][e] = __ldcg(reinterpret_cast<const uint4 *>(src + v.rpad + r0 + 16 * q) + e);
                                }
                            }
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (r0 + 16 * q < k.rank[i]) {
                                const uint32_t col = (k.off[i] + r0) / 2 + 8 * q;
                                tmem_st8(tmem + lanes + col, reinterpret_cast<const uint32_t(&)[8]>(h[q]));
                                tmem_st8(tmem + lanes + kLow + col, reinterpret_cast<const uint32_t(&)[8]>(l[q]));
                            }
                    }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            }
            if (warp < 8 || warp == 9) {
                tc_fence_before();
                asm volatile("bar.sync 3, 288;" ::: "memory");
                tc_fence_after();
            }
            // -------------------------------- the stretch's jobs
            if (warp == 8) {
                const CUtensorMap *from = p ? &tmO : &tmY;           // a later pass goes on from the output
                for (int n = a0; n < a1; ++n) {
                    const int i = job + n - a0, s = i % kYStages;
                    if (i >= kYStages) alive = wait_all(alive, y_empty(s), ((i / kYStages) & 1) ^ 1);
                    if (!alive) break;
                    if (elect_one()) {
                        const int halves = v.N - n * kTile > 64 ? 2 : 1;
                        mbar_arrive_expect_tx(y_full(s), halves * (kYBytes / 2));
                        for (int h = 0; h < halves; ++h)
                            tma_load_2d(base + s * kYBytes + h * (kYBytes / 2), from, y_full(s), n * kTile + 64 * h, m0);
                    }
                    __syncwarp();
                }
                if (!alive)
                    for (int i = max(job + a1 - a0 - kYStages, 0); i < job + a1 - a0; ++i)
                        wait_bounded(y_full(i % kYStages), (i / kYStages) & 1);
            } else if (warp == 10) {
                for (int n = a0; n < a1; ++n) {
                    const int i = job + n - a0, t = i & 1;
                    if (i >= 2) alive = wait_all(alive, b_empty(t), ((i >> 1) & 1) ^ 1);
                    if (!alive) break;
                    if (elect_one()) {
                        const int groups = min(kTile, v.N - n * kTile) / 8;
                        mbar_arrive_expect_tx(b_full(t), groups * ranks * 16);   // no adapter: no bytes
#pragma unroll 1
                        for (int j = c0; j < c1; ++j)
                            bulk_load(bring + t * kBBytes + k.off[j] * (kTile * 2),
                                      v.b + static_cast<size_t>(k.slot[j]) * v.rpad * v.N +
                                          static_cast<size_t>(n) * kTile * k.rank[j],
                                      groups * k.rank[j] * 16, b_full(t));
                    }
                    __syncwarp();
                }
                if (!alive)
                    for (int i = max(job + a1 - a0 - 2, 0); i < job + a1 - a0; ++i) wait_bounded(b_full(i & 1), (i >> 1) & 1);
            } else if (warp == 9) {
                if (elect_one()) {
                    constexpr uint32_t idesc = idesc_f16(128, kTile, false) | (BF ? (1u << 7) | (1u << 10) : 0u);
                    auto wait = [&](uint32_t bar, int n) {
                        if (alive) alive = wait_bounded(bar, n & 1);
                        tc_fence_after();
                    };
                    for (int n = a0; n < a1; ++n) {
                        const int i = job + n - a0, t = i & 1;
                        if (i >= 2) wait(d_empty(t), (i >> 1) + 1);
                        wait(b_full(t), i >> 1);
                        bool more = false;
                        for (int j = c0; j < c1; ++j) {
                            const uint32_t b = bring + t * kBBytes + k.off[j] * (kTile * 2);
#pragma unroll 1
                            for (int r = 0; r < k.rank[j]; r += 16) {
                                const uint64_t bd = smem_desc_core(b + 16 * r, 128, k.rank[j] * 16);
                                umma_f16_ta(tmem + kD + 128 * t, tmem + (k.off[j] + r) / 2, bd, idesc, more);
                                umma_f16_ta(tmem + kD + 128 * t, tmem + kLow + (k.off[j] + r) / 2, bd, idesc, 1);
                                more = true;
                            }
                        }
                        umma_commit(b_empty(t));
                        umma_commit(d_full(t));
                    }
                }
                __syncwarp();
            } else {
                const int set = warp >> 2, row = threadIdx.x & 127, mine = k.cls[row];
                const bool in = mine >= c0 && mine < c1;
                const float up = ranks ? s_up[row] : 1.f;
                for (int n = a0; n < a1; ++n) {
                    const int i = job + n - a0, s = i % kYStages;
                    if ((i & 1) != set) continue;
                    alive = wait_all(alive, y_full(s), (i / kYStages) & 1);
                    alive = wait_all(alive, d_full(set), (i >> 1) & 1);
                    tc_fence_after();
                    if (__any_sync(0xffffffffu, in))
#pragma unroll 1
                        for (int q = 0; q < 4; ++q) {
                            uint32_t d[32];
                            tmem_ld_x32(tmem + lanes + kD + 128 * set + 32 * q, d);
                            uint8_t *yr = sb + s * kYBytes + (q >> 1) * (kYBytes / 2) + row * 128;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint4 *at = reinterpret_cast<uint4 *>(yr + (((4 * (q & 1) + e) ^ (row & 7)) << 4));
                                uint4 w = *at;
                                uint32_t *x = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                                for (int f = 0; f < 4; ++f) {
                                    const float2 y = unpack2<BF>(x[f]);
                                    x[f] = pack2<BF>(fmaf(__uint_as_float(d[8 * e + 2 * f]), up, y.x),
                                                     fmaf(__uint_as_float(d[8 * e + 2 * f + 1]), up, y.y));
                                }
                                if (in) *at = w;
                            }
                        }
                    tc_fence_before();
                    mbar_arrive(d_empty(set));
                    fence_proxy_async();
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + set) : "memory");
                    if ((warp & 3) == 0 && elect_one()) {
                        for (int h = 0; h < (v.N - n * kTile > 64 ? 2 : 1); ++h)
                            tma_store_2d(&tmO, base + s * kYBytes + h * (kYBytes / 2), n * kTile + 64 * h, m0);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                        // a later pass reads what this one wrote; else only the buffer has to be free
                        if (single) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                        else asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
                        mbar_arrive(y_empty(s));
                    }
                    __syncwarp();
                }
            }
            job += a1 - a0;
            if (!single) asm volatile("fence.proxy.async;" ::: "memory");
            tc_fence_before();
            __syncthreads();         // t, the tile's adapters and the counters are free
            tc_fence_after();
        }
    }
    if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!alive) atomicOr(v.status, kLoraTimeout);
    __syncthreads();
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

}  // namespace

LoraTcPlan plan_lora_tc(const LoraView &v, int M, int sms) {
    LoraTcPlan p;
    p.ok = v.rpad <= kCap && v.rpad <= kShrinkCap;
    // Passes over a tile's output where it can hold few adapters: five passes at most (adapters of 96 ranks, one to a
    // pass; four of 64 ranks), and one more for each adapter with an infinity or NaN in B.  Marked tiles are the
    // faster way where rows do mix the adapters, and slower where they come in runs, which only the GPU knows.  8
    // adapters of 64 ranks, 8192 x 10240: 800 rows in 6 runs 26 us, 29 with marked tiles; rows that mix them 72 and 55.
    // 32 adapters: 27 and 30, 260 and 100.
    p.marks = std::min(kTile, v.slots) * v.rpad > 512;
    p.tiles = (M + kTile - 1) / kTile;
    const int blocks = (v.K + 63) / 64;
    // parts of K: as many CTAs as fill the GPU once, at least four blocks of 64 each
    const int parts = std::max(1, std::min({sms / std::max(p.tiles, 1), blocks / 4, 8}));
    p.blocks_each = (blocks + parts - 1) / parts;
    p.parts = (blocks + p.blocks_each - 1) / p.blocks_each;
    return p;
}

cudaError_t launch_lora_tc(const LoraView &v, const LoraCall &c, const LoraTcPlan &p, int sms, bool bf16,
                           cudaStream_t st, int *launches) {
    CUtensorMap tx, ty, to;
    const auto dt = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;        // 16-bit values either way
    cudaError_t e = encode_2d(&tx, dt, c.x, v.K, c.M, c.xs * 2, 64, kTile, CU_TENSOR_MAP_SWIZZLE_128B);
    if (!e) e = encode_2d(&ty, dt, c.y, v.N, c.M, c.ys * 2, 64, kTile, CU_TENSOR_MAP_SWIZZLE_128B);
    if (!e) e = encode_2d(&to, dt, c.out, v.N, c.M, c.os * 2, 64, kTile, CU_TENSOR_MAP_SWIZZLE_128B);
    if (e) return e;
    auto shrink = bf16 ? shrink_tc_kernel<true> : shrink_tc_kernel<false>;
    auto expand = bf16 ? expand_tc_kernel<true> : expand_tc_kernel<false>;
    const int S = shrink_stages(v.rpad), smem = S * kShrinkStage + sums_bytes(v.rpad) + kShrinkMisc;
    if ((e = cudaFuncSetAttribute(shrink, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) return e;
    if ((e = cudaFuncSetAttribute(expand, cudaFuncAttributeMaxDynamicSharedMemorySize, kExpandSmem))) return e;
    // t16 takes the place of the fp32 sums of the few-row kernels, the rows' scales come behind
    uint16_t *t16 = reinterpret_cast<uint16_t *>(v.t);
    float *up = v.t + static_cast<size_t>(c.M) * v.rpad;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = p.parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(p.parts) * p.tiles);
    cfg.blockDim = dim3(kShrinkThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    LoraCall marked = c;
    marked.chunk = kTile;
    marked.marks = p.marks ? reinterpret_cast<int *>(up + c.M) : nullptr;
    if ((e = cudaLaunchKernelEx(&cfg, shrink, tx, v, marked, t16, up, p.blocks_each, p.parts, S))) return e;
    cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(sms, static_cast<int64_t>(p.tiles) * ((v.N + kTile - 1) / kTile))));
    cfg.blockDim = dim3(kExpandThreads);
    cfg.dynamicSmemBytes = kExpandSmem;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = pdl_enabled() ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, expand, ty, to, v, marked, static_cast<const uint16_t *>(t16), static_cast<const float *>(up));
    if (!e) *launches += 2;
    return e || !p.marks ? e : launch_lora_marked(v, marked, bf16, st, launches);
}

}  // namespace q4
