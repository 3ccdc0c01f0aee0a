// Low-rank adapters of many requests beside a shared projection:
//     out[m] = y[m] + scale_a (x[m] . A_a^T) . B_a^T,   a = row_slot[m].
// Two launches: the sums t[m][r] = scale_a x[m] . A_a[r] in fp32, then the
// product with B and the sum with y, rounded once.  The second is let in while
// the first runs (programmatic dependent launch) and waits for t only.
//
// Here: the adapters' private layout, and the kernels for few rows (single
// tokens, decode steps; and the tiles of a larger call that mix too many
// adapters).  A call looks at chunks of 64 to 256 rows and sorts them by
// adapter.  First launch: a unit is 16 ranks of an adapter for up to 64 of its
// rows in the chunk, K split over a CTA's warps and, where units are few, a
// cluster; second: 32 columns for 16 rows.  Weights go straight into mma.sync fragments
// with 16-byte loads, A once, B once for every 16 rows.
//
// Bound by latency: 64 rows over 32 adapters of up to 64 ranks, 8192 x 10240,
// take 19.4 us where the bytes would take 6.2.  The first launch is done after
// 7.4 (2 to find the rows' adapters, 3 for its loads, 2 to join its sums); the
// second's CTAs find registers as the first's end, and have 4 to 5 units a
// warp at about 1 us, a load from L2 and its products, one unit after the other.
// At two CTAs for each SM, 128 registers, both spill (the first 52 to 60 bytes
// of stores, its form for 16 rows none; the second 60 to 72).  Tried and slower: B
// copied ahead through shared memory (24 us: the copies' instructions cost more
// than the loads), one CTA for each SM in the first launch (20.6), B prefetched
// by the first launch (20.8).  A single row of a small adapter is one launch
// (lora_one_kernel).
//
// Layout: 8 x 8 blocks of 16-bit values, 8 rows of 16 bytes (the
// tensor-core "core matrix").
//   A (r, k): [k / 64][r / 8][k % 64 / 8][r % 8][k % 8], ranks padded with
//             zeros to a multiple of 16, k to a multiple of 64
//   B (n, r): [n / 8][r / 8][n % 8][r % 8], ranks padded the same way
// A warp's fragment load (8 rows x 4 blocks along the sum) is 512 contiguous
// bytes of A, and any run of columns of B or 64 columns of A is contiguous
// for a bulk copy.  The sum's index may be permuted as long as both operands
// agree: lane (g, q) takes the 8 consecutive values of block q in row g,
// which are the k slots {2q, 2q+1, 2q+8, 2q+9} of two k16 steps.
#include <algorithm>
#include <cstdint>

#include "q4_lora.cuh"

namespace q4 {

bool pdl_enabled();

namespace {

__global__ void lora_slot_kernel(LoraSlot *slot, int rank, float scale) { *slot = LoraSlot{rank, scale, 1}; }

// Copies one adapter into its slot.
__global__ void lora_set_kernel(uint16_t *a, uint16_t *b, LoraSlot *slot, const uint16_t *src_a,
                                const uint16_t *src_b, int K, int N, int rank, int r16, uint16_t exponent) {
    const size_t na = static_cast<size_t>(r16) * ceil64(K), nb = static_cast<size_t>(r16) * N;
    const size_t step = static_cast<size_t>(gridDim.x) * blockDim.x;
    const size_t i0 = static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    const int rg = r16 / 8;
    for (size_t i = i0; i < na; i += step) {             // [k / 64][r / 8][k % 64 / 8][r % 8][k % 8]
        const int e = i & 7, r8 = i >> 3 & 7, kg = i >> 6 & 7;
        const size_t u = i >> 9;
        const int r = static_cast<int>(u % rg) * 8 + r8;
        const size_t k = u / rg * 64 + kg * 8 + e;
        a[i] = r < rank && k < static_cast<size_t>(K) ? src_a[static_cast<size_t>(r) * K + k] : 0;
    }
    for (size_t i = i0; i < nb; i += step) {             // [n / 8][r / 8][n % 8][r % 8]
        const int e = i & 7, n8 = i >> 3 & 7;
        const size_t u = i >> 6;
        const int r = static_cast<int>(u % rg) * 8 + e;
        b[i] = r < rank ? src_b[(u / rg * 8 + n8) * rank + r] : 0;
        if ((b[i] & exponent) == exponent) slot->finite = 0;         // an infinity or NaN
    }
}

constexpr int kWarps = 8;
constexpr int kCluster = 8;          // CTAs that split K, at most
constexpr int kRows = 64;            // rows of a class that one unit of the first launch takes

// The rows of a chunk of up to R, by adapter.  An adapter in use is a class,
// in the order of its first row; the rows without one are a class as well.
template <int R>
struct Classes {
    int slot[R], rank[R];            // of each class; rank padded to 16, 0: no adapter
    int first[R + 1];                // its first place in `row`
    int units[R + 1];                // units of work of earlier classes
    int row[R];                      // chunk-relative rows, class after class
    int n;
};
// While they are found: the first rows' bits, and more.
template <int R>
struct Scratch {
    static constexpr int kMaxSlots = 4096;
    uint32_t lead[R / 32];
    __align__(4) uint8_t in[R / 32][R];      // of each warp's 32 rows those of a class
    uint16_t before[R / 32][R];              // rows of a class in earlier warps
    int2 sum[R / 32];
    int first[kMaxSlots + 1];                // first row of a slot (of none: at 0)
};
template <>
struct Scratch<64> {
    uint32_t lead[2];
    __align__(16) int slot[64];
    int count[64], units[64];
};
// Called by the whole CTA.  work(rows, rank): the units of a class.  A chunk
// of 64 compares all its rows with one another.
template <class Work>
__device__ __forceinline__ void find_classes(const LoraView &v, const LoraCall &c, int m0, Classes<64> &k,
                                             Scratch<64> &z, Work work) {
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    int slot = -2, rank = 0;                             // -2: no row, -1: no adapter
    if (i < 64) {
        if (i < c.chunk && m0 + i < c.M) {
            slot = c.row_slot[m0 + i];
            if (slot >= v.slots) {
                atomicOr(v.status, kLoraBadSlot);
                slot = -1;
            }
            slot = max(slot, -1);
        }
        z.slot[i] = slot;
        z.count[i] = z.units[i] = 0;
        if (slot >= 0) rank = ceil16(v.slot[slot].rank);
    }
    __syncthreads();
    uint32_t same[2] = {0, 0};                           // the rows of the same slot
    int lead = 0;
    if (i < 64) {
#pragma unroll
        for (int j = 0; j < 64 / 4; ++j) {
            const int4 o = reinterpret_cast<const int4 *>(z.slot)[j];
            same[j / 8] |= (o.x == slot ? 1u : 0u) << (4 * j & 31) | (o.y == slot ? 2u : 0u) << (4 * j & 31) |
                           (o.z == slot ? 4u : 0u) << (4 * j & 31) | (o.w == slot ? 8u : 0u) << (4 * j & 31);
        }
        lead = same[0] ? __ffs(same[0]) - 1 : 31 + __ffs(same[1]);
        const unsigned leads = __ballot_sync(0xffffffffu, slot != -2 && lead == i);
        if (lane == 0) z.lead[warp] = leads;
    }
    __syncthreads();
    auto below = [](uint32_t m, int n) { return __popc(n >= 32 ? m : m & ((1u << n) - 1)); };
    auto earlier = [&](const auto *m, int n) { return below(m[0], n) + (n > 32 ? below(m[1], n - 32) : 0); };
    int id = 0;
    if (i < 64 && slot != -2) {
        id = earlier(z.lead, lead);
        if (lead == i) {
            const int count = __popc(same[0]) + __popc(same[1]);
            k.slot[id] = slot;
            k.rank[id] = rank;
            z.count[id] = count;
            z.units[id] = work(count, rank);
        }
    }
    __syncthreads();
    if (i < 64) {                                     // prefix sums, by either warp for itself
        int rows[2] = {z.count[lane], z.count[lane + 32]}, units[2] = {z.units[lane], z.units[lane + 32]};
#pragma unroll
        for (int o = 1; o < 32; o <<= 1)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int x = __shfl_up_sync(0xffffffffu, rows[h], o), y = __shfl_up_sync(0xffffffffu, units[h], o);
                if (lane >= o) {
                    rows[h] += x;
                    units[h] += y;
                }
            }
        rows[1] += __shfl_sync(0xffffffffu, rows[0], 31);
        units[1] += __shfl_sync(0xffffffffu, units[0], 31);
        if (warp == 0)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                k.first[lane + 32 * h + 1] = rows[h];
                k.units[lane + 32 * h + 1] = units[h];
            }
        if (i == 0) {
            k.first[0] = k.units[0] = 0;
            k.n = __popc(z.lead[0]) + __popc(z.lead[1]);
        }
        // the row's place: the rows of the classes before its own, and its own class's before it
        const int upto[2] = {__shfl_sync(0xffffffffu, rows[0], id & 31), __shfl_sync(0xffffffffu, rows[1], id & 31)};
        if (slot != -2) k.row[upto[id >> 5] - z.count[id] + earlier(same, i)] = i;
    }
    __syncthreads();
}
// The same for larger chunks, by way of a table of the slots.
template <int R, class Work>
__device__ __forceinline__ void find_classes(const LoraView &v, const LoraCall &c, int m0, Classes<R> &k,
                                             Scratch<R> &z, Work work) {
    constexpr int W = R / 32;
    static_assert(R <= 32 * kWarps, "a thread for each row");
    const int i = threadIdx.x, lane = i & 31, warp = i >> 5;
    int slot = -2, rank = 0;                             // -2: no row, -1: no adapter
    if (i < c.chunk && m0 + i < c.M) {
        slot = c.row_slot[m0 + i];
        if (slot >= v.slots) {
            atomicOr(v.status, kLoraBadSlot);
            slot = -1;
        }
        slot = max(slot, -1);
        if (slot >= 0) rank = ceil16(v.slot[slot].rank);
    }
    for (int j = i; j <= v.slots; j += blockDim.x) z.first[j] = R;
    for (int j = i; j < W * R / 4; j += blockDim.x) reinterpret_cast<uint32_t *>(&z.in[0][0])[j] = 0;
    __syncthreads();
    uint32_t same = 0;                                   // the warp's rows of the same slot
    bool head = false;
    if (i < R) {
        same = __match_any_sync(0xffffffffu, slot);
        head = slot != -2 && lane == __ffs(same) - 1;
        if (head) atomicMin(z.first + slot + 1, i);        // the first row of a slot: any order gives the same
    }
    __syncthreads();
    const int lead = slot != -2 ? z.first[slot + 1] : -1;
    if (i < R) {
        const unsigned leads = __ballot_sync(0xffffffffu, lead == i);
        if (lane == 0) z.lead[warp] = leads;
    }
    __syncthreads();
    auto earlier = [](const uint32_t (&m)[W], int n) {   // bits below bit n
        int sum = 0;
#pragma unroll
        for (int w = 0; w < W; ++w)
            sum += __popc(n >= 32 * (w + 1) ? m[w] : n > 32 * w ? m[w] & ((1u << (n - 32 * w)) - 1) : 0);
        return sum;
    };
    const int n = earlier(z.lead, R), id = slot != -2 ? earlier(z.lead, lead) : 0;
    if (head) z.in[warp][id] = static_cast<uint8_t>(__popc(same));
    if (lead == i) {
        k.slot[id] = slot;
        k.rank[id] = rank;
    }
    __syncthreads();
    int rows = 0, units = 0;                             // prefix sums over the classes
    if (i < R) {
#pragma unroll
        for (int w = 0; w < W; ++w) {
            z.before[w][i] = static_cast<uint16_t>(rows);
            rows += z.in[w][i];
        }
        units = i < n ? work(rows, k.rank[i]) : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, rows, o), y = __shfl_up_sync(0xffffffffu, units, o);
            if (lane >= o) {
                rows += x;
                units += y;
            }
        }
        if (lane == 31) z.sum[warp] = make_int2(rows, units);
    }
    __syncthreads();
    if (i < R) {
#pragma unroll
        for (int w = 0; w < W - 1; ++w) {
            const int2 o = z.sum[w];
            rows += w < warp ? o.x : 0;
            units += w < warp ? o.y : 0;
        }
        k.first[i + 1] = rows;
        k.units[i + 1] = units;
        if (i == 0) {
            k.first[0] = k.units[0] = 0;
            k.n = n;
        }
    }
    __syncthreads();
    // the row's place: behind the rows of the classes before its own, and its own class's before it
    if (i < R && slot != -2)
        k.row[k.first[id] + z.before[warp][id] + __popc(same & ((1u << lane) - 1))] = i;
    __syncthreads();
}
// The class of a unit, by a whole warp.
template <int R>
__device__ __forceinline__ int class_of(const Classes<R> &k, int unit) {
    int id = 0;
#pragma unroll
    for (int w = 0; w < R / 32; ++w) id += __popc(__ballot_sync(0xffffffffu, k.units[32 * w + (threadIdx.x & 31) + 1] <= unit));
    return id;
}

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
__device__ __forceinline__ uint4 ldg_stream(const uint16_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// t of 16 ranks for 8 NT rows, this warp's part of K: ranks are the MMA's
// rows, the call's rows its columns.  Row tile j's 16 x 8 sums go to
// red[j pitch ..]: element e of the MMA's result, lane (g, q), value v, is
// rank g + 8 (v / 2), row 2 q + v % 2.
template <bool BF, int NT>
__device__ __forceinline__ void shrink_rows(const LoraView &v, const LoraCall &c, const uint16_t *a, int rg,
                                            const int *s_rows, int n, int first, int step, float4 *red, int pitch) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const uint16_t *x[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) x[i] = 8 * i + g < n ? c.x + s_rows[8 * i + g] * c.xs + 8 * q : nullptr;
    float acc[NT][4] = {};
    const int steps = (v.K + 31) / 32, blocks = v.K / 8;             // of 32 values of k; of 8
    constexpr int U = NT <= 2 ? 4 : 2;
    for (int i0 = first; i0 < steps; i0 += U * step) {
        uint4 w[U][2], p[U][NT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * step;
            w[u][0] = w[u][1] = make_uint4(0, 0, 0, 0);
            if (i < steps) {
                const uint16_t *at = a + (static_cast<size_t>(i >> 1) * rg * 8 + (i & 1) * 4 + q) * 64 + g * 8;
                w[u][0] = ldg_stream(at);
                w[u][1] = ldg_stream(at + 512);
            }
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                p[u][j] = make_uint4(0, 0, 0, 0);
                if (i < steps && 4 * i + q < blocks && x[j]) p[u][j] = *reinterpret_cast<const uint4 *>(x[j] + 32 * i);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                mma16816<BF>(acc[j], w[u][0].x, w[u][1].x, w[u][0].y, w[u][1].y, p[u][j].x, p[u][j].y);
                mma16816<BF>(acc[j], w[u][0].z, w[u][1].z, w[u][0].w, w[u][1].w, p[u][j].z, p[u][j].w);
            }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) red[j * pitch + lane] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// *p of the cluster's CTA `rank`.
__device__ __forceinline__ float load_of(const float *p, int rank) {
    uint32_t from;
    float x;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(from)
        : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(from) : "memory");
    return x;
}

// The chunks that a CTA (or a cluster, `me` of `all`) looks at, and its place
// among those that share one: the chunk of its blockIdx.y, or every so many of
// the marked ones.
template <int R>
struct Chunks {
    int step, at, marked;    // in the order of the marked ones; of them all
    int me, all;             // of those that share a chunk
    __device__ __forceinline__ Chunks(const LoraCall &c, int me_, int all_) : step(1), at(0), marked(1), me(me_), all(all_) {
        if constexpr (R > 64)
            if (c.marks) {
                marked = 0;
                for (int base = 0; base < count(c); base += 32) marked += __popc(marks(c, base));
                step = max(min(marked, all_), 1);
                at = me_ % step;
                me = me_ / step;
                all = (all_ - at + step - 1) / step;
            }
    }
    __device__ __forceinline__ bool more() const { return at < marked; }
    __device__ __forceinline__ void next() { at += step; }
    __device__ __forceinline__ int chunk(const LoraCall &c) const {
        if constexpr (R > 64)
            if (c.marks) {
                int left = at, base = 0;
                unsigned b = marks(c, 0);
                for (int n; (n = __popc(b)) <= left; left -= n) b = marks(c, base += 32);
                return base + static_cast<int>(__fns(b, 0, left + 1));
            }
        return blockIdx.y;
    }
    static __device__ __forceinline__ int count(const LoraCall &c) { return (c.M - 1) / c.chunk + 1; }
    static __device__ __forceinline__ unsigned marks(const LoraCall &c, int base) {
        const int i = base + (threadIdx.x & 31);
        return __ballot_sync(0xffffffffu, i < count(c) && c.marks[i]);
    }
};

// Grid: (clusters over the chunk's (class, 64 of its rows, block of 16 ranks)
// units x CTAs of a cluster along K, chunks of R rows).  Few: at most 16 rows
// in all, for fewer registers.
template <bool BF, bool Few, int R>
__global__ void __launch_bounds__(32 * kWarps, 2) lora_shrink_kernel(LoraView v, LoraCall call, int ck) {
    __shared__ Classes<R> k;
    __shared__ __align__(16) float red[kRows / 8 * kWarps * 128];
    __shared__ __align__(16) float sum[kRows / 8 * 128];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int part = blockIdx.x % ck, warp = threadIdx.x >> 5;
    for (Chunks<R> chunks(call, blockIdx.x / ck, gridDim.x / ck); chunks.more(); chunks.next()) {
        LoraCall c = call;
        const int m0 = chunks.chunk(c) * c.chunk;
        static_assert(sizeof(Scratch<R>) <= sizeof(red), "in the same place");
        find_classes(v, c, m0, k, *reinterpret_cast<Scratch<R> *>(red),
                     [](int rows, int rank) { return (rows + kRows - 1) / kRows * (rank / 16); });
        c.x += m0 * c.xs;
        float *t = v.t + static_cast<size_t>(m0) * v.rpad;
        // every CTA of a cluster takes the same way through this loop
        for (int unit = chunks.me; unit < k.units[k.n]; unit += chunks.all) {
            const int id = class_of(k, unit), slot = k.slot[id], rank = k.rank[id];
            const int group = (unit - k.units[id]) / (rank / 16), r0 = 16 * (unit - k.units[id]) - group * rank;
            const int n = min(k.first[id + 1] - k.first[id] - group * kRows, kRows), nt = (n + 7) / 8;
            const int *s_rows = k.row + k.first[id] + group * kRows;
            const uint16_t *a = v.a + static_cast<size_t>(slot) * v.rpad * ceil64(v.K) + static_cast<size_t>(r0) * 64;
            const int first = part * kWarps + warp, step = ck * kWarps, rg = rank / 8;
            float4 *mine = reinterpret_cast<float4 *>(red) + 32 * warp;
            if (nt == 1) shrink_rows<BF, 1>(v, c, a, rg, s_rows, n, first, step, mine, 32 * kWarps);
            else if (Few || nt == 2) shrink_rows<BF, 2>(v, c, a, rg, s_rows, n, first, step, mine, 32 * kWarps);
            else if (nt <= 4) shrink_rows<BF, 4>(v, c, a, rg, s_rows, n, first, step, mine, 32 * kWarps);
            else shrink_rows<BF, 8>(v, c, a, rg, s_rows, n, first, step, mine, 32 * kWarps);
            __syncthreads();
            // the warps' parts of K in order, then the cluster's
            for (int e = threadIdx.x; e < nt * 128; e += blockDim.x) {
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) s += red[(e >> 7) * kWarps * 128 + w * 128 + (e & 127)];
                sum[e] = s;
            }
            if (ck > 1) cluster_sync();
            else __syncthreads();
            if (part == 0) {
                const LoraSlot info = v.slot[slot];
                for (int e = threadIdx.x; e < nt * 128; e += blockDim.x) {
                    float x[kCluster], s = 0.f;              // on their way together, added in order
#pragma unroll
                    for (int p = 0; p < kCluster; ++p) x[p] = p < ck ? load_of(sum + e, p) : 0.f;
#pragma unroll
                    for (int p = 0; p < kCluster; ++p) s += x[p];
                    const int lane = e >> 2 & 31, row = (e >> 7) * 8 + 2 * (lane & 3) + (e & 1);
                    const int r = r0 + (lane >> 2) + 8 * (e >> 1 & 1);
                    // a rank of the padding would be NaN in a row of x with an infinity
                    if (row < n) t[static_cast<size_t>(s_rows[row]) * v.rpad + r] = r < info.rank ? s * info.scale : 0.f;
                }
            }
            if (ck > 1) cluster_sync();                      // nobody goes on while its sums are read
            else __syncthreads();
        }
    }
}

// out = y + t . B^T.  A unit is 32 columns of 16 rows of a class; every warp
// takes an equal run of units, class after class, and keeps t of its 16 rows
// in registers as MMA fragments, high and low part.  Rows are the MMA's rows,
// columns its columns, in the order that gives a thread 8 consecutive ones.
struct Run {
    int nb;                  // column blocks of a group of 16 rows
    int64_t u, end;          // the warp's units
    template <int R>
    __device__ Run(const Classes<R> &k, int N, int cta, int ctas) : nb((N + 31) / 32) {
        const int warps = ctas * kWarps, me = cta * kWarps + (threadIdx.x >> 5);
        const int64_t units = static_cast<int64_t>(k.units[k.n]) * nb;
        u = units * me / warps;
        end = units * (me + 1) / warps;
    }
};
// B and y of the warp's units into L2.
template <int R>
__device__ __forceinline__ void prefetch_units(const LoraView &v, const LoraCall &c, const Classes<R> &k, const Run &run) {
    const int lane = threadIdx.x & 31, nb = run.nb;
    auto prefetch = [](const uint16_t *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory"); };
    for (int64_t w = run.u; w < run.end;) {
        const int group = static_cast<int>(w / nb), b0 = static_cast<int>(w % nb);
        const int b1 = static_cast<int>(min(static_cast<int64_t>(nb), b0 + (run.end - w)));
        w += b1 - b0;
        const int id = class_of(k, group), rank = k.rank[id];
        const int r0 = k.first[id] + 16 * (group - k.units[id]), n = min(16, k.first[id + 1] - r0);
        if (rank) {
            const uint16_t *b = v.b + static_cast<size_t>(k.slot[id]) * v.rpad * v.N;
            const int64_t last = static_cast<int64_t>(min(32 * b1, v.N)) * rank;
            for (int64_t e = static_cast<int64_t>(32 * b0) * rank + 64 * lane; e < last; e += 64 * 32) prefetch(b + e);
        }
        for (int e = lane; e < n * (b1 - b0); e += 32)
            prefetch(c.y + k.row[r0 + e % n] * c.ys + 32 * (b0 + e / n));
    }
}
// t: [row][pitch] in global memory, written by another launch, or in shared memory.
template <bool BF, bool Shared, int R>
__device__ __forceinline__ void expand_units(const LoraView &v, const LoraCall &c, const Classes<R> &k, const Run &run,
                                             const float *t, int pitch) {
    const int lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3, nb = run.nb;
    auto load4 = [](const float4 *p) {
        if constexpr (Shared) return *p;
        else return __ldcg(p);
    };
    const int64_t end = run.end;
    for (int64_t u = run.u; u < end;) {
        const int group = static_cast<int>(u / nb), b0 = static_cast<int>(u % nb);
        const int b1 = static_cast<int>(min(static_cast<int64_t>(nb), b0 + (end - u)));
        u += b1 - b0;
        const int id = class_of(k, group), rank = k.rank[id], steps = (rank + 31) / 32, rg = rank / 8;
        const int r0 = k.first[id] + 16 * (group - k.units[id]) + g, r1 = k.first[id + 1];
        const uint16_t *b = v.b + (rank ? static_cast<size_t>(k.slot[id]) * v.rpad * v.N : 0);
        const bool have[2] = {r0 < r1, r0 + 8 < r1};
        const int64_t row[2] = {have[0] ? k.row[r0] : 0, have[1] ? k.row[r0 + 8] : 0};
        if (rank == 0 && c.out == c.y) continue;
        // t of 32 ranks: the lane's 8 ranks of its two rows
        float x[2][8];
        auto load = [&](int s) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4 p = make_float4(0.f, 0.f, 0.f, 0.f), r = p;
                if (have[h] && 32 * s + 8 * q < rank) {
                    const float4 *at = reinterpret_cast<const float4 *>(t + row[h] * pitch + 32 * s + 8 * q);
                    p = load4(at);
                    r = load4(at + 1);
                }
                x[h][0] = p.x, x[h][1] = p.y, x[h][2] = p.z, x[h][3] = p.w;
                x[h][4] = r.x, x[h][5] = r.y, x[h][6] = r.z, x[h][7] = r.w;
            }
        };
        float up[2] = {1.f, 1.f}, down[2] = {1.f, 1.f};
        if constexpr (!BF) {
            float top[2] = {0.f, 0.f};
            for (int s = 0; s < steps; ++s) {
                load(s);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 8; ++e) top[h] = fmaxf(top[h], fabsf(x[h][e]));
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
                up[h] = split_scale_of(top[h]);
                down[h] = 1.f / up[h];               // a power of two: exact
            }
        }
        uint32_t f[2][4][4];                         // fragments of 64 ranks: [32 ranks][k16 half, part][register]
        auto fragments = [&](int s, uint32_t (&o)[4][4]) {
            load(s);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const float y0 = x[h][e] * down[h], y1 = x[h][e + 1] * down[h];
                    const uint16_t h0 = to16<BF>(y0), h1 = to16<BF>(y1);
                    const int half = e >> 2, reg = (e >> 1 & 1) * 2 + h;
                    o[2 * half][reg] = h0 | static_cast<uint32_t>(h1) << 16;
                    o[2 * half + 1][reg] = split_low<BF>(y0, h0) | static_cast<uint32_t>(split_low<BF>(y1, h1)) << 16;
                }
        };
#pragma unroll
        for (int s = 0; s < 2; ++s)
            if (s < steps) fragments(s, f[s]);
        for (int blk = b0; blk < b1; ++blk) {
            const int col = 32 * blk + 8 * q;        // the thread's 8 columns of out
            uint4 y[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                y[h] = make_uint4(0, 0, 0, 0);
                if (have[h] && col < v.N) y[h] = *reinterpret_cast<const uint4 *>(c.y + row[h] * c.ys + col);
            }
            float acc[4][4] = {};
            auto product = [&](int s, const uint32_t (&t)[4][4]) {
                uint4 w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    // MMA column g of tile j is column 8 (g / 2) + 2 j + g % 2 of the 32
                    const int cg = 4 * blk + (g >> 1), in = 2 * j + (g & 1), kb = 4 * s + q;
                    w[j] = make_uint4(0, 0, 0, 0);
                    if (cg * 8 < v.N && kb < rg) w[j] = ldg_stream(b + (static_cast<size_t>(cg) * rg + kb) * 64 + in * 8);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma16816<BF>(acc[j], t[i][0], t[i][1], t[i][2], t[i][3], i < 2 ? w[j].x : w[j].z,
                                     i < 2 ? w[j].y : w[j].w);
            };
            if (steps > 0) product(0, f[0]);
            if (steps > 1) product(1, f[1]);
            for (int s = 2; s < steps; ++s) {        // ranks past 64: their fragments are made anew
                uint32_t more[4][4];
                fragments(s, more);
                product(s, more);
            }
            if (col >= v.N) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!have[h]) continue;
                uint32_t *yw = reinterpret_cast<uint32_t *>(&y[h]);
                if (rank)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 o = unpack2<BF>(yw[j]);
                        yw[j] = pack2<BF>(fmaf(acc[j][2 * h], up[h], o.x), fmaf(acc[j][2 * h + 1], up[h], o.y));
                    }
                *reinterpret_cast<uint4 *>(c.out + row[h] * c.os + col) = y[h];
            }
        }
    }
}

template <bool BF, int R>
__global__ void __launch_bounds__(32 * kWarps, 2) lora_expand_kernel(LoraView v, LoraCall call) {
    __shared__ Classes<R> k;
    __shared__ Scratch<R> scratch;
    for (Chunks<R> chunks(call, blockIdx.x, gridDim.x); chunks.more(); chunks.next()) {
        LoraCall c = call;
        const int m0 = chunks.chunk(c) * c.chunk;
        find_classes(v, c, m0, k, scratch, [](int rows, int) { return (rows + 15) / 16; });
        c.y += m0 * c.ys;
        c.out += m0 * c.os;
        const Run run(k, v.N, chunks.me, chunks.all);
        prefetch_units(v, c, k, run);                    // while the first launch runs
        asm volatile("griddepcontrol.wait;" ::: "memory");
        expand_units<BF, false>(v, c, k, run, v.t + static_cast<size_t>(m0) * v.rpad, v.rpad);
        __syncthreads();                                 // the classes have been read
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // without a chunk, too
}

// Both products in one launch, for a single row whose adapter has few values:
// every cluster forms all of t for itself, its CTAs a part of K each, and its
// warps then have their share of the columns.  At 4096 x 4096, rank 16, the
// GPU takes 5.4 us instead of 7.3 and a call from the host 9.5 instead of 12;
// at 8192 x 28672, rank 64, the GPU 5.8 instead of 8.4.  The same with the
// classes of two to four rows was no faster than two launches (4 rows of 4096 x
// 11008, rank 16: 9.2 and 8.5 us; 3 rows, rank 64: 14 and 9.7).
constexpr int kOneCtas = 8;          // of a cluster
constexpr int kOneClusters = 16;     // at most: one wave
constexpr int kOneRank = 256;
constexpr int64_t kOneValues = 1 << 19;      // of A
template <bool BF>
__global__ void __launch_bounds__(32 * kWarps, 2) lora_one_kernel(LoraView v, LoraCall c) {
    __shared__ Classes<32> k;
    __shared__ __align__(16) float part[kOneRank / 16 * 128];                // [16 ranks, part of K][128]
    __shared__ __align__(16) float t[kOneRank];
    const int warp = threadIdx.x >> 5, cta = blockIdx.x % kOneCtas;
    int slot = c.row_slot[0];
    if (slot >= v.slots) {
        if (threadIdx.x == 0) atomicOr(v.status, kLoraBadSlot);
        slot = -1;
    }
    slot = max(slot, -1);
    LoraSlot info{0, 0.f, 1};
    if (slot >= 0) info = v.slot[slot];
    const int rank = ceil16(info.rank);
    if (threadIdx.x <= 32) k.units[threadIdx.x] = threadIdx.x > 0;           // one class, of one row
    if (threadIdx.x == 0) {
        k.n = 1;
        k.slot[0] = slot;
        k.rank[0] = rank;
        k.first[0] = k.row[0] = 0;
        k.first[1] = 1;
    }
    __syncthreads();
    const Run run(k, v.N, blockIdx.x, gridDim.x);
    prefetch_units(v, c, k, run);
    const int units = rank / 16, split = max(1, kWarps / max(units, 1));     // warps of 16 ranks along K
    for (int job = warp; job < units * split; job += kWarps)
        shrink_rows<BF, 1>(v, c, v.a + static_cast<size_t>(slot) * v.rpad * ceil64(v.K) + static_cast<size_t>(job / split) * 1024,
                           rank / 8, k.row, 1, cta * split + job % split, kOneCtas * split,
                           reinterpret_cast<float4 *>(part) + job * 32, 0);
    __syncthreads();
    // the warps' parts of K in order, then the cluster's; a thread has a rank, at its place as shrink_rows left it
    const int r = threadIdx.x;
    float *at = part + r / 16 * split * 128 + (r & 7) * 16 + (r >> 3 & 1) * 2;
    if (r < rank)
        for (int w = 1; w < split; ++w) *at += at[w * 128];
    __syncwarp();
    cluster_sync();
    if (r < rank) {
        float x[kOneCtas], sum = 0.f;
#pragma unroll
        for (int p = 0; p < kOneCtas; ++p) x[p] = load_of(at, p);
#pragma unroll
        for (int p = 0; p < kOneCtas; ++p) sum += x[p];
        t[r] = r < info.rank ? sum * info.scale : 0.f;
    }
    __syncthreads();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");    // nobody leaves while its sums are read
    expand_units<BF, true>(v, c, k, run, t, 0);
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
static_assert(kOneRank <= 32 * kWarps && kOneRank / 16 >= kWarps, "a thread for each rank, a part for every warp");

template <class... P, class... T>
cudaError_t start(void (*k)(P...), dim3 grid, int threads, int smem, int cluster, bool dependent, cudaStream_t st,
                  T... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (cluster > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = cluster;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    if (dependent && pdl_enabled()) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
        ++cfg.numAttrs;
    }
    return cudaLaunchKernelEx(&cfg, k, args...);
}

}  // namespace

cudaError_t launch_lora_set(const LoraView &v, uint16_t *a, uint16_t *b, LoraSlot *slot, int s, const uint16_t *src_a,
                            const uint16_t *src_b, int rank, float scale, bool bf16, cudaStream_t st) {
    const int r16 = ceil16(rank);
    const size_t n = static_cast<size_t>(r16) * std::max(ceil64(v.K), v.N);
    const int grid = static_cast<int>(std::min<size_t>(n / 256 + 1, 1216));
    lora_slot_kernel<<<1, 1, 0, st>>>(slot + s, rank, scale);
    if (rank)
        lora_set_kernel<<<grid, 256, 0, st>>>(a + static_cast<size_t>(s) * v.rpad * ceil64(v.K),
                                              b + static_cast<size_t>(s) * v.rpad * v.N, slot + s, src_a, src_b, v.K,
                                              v.N, rank, r16, bf16 ? 0x7f80 : 0x7c00);
    return cudaGetLastError();
}

// The two launches.
template <int R>
cudaError_t launch_pair(const LoraView &v, const LoraCall &c, int chunks, bool bf16, cudaStream_t st, int *launches) {
    const int rows = std::min(c.M, c.chunk);
    // units that one chunk can hold, and two CTAs for each SM over them; K is split over a cluster where the units
    // alone are fewer
    const int units = (std::min(rows, v.slots) + (rows - 1) / kRows) * (v.rpad / 16);
    int ck = kCluster;
    while (ck > 1 && (static_cast<int64_t>(units) * chunks * ck > 2 * 304 || v.K / ck < 512)) ck /= 2;
    if (c.marks) ck = 2;                                 // how many chunks are marked is not known here
    const int gx = static_cast<int>(std::min<int64_t>(c.marks ? 304 : units, std::max<int64_t>(1, 304 / (static_cast<int64_t>(ck) * chunks))));
    // two CTAs for each SM, as long as every warp has a unit
    const int groups = (rows + 15) / 16 + std::min(rows, v.slots + 1);
    const int64_t most = static_cast<int64_t>(groups) * ((v.N + 31) / 32);
    const int ex = static_cast<int>(std::min<int64_t>((most + kWarps - 1) / kWarps, std::max(1, 304 / chunks)));
    const dim3 gs(gx * ck, chunks), ge(ex, chunks);
    auto shrink = bf16 ? lora_shrink_kernel<true, false, R> : lora_shrink_kernel<false, false, R>;
    if constexpr (R == 64)
        if (rows <= 16) shrink = bf16 ? lora_shrink_kernel<true, true, R> : lora_shrink_kernel<false, true, R>;
    cudaError_t e = start(shrink, gs, 32 * kWarps, 0, ck, false, st, v, c, ck);
    if (!e) e = start(bf16 ? lora_expand_kernel<true, R> : lora_expand_kernel<false, R>, ge, 32 * kWarps, 0, 1, true, st, v, c);
    if (!e) *launches += 2;
    return e;
}
// For chunks of R rows (the grid's y dimension); the chunks of 256 share the
// rows equally, as one is most of a call.
template <int R>
cudaError_t launch_chunks(const LoraView &v, const LoraCall &c, bool bf16, cudaStream_t st, int *launches) {
    const int chunks_all = (c.M + R - 1) / R;
    const int each = R == 64 ? R : (c.M + chunks_all - 1) / chunks_all;
    for (int c0 = 0; c0 < chunks_all; c0 += 65535) {
        LoraCall d = c;
        LoraView w = v;
        const int64_t m0 = static_cast<int64_t>(c0) * each;
        const int chunks = std::min(chunks_all - c0, 65535);
        d.M = static_cast<int>(std::min<int64_t>(c.M - m0, static_cast<int64_t>(chunks) * each));
        d.chunk = each;
        d.x += m0 * c.xs;
        d.y += m0 * c.ys;
        d.out += m0 * c.os;
        d.row_slot += m0;
        w.t += m0 * v.rpad;
        if (cudaError_t e = launch_pair<R>(w, d, chunks, bf16, st, launches)) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_lora_add(const LoraView &v, const LoraCall &c, bool bf16, cudaStream_t st, int *launches) {
    if (c.M == 1 && v.rpad <= kOneRank && static_cast<int64_t>(v.rpad) * v.K <= kOneValues) {
        const int clusters = std::min((v.N + 32 * kWarps * kOneCtas - 1) / (32 * kWarps * kOneCtas), kOneClusters);
        *launches += 1;
        return start(bf16 ? lora_one_kernel<true> : lora_one_kernel<false>, dim3(clusters * kOneCtas), 32 * kWarps, 0,
                     kOneCtas, false, st, v, c);
    }
    // Chunks of 256 read an adapter that their rows share once, but sort and sum them more slowly than chunks of 64.
    // Where those could read more than 96 MB again: 256 rows over 32 adapters of up to 64 ranks, 8192 x 28672, 44 us
    // instead of 101; 256 rows in 4 runs 32 instead of 37.  Where not: 100 rows over 32 adapters of up to 32
    // ranks, 8192 x 10240, 20 us by 256, 17 by 64; 200 rows over 8 of 16, 4096 x 4096, 13.4 and 11.8.
    const int64_t again = static_cast<int64_t>((c.M - 1) / 64) * std::min(64, v.slots) * v.rpad * (v.K + v.N) * 2;
    return again > 96 << 20 ? launch_chunks<256>(v, c, bf16, st, launches) : launch_chunks<64>(v, c, bf16, st, launches);
}

cudaError_t launch_lora_marked(const LoraView &v, const LoraCall &c, bool bf16, cudaStream_t st, int *launches) {
    return launch_pair<256>(v, c, 1, bf16, st, launches);
}

}  // namespace q4
