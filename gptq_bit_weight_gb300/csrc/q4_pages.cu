// The pages of a cache: which are in use, forks, copies, and moving those in
// use together.
//
// A page is in use if a row of the table names it below the row's length: one
// bit a page, set by every entry (or-ing bits gives the same bits in any
// order).  Ranks among used and unused pages are counts of bits; every CTA
// counts those before its own words for itself (2^22 pages are 512 KB, which
// stay in L2), so no CTA waits for another.  Bound by the contents that move:
// read once and written once, in 16-byte vectors, four on their way in a thread.
#include "q4_pages.cuh"

#include <algorithm>

namespace q4 {
namespace {

constexpr int kThreads = 256;

// Whether a request of n tokens needs its j-th page.
__device__ __forceinline__ bool needed(const PageRows &r, int page_size, int64_t j, int64_t n) {
    const int64_t at = j * page_size;
    return at < n && (r.window == 0 || at < r.sinks || at + page_size > n - r.window);
}

__global__ void __launch_bounds__(kThreads) mark_kernel(PagesView v, PageRows r) {
    const int64_t n = static_cast<int64_t>(r.batch) * r.width, step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n; i += step) {
        const int64_t b = i / r.width, j = i - b * r.width;
        if (!needed(r, v.page_size, j, r.kv_len[b])) continue;
        const int id = r.table[b * r.stride + j];
        if (id >= v.pages) atomicOr(v.status, kPagesBadIndex);
        else if (id >= 0) atomicOr(v.used + (id >> 5), 1u << (id & 31));
    }
}

// The sum of `mine` over the CTA's threads, for all of them.
__device__ __forceinline__ int sum_all(int mine, int *s_sum) {
    mine = __reduce_add_sync(0xffffffffu, mine);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = mine;
    __syncthreads();
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) sum += s_sum[w];
    return sum;
}
// Bits of `used` below bit `end`, counted by the whole CTA.
__device__ __forceinline__ int used_below(const PagesView &v, int end, int *s_sum) {
    int mine = 0;
    const int words = end >> 5;
    for (int i = threadIdx.x; i < words / 4; i += kThreads) {
        const uint4 w = reinterpret_cast<const uint4 *>(v.used)[i];
        mine += __popc(w.x) + __popc(w.y) + __popc(w.z) + __popc(w.w);
    }
    if (threadIdx.x < words % 4) mine += __popc(v.used[(words & ~3) + threadIdx.x]);
    if (threadIdx.x == 0 && (end & 31)) mine += __popc(v.used[words] & ((1u << (end & 31)) - 1));
    return sum_all(mine, s_sum);
}
// A CTA goes over pages [first, first + 1024), a warp over 128 of them, a lane
// over those of four words' bit `lane`: f(id, used, rank among used pages).
template <class F>
__device__ __forceinline__ void for_pages(const PagesView &v, int first, int *s_sum, F f) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int before = used_below(v, min(first, v.pages), s_sum);
    for (int w = 0; w < 4 * (kThreads / 32); ++w) {
        const int id0 = first + 32 * w;
        if (id0 >= v.pages) return;
        const uint32_t bits = v.used[id0 >> 5];
        if (w / 4 == warp && id0 + lane < v.pages)
            f(id0 + lane, (bits >> lane & 1) != 0, before + __popc(bits & ((1u << lane) - 1)));
        before += __popc(bits);
    }
}
constexpr int kPagesOfCta = 4 * kThreads;

__global__ void __launch_bounds__(kThreads) free_list_kernel(PagesView v, int32_t *ids, int32_t *count) {
    __shared__ int s_sum[kThreads / 32];
    const int used = used_below(v, v.pages, s_sum), free = v.pages - used;
    if (blockIdx.x == 0 && threadIdx.x == 0) *count = free;
    for_pages(v, blockIdx.x * kPagesOfCta, s_sum, [&](int id, bool in_use, int rank) {
        if (in_use) ids[free + rank] = -1;
        else ids[id - rank] = id;
    });
}

// Of a compaction: the i-th page that has to move and the i-th number that it may take.
__global__ void __launch_bounds__(kThreads) plan_kernel(PagesView v, int32_t *count) {
    __shared__ int s_sum[kThreads / 32];
    const int used = used_below(v, v.pages, s_sum), stay = used_below(v, used, s_sum);
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        *count = used;
        *v.moves = used - stay;
    }
    for_pages(v, blockIdx.x * kPagesOfCta, s_sum, [&](int id, bool in_use, int rank) {
        if (in_use && id >= used) {
            v.source[rank - stay] = id;
            v.rank[id] = rank - stay;
        } else if (!in_use && id < used) {
            v.hole[id - rank] = id;
        }
    });
}

// Copies a chunk of page src to page dst, by the CTA.
__device__ __forceinline__ void copy_chunk(const PageChunk &c, int src, int dst) {
    const uint4 *from = reinterpret_cast<const uint4 *>(c.data + src * c.stride);
    uint4 *to = reinterpret_cast<uint4 *>(c.data + dst * c.stride);
    const int n = c.bytes / 16;
    uint4 x[kPageChunk / 16 / kThreads];
#pragma unroll
    for (int i = 0; i < kPageChunk / 16 / kThreads; ++i)
        if (static_cast<int>(threadIdx.x) + i * kThreads < n) x[i] = __ldcs(from + threadIdx.x + i * kThreads);
#pragma unroll
    for (int i = 0; i < kPageChunk / 16 / kThreads; ++i)
        if (static_cast<int>(threadIdx.x) + i * kThreads < n) __stcs(to + threadIdx.x + i * kThreads, x[i]);
}

__global__ void __launch_bounds__(kThreads)
    move_kernel(PagesView v, PageRows r, int32_t *out, int64_t out_stride, const int32_t *count) {
    const int used = *count, moves = *v.moves;
    const int64_t entries = static_cast<int64_t>(r.batch) * r.width, step = static_cast<int64_t>(gridDim.x) * kThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < entries; i += step) {
        const int64_t b = i / r.width, j = i - b * r.width;
        int id = -1;
        if (needed(r, v.page_size, j, r.kv_len[b])) id = r.table[b * r.stride + j];
        if (id >= v.pages || id < 0) id = -1;
        else if (id >= used) id = v.hole[v.rank[id]];
        out[b * out_stride + j] = id;
    }
    const int64_t work = static_cast<int64_t>(moves) * v.chunks;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int m = static_cast<int>(w / v.chunks);
        copy_chunk(v.chunk[w - static_cast<int64_t>(m) * v.chunks], v.source[m], v.hole[m]);
    }
}

__global__ void __launch_bounds__(kThreads) copy_kernel(PagesView v, const int32_t *src, const int32_t *dst, int n) {
    const int64_t work = static_cast<int64_t>(n) * v.chunks;
    for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
        const int m = static_cast<int>(w / v.chunks), c = static_cast<int>(w - static_cast<int64_t>(m) * v.chunks);
        const int s = src[m], d = dst[m];
        if (s >= v.pages || d >= v.pages) {
            if (c == 0 && threadIdx.x == 0) atomicOr(v.status, kPagesBadIndex);
        } else if (s >= 0 && d >= 0 && s != d) {
            copy_chunk(v.chunk[c], s, d);
        }
    }
}

// CTAs (x, i): fork i, its chunks x, x + gridDim.x, ..; x = 0 writes the row.
// Each finds out for itself whether the fork is to be done, from what no CTA writes: rows of
// parents are not written, since no child is a parent.
__global__ void __launch_bounds__(kThreads)
    fork_kernel(PagesView v, PageRows r, const int32_t *parent, const int32_t *child, const int32_t *fresh, int n) {
    __shared__ int s_sum[kThreads / 32];
    const int i = blockIdx.y, p = parent[i], c = child[i];
    if (p < 0 || c < 0 || p == c) return;
    const bool rows_ok = p < r.batch && c < r.batch;
    const int64_t len = rows_ok ? r.kv_len[p] : 0;
    bool ok = rows_ok && len >= 0 && len <= static_cast<int64_t>(r.width) * v.page_size;
    const int64_t last = len / v.page_size;
    const bool part = ok && len % v.page_size;
    const int from = part ? r.table[p * r.stride + last] : 0, to = part ? fresh[i] : 0;
    ok = ok && from >= 0 && from < v.pages && to >= 0 && to < v.pages;
    int clash = 0;
    if (ok)
        for (int k = threadIdx.x; k < n; k += kThreads) {
            const int pk = parent[k], ck = child[k];
            if (pk < 0 || ck < 0 || pk == ck) {
                clash |= pk >= 0 && pk == ck && pk == c;             // a row that is to stay
                continue;
            }
            clash |= pk == c || (k < i && (ck == c || (part && fresh[k] == to)));
        }
    if (sum_all(clash, s_sum)) ok = false;
    if (!ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(v.status, kPagesBadFork);
        return;
    }
    if (blockIdx.x == 0) {
        for (int j = threadIdx.x; j < r.width; j += kThreads) {
            const int64_t at = static_cast<int64_t>(j) * v.page_size;
            r.table[c * r.stride + j] = at >= len ? -1 : part && j == last ? to : r.table[p * r.stride + j];
        }
        if (threadIdx.x == 0) r.kv_len[c] = static_cast<int32_t>(len);
    }
    if (part)
        for (int k = blockIdx.x; k < v.chunks; k += gridDim.x) copy_chunk(v.chunk[k], from, to);
}

int grid_of(int64_t work, int most) { return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(work, most))); }

cudaError_t launch_mark(const PagesView &v, const PageRows &r, cudaStream_t st, int *launches) {
    if (cudaError_t e = cudaMemsetAsync(v.used, 0, sizeof(uint32_t) * v.words, st)) return e;
    const int64_t entries = static_cast<int64_t>(r.batch) * r.width;
    if (entries == 0) return cudaSuccess;
    mark_kernel<<<grid_of((entries + kThreads - 1) / kThreads, 8 * v.sms), kThreads, 0, st>>>(v, r);
    *launches += 1;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_pages_free_list(const PagesView &v, const PageRows &r, int32_t *ids, int32_t *count, cudaStream_t st,
                                   int *launches) {
    if (cudaError_t e = launch_mark(v, r, st, launches)) return e;
    free_list_kernel<<<(v.pages + kPagesOfCta - 1) / kPagesOfCta, kThreads, 0, st>>>(v, ids, count);
    *launches += 1;
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PagesView &v, const PageRows &r, int32_t *out, int64_t out_stride, int32_t *count,
                                 cudaStream_t st, int *launches) {
    if (cudaError_t e = launch_mark(v, r, st, launches)) return e;
    plan_kernel<<<(v.pages + kPagesOfCta - 1) / kPagesOfCta, kThreads, 0, st>>>(v, count);
    *launches += 1;
    if (cudaError_t e = cudaGetLastError()) return e;
    move_kernel<<<8 * v.sms, kThreads, 0, st>>>(v, r, out, out_stride, count);
    *launches += 1;
    return cudaGetLastError();
}

cudaError_t launch_pages_copy(const PagesView &v, const int32_t *src, const int32_t *dst, int n, cudaStream_t st) {
    copy_kernel<<<grid_of(static_cast<int64_t>(n) * std::max(v.chunks, 1), 8 * v.sms), kThreads, 0, st>>>(v, src, dst, n);
    return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PagesView &v, const PageRows &r, const int32_t *parent, const int32_t *child,
                              const int32_t *fresh, int n, cudaStream_t st) {
    const int x = std::max(1, std::min(v.chunks, 8 * v.sms / n + 1));
    fork_kernel<<<dim3(x, n), kThreads, 0, st>>>(v, r, parent, child, fresh, n);
    return cudaGetLastError();
}

}  // namespace q4
