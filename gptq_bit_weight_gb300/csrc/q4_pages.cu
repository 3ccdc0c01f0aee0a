// The pages of a cache: which are in use, forks, copies, and moving those in
// use together.
//
// A page is in use if a row of the table names it below the row's length: one
// bit a page, set by every entry (or-ing bits gives the same bits in any
// order).  Ranks among used and unused pages are counts of bits; every CTA
// counts those before its own words for itself (2^22 pages are 512 KB, which
// stay in L2), so no CTA waits for another.  Bound by the contents that move:
// read once and written once, in 16-byte vectors, four on their way in a thread,
// where the next ones lie read meanwhile.  Compaction of 16384 pages over 32 layers,
// 5.03 GB moved: 826 us, 6.1 TB/s; of 600 pages, 128 MB: 27; 48 forks that copy
// 4 MiB each: 60 (6.7 TB/s, L2 among it).  Small pools are latency, and mostly the
// host's: one launch for their bits and counts instead of three.
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

// A chunk of one page to another.
struct Job {
    const uint4 *from;
    uint4 *to;
    int n;                   // 16-byte vectors; 0: nothing
};
__device__ __forceinline__ Job job_of(const PageChunk &c, int src, int dst) {
    return Job{reinterpret_cast<const uint4 *>(c.data + src * c.stride), reinterpret_cast<uint4 *>(c.data + dst * c.stride), c.bytes / 16};
}
constexpr int kVectors = kPageChunk / 16 / kThreads;         // of a thread
__device__ __forceinline__ void load_job(const Job &j, uint4 (&x)[kVectors]) {
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
        if (static_cast<int>(threadIdx.x) + i * kThreads < j.n) x[i] = __ldcs(j.from + threadIdx.x + i * kThreads);
}
__device__ __forceinline__ void store_job(const Job &j, const uint4 (&x)[kVectors]) {
#pragma unroll
    for (int i = 0; i < kVectors; ++i)
        if (static_cast<int>(threadIdx.x) + i * kThreads < j.n) __stcs(j.to + threadIdx.x + i * kThreads, x[i]);
}
// Jobs of(w) for w = first, first + step, .. below `work`, by the CTA: where a job's data is and goes is read while the
// job before is on its way.
template <class F>
__device__ __forceinline__ void copy_jobs(int64_t first, int64_t step, int64_t work, F of) {
    if (first >= work) return;
    Job j = of(first);
    for (int64_t w = first; w < work; w += step) {
        uint4 x[kVectors];
        load_job(j, x);
        Job next{};
        if (w + step < work) next = of(w + step);
        store_job(j, x);
        j = next;
    }
}

__global__ void __launch_bounds__(kThreads, 4)
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
    copy_jobs(blockIdx.x, gridDim.x, static_cast<int64_t>(moves) * v.chunks, [&](int64_t w) {
        const int m = static_cast<int>(w / v.chunks);
        return job_of(v.chunk[w - static_cast<int64_t>(m) * v.chunks], v.source[m], v.hole[m]);
    });
}

__global__ void __launch_bounds__(kThreads, 4) copy_kernel(PagesView v, const int32_t *src, const int32_t *dst, int n) {
    copy_jobs(blockIdx.x, gridDim.x, static_cast<int64_t>(n) * v.chunks, [&](int64_t w) {
        const int m = static_cast<int>(w / v.chunks), c = static_cast<int>(w - static_cast<int64_t>(m) * v.chunks);
        const int s = src[m], d = dst[m];
        if (s >= v.pages || d >= v.pages) {
            if (c == 0 && threadIdx.x == 0) atomicOr(v.status, kPagesBadIndex);
            return Job{};
        }
        return s >= 0 && d >= 0 && s != d ? job_of(v.chunk[c], s, d) : Job{};
    });
}

// CTAs (x, i): fork i, its chunks x, x + gridDim.x, ..; x = 0 writes the row.
// Each finds out for itself whether the fork is to be done, from what no CTA writes: rows and
// lengths of parents are not written, since no child is a parent.
__global__ void __launch_bounds__(kThreads, 5)
    fork_kernel(PagesView v, PageRows r, const int32_t *parent, const int32_t *child, const int32_t *fresh, int n) {
    __shared__ int s_sum[kThreads / 32];
    const int i = blockIdx.y, p = parent[i], c = child[i];
    if (p < 0 || c < 0 || p == c) return;
    const bool rows_ok = p < r.batch && c < r.batch;
    const int64_t len = rows_ok ? r.kv_len[p] : 0, most = static_cast<int64_t>(r.width) * v.page_size;
    bool ok = rows_ok && len >= 0 && len <= most;
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
            clash |= pk == c || (k < i && ck == c);
            if (part && k < i && fresh[k] == to && pk < r.batch) {   // an earlier fork's, if that needs one
                const int64_t lk = r.kv_len[pk];
                clash |= lk >= 0 && lk <= most && lk % v.page_size != 0;
            }
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
    if (part) copy_jobs(blockIdx.x, gridDim.x, v.chunks, [&](int64_t k) { return job_of(v.chunk[k], from, to); });
}

// A small pool and table in one launch of one CTA: bits, their counts and what follows from them in shared memory.
constexpr int kSmallThreads = 1024, kSmallPages = 32 * kSmallThreads, kSmallEntries = 8 * kSmallThreads;
bool is_small(const PagesView &v, const PageRows &r) {
    return v.pages <= kSmallPages && static_cast<int64_t>(r.batch) * r.width <= kSmallEntries;
}
// PLAN: a compaction's moves; else the free list.
template <bool PLAN>
__global__ void __launch_bounds__(kSmallThreads) small_kernel(PagesView v, PageRows r, int32_t *ids, int32_t *count) {
    __shared__ uint32_t bits[kSmallThreads], below[kSmallThreads], of_warp[kSmallThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bits[tid] = 0;
    __syncthreads();
    const int entries = r.batch * r.width;
#pragma unroll 4
    for (int i = tid; i < entries; i += kSmallThreads) {
        const int b = i / r.width, j = i - b * r.width;
        const int id = r.table[b * r.stride + j], n = r.kv_len[b];           // (both on their way at once)
        if (!needed(r, v.page_size, j, n)) continue;
        if (id >= v.pages) atomicOr(v.status, kPagesBadIndex);
        else if (id >= 0) atomicOr(bits + (id >> 5), 1u << (id & 31));
    }
    __syncthreads();
    const uint32_t mine = __popc(bits[tid]);
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) of_warp[warp] = upto;
    __syncthreads();
    uint32_t before = 0, used = 0;
#pragma unroll
    for (int w = 0; w < kSmallThreads / 32; ++w) {
        if (w < warp) before += of_warp[w];
        used += of_warp[w];
    }
    below[tid] = before + upto - mine;
    __syncthreads();
    auto rank_of = [&](int id) { return static_cast<int>(below[id >> 5] + __popc(bits[id >> 5] & ((1u << (id & 31)) - 1))); };
    const int n = static_cast<int>(used), free = v.pages - n, stay = n < v.pages ? rank_of(n) : n;
    if (tid == 0) {
        *count = PLAN ? n : free;
        if (PLAN) *v.moves = n - stay;
    }
    for (int id = tid; id < v.pages; id += kSmallThreads) {
        const bool in_use = bits[id >> 5] >> (id & 31) & 1;
        const int rank = rank_of(id);
        if constexpr (PLAN) {
            if (in_use && id >= n) {
                v.source[rank - stay] = id;
                v.rank[id] = rank - stay;
            } else if (!in_use && id < n) {
                v.hole[id - rank] = id;
            }
        } else if (in_use) {
            ids[free + rank] = -1;
        } else {
            ids[id - rank] = id;
        }
    }
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
    if (is_small(v, r)) {
        small_kernel<false><<<1, kSmallThreads, 0, st>>>(v, r, ids, count);
        *launches += 1;
        return cudaGetLastError();
    }
    if (cudaError_t e = launch_mark(v, r, st, launches)) return e;
    free_list_kernel<<<(v.pages + kPagesOfCta - 1) / kPagesOfCta, kThreads, 0, st>>>(v, ids, count);
    *launches += 1;
    return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PagesView &v, const PageRows &r, int32_t *out, int64_t out_stride, int32_t *count,
                                 cudaStream_t st, int *launches) {
    if (is_small(v, r)) {
        small_kernel<true><<<1, kSmallThreads, 0, st>>>(v, r, nullptr, count);
    } else {
        if (cudaError_t e = launch_mark(v, r, st, launches)) return e;
        plan_kernel<<<(v.pages + kPagesOfCta - 1) / kPagesOfCta, kThreads, 0, st>>>(v, count);
    }
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
