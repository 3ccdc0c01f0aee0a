// C ABI of the pages of a cache (gptq_q4_pages_*): argument checks and the
// handle's memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <new>

#include "q4_handle.h"
#include "q4_pages.cuh"

struct gptq_q4_pages_s {
    int device = -1;
    q4::PagesView view{};
    q4::PageChunk *chunk = nullptr;
};

namespace {

using q4::api_cuda_fail;
using q4::api_failf;
using q4::api_set_status;

constexpr int kMaxForks = 4096;
constexpr int kMaxRows = 1 << 20;

bool aligned(const void *p, int n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int check(gptq_q4_pages h) {
    if (!h) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "pages handle is NULL");
    int dev = -1;
    if (cudaError_t e = cudaGetDevice(&dev)) return api_cuda_fail(e, "cudaGetDevice");
    if (dev != h->device)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "the pages handle was made on device %d, current device is %d",
                         h->device, dev);
    return GPTQ_Q4_OK;
}

int check_rows(const gptq_q4_rows *r, int window, int sinks) {
    if (!r) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "rows must not be NULL");
    if (r->batch < 0 || r->batch > kMaxRows || r->width < 0 || r->table_stride < r->width)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "batch=%d must be 0 .. %d, width=%d not negative and table_stride=%lld at least width", r->batch,
                         kMaxRows, r->width, static_cast<long long>(r->table_stride));
    if (window < 0 || sinks < 0)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "window=%d and sinks=%d must not be negative", window, sinks);
    if (r->batch && (!r->kv_len || (r->width && !r->table) || !aligned(r->kv_len, 4) || !aligned(r->table, 4)))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "kv_len and (unless its width is 0) table must be 4-byte aligned and not NULL");
    return GPTQ_Q4_OK;
}

int check_ints(const void *p, const char *name) {
    return p && aligned(p, 4) ? GPTQ_Q4_OK
                              : api_failf(GPTQ_Q4_INVALID_ARGUMENT, "%s must be 4-byte aligned and not NULL", name);
}

q4::PageRows rows_view(const gptq_q4_rows *r, int window, int sinks) {
    return q4::PageRows{r->table, r->kv_len, r->table_stride, r->width, r->batch, window, sinks};
}

void release(gptq_q4_pages_s *h) {
    if (!h) return;
    const q4::FreeScope scope(h->device);
    cudaFree(h->view.status);                                  // the first: see FreeScope
    cudaFree(h->chunk);
    cudaFree(h->view.used);
    cudaFree(h->view.rank);
    delete h;
}

}  // namespace

extern "C" {

gptq_q4_pages gptq_q4_pages_make(const gptq_q4_buffer *buffers, int n, int pages, int page_size) {
    if (n < 0 || (n && !buffers) || pages < 1 || pages > 1 << 22 || page_size < 1) {
        api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                  "n=%d must not be negative, buffers not NULL, pages=%d from 1 to 2^22 and page_size=%d positive", n, pages,
                  page_size);
        return nullptr;
    }
    int64_t chunks = 0;
    for (int i = 0; i < n; ++i) {
        const gptq_q4_buffer &b = buffers[i];
        if (!b.data || !aligned(b.data, 16) || b.bytes < 16 || b.bytes % 16 || b.stride < b.bytes || b.stride % 16 ||
            b.stride >= int64_t{1} << 39) {
            api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                      "buffer %d: data must be 16-byte aligned and not NULL, bytes=%lld a positive multiple of 16, "
                      "stride=%lld one at least as large and below 2^39",
                      i, static_cast<long long>(b.bytes), static_cast<long long>(b.stride));
            return nullptr;
        }
        chunks += (b.bytes + q4::kPageChunk - 1) / q4::kPageChunk;
    }
    if (chunks > 1 << 24) {
        api_failf(GPTQ_Q4_INVALID_ARGUMENT, "the buffers hold more than 2^24 parts of 16384 bytes of a page");
        return nullptr;
    }
    int dev = -1;
    if (q4::api_check_device_sm103(&dev)) return nullptr;
    for (int i = 0; i < n; ++i)
        if (q4::api_check_device_ptr(buffers[i].data, dev, "a buffer's data")) return nullptr;
    gptq_q4_pages_s *h = new (std::nothrow) gptq_q4_pages_s();
    q4::PageChunk *host = new (std::nothrow) q4::PageChunk[std::max<int64_t>(chunks, 1)];
    if (!h || !host) {
        delete h;
        delete[] host;
        api_failf(GPTQ_Q4_OUT_OF_MEMORY, "host allocation of the pages handle failed");
        return nullptr;
    }
    int64_t at = 0;
    for (int i = 0; i < n; ++i)
        for (int64_t o = 0; o < buffers[i].bytes; o += q4::kPageChunk)
            host[at++] = q4::PageChunk{static_cast<uint8_t *>(buffers[i].data) + o, buffers[i].stride,
                                       static_cast<int>(std::min<int64_t>(q4::kPageChunk, buffers[i].bytes - o))};
    h->device = dev;
    q4::PagesView &v = h->view;
    v.pages = pages;
    v.page_size = page_size;
    v.chunks = static_cast<int>(chunks);
    v.words = (pages + 127) / 128 * 4;
    v.sms = q4::device_sm_count();
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(&h->chunk), std::max<int64_t>(chunks, 1) * sizeof(q4::PageChunk));
    if (!e) e = cudaMemcpy(h->chunk, host, chunks * sizeof(q4::PageChunk), cudaMemcpyHostToDevice);
    if (!e) e = cudaMalloc(reinterpret_cast<void **>(&v.used), v.words * sizeof(uint32_t));
    if (!e) e = cudaMalloc(reinterpret_cast<void **>(&v.rank), size_t{3} * pages * sizeof(int));
    if (!e) e = cudaMalloc(reinterpret_cast<void **>(&v.status), 2 * sizeof(int));
    if (!e) e = cudaMemset(v.status, 0, 2 * sizeof(int));
    if (!e) e = cudaDeviceSynchronize();
    delete[] host;
    if (e) {
        api_cuda_fail(e, "allocating the pages handle");
        release(h);
        return nullptr;
    }
    v.chunk = h->chunk;
    v.source = v.rank + pages;
    v.hole = v.source + pages;
    v.moves = v.status + 1;
    api_set_status(GPTQ_Q4_OK, nullptr);
    return h;
}

int gptq_q4_pages_free_list(gptq_q4_pages h, const gptq_q4_rows *rows, int window, int sinks, int32_t *ids,
                            int32_t *count, cudaStream_t stream) {
    if (int r = check(h)) return r;
    if (int r = check_rows(rows, window, sinks)) return r;
    if (int r = check_ints(ids, "ids")) return r;
    if (int r = check_ints(count, "count")) return r;
    int launches = 0;
    const cudaError_t e = q4::launch_pages_free_list(h->view, rows_view(rows, window, sinks), ids, count, stream, &launches);
    q4::api_count_launches(launches);
    return e ? api_cuda_fail(e, "free list launch") : api_set_status(GPTQ_Q4_OK, nullptr);
}

int gptq_q4_pages_fork(gptq_q4_pages h, const gptq_q4_rows *rows, const int32_t *parent, const int32_t *child,
                       const int32_t *fresh, int n, cudaStream_t stream) {
    if (int r = check(h)) return r;
    if (int r = check_rows(rows, 0, 0)) return r;
    if (n < 0) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "n=%d must not be negative", n);
    if (n > kMaxForks) return api_failf(GPTQ_Q4_UNSUPPORTED, "n=%d: at most %d forks in a call", n, kMaxForks);
    if (n == 0) return api_set_status(GPTQ_Q4_OK, nullptr);
    if (int r = check_ints(parent, "parent")) return r;
    if (int r = check_ints(child, "child")) return r;
    if (int r = check_ints(fresh, "fresh")) return r;
    if (cudaError_t e = q4::launch_pages_fork(h->view, rows_view(rows, 0, 0), parent, child, fresh, n, stream))
        return api_cuda_fail(e, "fork launch");
    q4::api_count_launches(1);
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

int gptq_q4_pages_copy(gptq_q4_pages h, const int32_t *src, const int32_t *dst, int n, cudaStream_t stream) {
    if (int r = check(h)) return r;
    if (n < 0) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "n=%d must not be negative", n);
    if (n == 0 || h->view.chunks == 0) return api_set_status(GPTQ_Q4_OK, nullptr);
    if (int r = check_ints(src, "src")) return r;
    if (int r = check_ints(dst, "dst")) return r;
    if (cudaError_t e = q4::launch_pages_copy(h->view, src, dst, n, stream)) return api_cuda_fail(e, "copy launch");
    q4::api_count_launches(1);
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

int gptq_q4_pages_compact(gptq_q4_pages h, const gptq_q4_rows *rows, int window, int sinks, int32_t *table_out,
                          int64_t out_stride, int32_t *count, cudaStream_t stream) {
    if (int r = check(h)) return r;
    if (int r = check_rows(rows, window, sinks)) return r;
    if (out_stride < rows->width || (table_out == rows->table && out_stride != rows->table_stride))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "out_stride=%lld must be at least width=%d, and table_stride=%lld in place",
                         static_cast<long long>(out_stride), rows->width, static_cast<long long>(rows->table_stride));
    if (rows->batch && rows->width)
        if (int r = check_ints(table_out, "table_out")) return r;
    if (int r = check_ints(count, "count")) return r;
    int launches = 0;
    const cudaError_t e = q4::launch_pages_compact(h->view, rows_view(rows, window, sinks), table_out, out_stride, count,
                                                   stream, &launches);
    q4::api_count_launches(launches);
    return e ? api_cuda_fail(e, "compaction launch") : api_set_status(GPTQ_Q4_OK, nullptr);
}

int gptq_q4_pages_device_error(gptq_q4_pages h) {
    if (int r = check(h)) return r;
    int flag = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (!e) e = cudaMemcpy(&flag, h->view.status, sizeof(int), cudaMemcpyDeviceToHost);
    if (!e && flag) e = cudaMemset(h->view.status, 0, sizeof(int));
    if (e) return api_cuda_fail(e, "reading the pages handle's status word");
    if (flag)
        return api_failf(GPTQ_Q4_DEVICE_FAULT, "page kernels reported status 0x%x:%s%s", flag,
                         flag & q4::kPagesBadIndex ? " a page number past the last page;" : "",
                         flag & q4::kPagesBadFork ? " a fork that was left out;" : "");
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

void gptq_q4_pages_free(gptq_q4_pages h) {
    release(h);
    api_set_status(GPTQ_Q4_OK, nullptr);
}

}  // extern "C"
