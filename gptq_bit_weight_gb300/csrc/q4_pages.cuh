// The pages of a cache: what the kernels of q4_pages.cu work on.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/gptq_q4.h"

namespace q4 {

constexpr int kPagesBadIndex = 0x1;      // a page number past the last page
constexpr int kPagesBadFork = 0x2;       // a fork that was left out
constexpr int kPageChunk = 16384;        // bytes that a CTA copies at a time

// A part of a page in one buffer.
struct PageChunk {
    uint8_t *data;
    int64_t stride;
    int bytes;
};

struct PagesView {
    int pages, page_size, chunks;
    const PageChunk *chunk;      // [chunks]: all of a page, in all buffers
    uint32_t *used;              // [words]: one bit a page, 128-byte aligned
    int *rank, *source, *hole;   // [pages] each, of a compaction
    int *status, *moves;
    int words;                   // of `used`, a multiple of 4
    int sms;
};

struct PageRows {
    int32_t *table, *kv_len;
    int64_t stride;
    int width, batch, window, sinks;
};

cudaError_t launch_pages_free_list(const PagesView &v, const PageRows &r, int32_t *ids, int32_t *count, cudaStream_t st,
                                   int *launches);
cudaError_t launch_pages_fork(const PagesView &v, const PageRows &r, const int32_t *parent, const int32_t *child,
                              const int32_t *fresh, int n, cudaStream_t st);
cudaError_t launch_pages_copy(const PagesView &v, const int32_t *src, const int32_t *dst, int n, cudaStream_t st);
cudaError_t launch_pages_compact(const PagesView &v, const PageRows &r, int32_t *out, int64_t out_stride, int32_t *count,
                                 cudaStream_t st, int *launches);

}  // namespace q4
