// Handles and launchers of the operators around the projection: the adapter
// pool (q4_lora*.cu) and paged attention with its cache append (q4_attn*.cu).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <type_traits>

#include "../../include/gptq_q4.h"

namespace q4 {

// One adapter of a pool, as the kernels read it.
struct LoraSlot {
    int rank;        // of the adapter; 0: empty
    float scale;
    int finite;      // no infinity or NaN in B
};

// Status bits of the two handles.
constexpr int kLoraBadSlot = 0x1;      // row_slot entry >= slots
constexpr int kLoraTimeout = 0x2;      // a bounded wait ran out
constexpr int kAttnBadBatch = 0x1;     // a length outside its range, or cu_q not ascending
constexpr int kAttnBadPage = 0x2;      // a page index outside the cache
constexpr int kAttnBadPosition = 0x4;  // a position outside the rotary table
constexpr int kAttnTimeout = 0x8;      // a bounded wait ran out
constexpr int kAttnTooLong = 0x10;     // 2^31 or more units of work in a call

constexpr int ceil16(int r) { return (r + 15) / 16 * 16; }
constexpr int ceil64(int k) { return (k + 63) / 64 * 64; }

struct LoraView {
    int K, N, slots, rpad;       // rpad: ceil16(max_rank)
    const uint16_t *a;           // [slots][rpad * ceil64(K)], layout in q4_lora.cu
    const uint16_t *b;           // [slots][rpad * N]
    const LoraSlot *slot;        // [slots]
    float *t;                    // [rows][rpad] fp32: scale * x . A^T; and room for two more each row
    int *status;
};

struct LoraCall {
    const uint16_t *x, *y;
    uint16_t *out;
    const int32_t *row_slot;
    int64_t xs, ys, os;
    int M;
    int chunk;                   // rows that a CTA of the few-row kernels looks over
    int *marks;                  // [chunks] or NULL: only the chunks that are marked
};

cudaError_t launch_lora_set(const LoraView &v, uint16_t *a, uint16_t *b, LoraSlot *slot, int s, const uint16_t *src_a,
                            const uint16_t *src_b, int rank, float scale, bool bf16, cudaStream_t st);
// few rows, and ranks over 176 (q4_lora.cu)
cudaError_t launch_lora_add(const LoraView &v, const LoraCall &c, bool bf16, cudaStream_t st, int *launches);
// the marked chunks of c.chunk rows
cudaError_t launch_lora_marked(const LoraView &v, const LoraCall &c, bool bf16, cudaStream_t st, int *launches);
// many rows (q4_lora_tc.cu); marks the tiles of 128 rows whose adapters have too many ranks, which it leaves out
struct LoraTcPlan {
    bool ok, marks;              // whether there can be marked tiles
    int tiles, parts, blocks_each;
};
LoraTcPlan plan_lora_tc(const LoraView &v, int M, int sms);
cudaError_t launch_lora_tc(const LoraView &v, const LoraCall &c, const LoraTcPlan &p, int sms, bool bf16,
                           cudaStream_t st, int *launches);

// The step's requests and one layer's cache, as the kernels read them.
struct AttnBatch {
    const int32_t *cu_q, *kv_len, *table;
    int64_t table_stride;
    int width, batch, tokens;
};
struct AttnCache {
    uint16_t *k, *v;
    int pages;
    int64_t page_stride;
};
struct AttnShape {
    int hq, hkv, group, d, page, page_log2;
};

struct AppendCall {
    const uint16_t *qkv;
    uint16_t *q_out;
    int64_t qkv_stride, q_stride;
    const int32_t *positions;
    const float2 *rope;          // [max_pos][rot / 2] (cos, sin), NULL: no rotation
    int rot, interleaved, max_pos;
    int *status;
};
cudaError_t launch_rope_table(float2 *table, const double *inv_freq, double length_scale, int half, int max_pos,
                              cudaStream_t st);
cudaError_t launch_attn_append(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AppendCall &a,
                               bool bf16, cudaStream_t st);

// A cache of 4 bits (q4_cache4.cuh).
struct Cache4;
cudaError_t launch_attn_append4(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AppendCall &a, bool bf16,
                                cudaStream_t st);
// The step's new tokens out of either cache (the other one is NULL).
cudaError_t launch_attn_read(const AttnShape &s, const AttnBatch &b, const AttnCache *c, const Cache4 *c4, uint16_t *k,
                             int64_t k_stride, uint16_t *v, int64_t v_stride, bool bf16, int *status, cudaStream_t st);

struct AttendCall {
    const uint16_t *q;
    uint16_t *out;
    int64_t q_stride, out_stride;
    float scale;
    int window;
    int sinks;                   // first tokens seen besides the window; 0 without one
    int max_q;
    int *status;
    float *ws;                   // pieces of cut items
    int *tickets;                // [4 * ctas], zero between calls
    int ctas;                    // one for each SM
    uint32_t *allowed;           // kernels of this handle that have their shared memory (host)
};
// few rows for each key/value head (q4_attn_stream.cu)
size_t attend_stream_ws_bytes(int ctas);
cudaError_t launch_attend_stream(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a,
                                 bool bf16, cudaStream_t st);
// chunks (q4_attn_tc.cu); scale > 0
size_t attend_tc_ws_bytes(int ctas);
cudaError_t launch_attend_tc(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a, bool bf16,
                             cudaStream_t st);
// few rows over a cache of 4 bits (q4_attn_stream4.cu); pieces as launch_attend_tc's
cudaError_t launch_attend_stream4(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                                  cudaStream_t st);
// chunks over a cache of 4 bits; scale > 0
cudaError_t launch_attend_tc4_64(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                                 cudaStream_t st);
cudaError_t launch_attend_tc4_128(const AttnShape &s, const AttnBatch &b, const Cache4 &c, const AttendCall &a, bool bf16,
                                  cudaStream_t st);
// with a window and first tokens that stay visible
cudaError_t launch_attend_stream_sinks(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a,
                                       bool bf16, cudaStream_t st);
cudaError_t launch_attend_tc_sinks(const AttnShape &s, const AttnBatch &b, const AttnCache &c, const AttendCall &a,
                                   bool bf16, cudaStream_t st);
// Tensor map of the queries [tokens][heads][d]: boxes of 64 columns, a
// group's heads and `rows` tokens.
cudaError_t encode_queries(CUtensorMap *map, const void *ptr, const AttnShape &s, int64_t stride, int tokens,
                           uint32_t rows);
// Tensor map of a cache's keys or values [pages][heads][page][d]: boxes of
// 64 columns (128 bytes, swizzled) and `rows` tokens (q4_gemm_tc.cu).
cudaError_t encode_pages(CUtensorMap *map, const void *ptr, const AttnShape &s, const AttnCache &c, uint32_t rows);

// Lets `kernel` have `bytes` of dynamic shared memory, once for a handle: the call costs a small launch's host time
// again.  allowed: the handle's, a bit for each kernel that it may launch.
enum AttnKernel { kStream, kStreamSinks, kChunk, kChunkSinks, kStream4, kChunk4 = kStream4 + 2 };     // (two of groups each)
inline cudaError_t allow_smem(const void *kernel, int bytes, uint32_t *allowed, int bit) {
    if (*allowed >> bit & 1) return cudaSuccess;
    if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
    *allowed |= 1u << bit;
    return cudaSuccess;
}

// ------------------------------------------------------------ device helpers
template <bool BF>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if constexpr (BF) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&v));
    else return __half22float2(*reinterpret_cast<__half2 *>(&v));
}
template <bool BF>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    if constexpr (BF) {
        __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&r);
    } else {
        __half2 r = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t *>(&r);
    }
}

// A request's rows and context length, cut to their ranges: 0 <= q0,
// q0 + ql <= tokens, 0 <= kv <= width * page and 2^30.  bad: something had to be cut.
struct Request {
    int q0, ql, kv;
    bool bad;
};
__device__ __forceinline__ Request load_request(const AttnBatch &b, int i, int page_log2) {
    const int a = b.cu_q[i], e = b.cu_q[i + 1], n = b.kv_len[i];
    const long long cap = min(static_cast<long long>(b.width) << page_log2, 1ll << 30);
    Request r;
    r.q0 = min(max(a, 0), b.tokens);
    r.ql = max(min(e, b.tokens), r.q0) - r.q0;           // (any cu_q: the difference stays within the rows)
    r.kv = static_cast<int>(min(static_cast<long long>(max(n, 0)), cap));
    r.bad = r.q0 != a || r.q0 + r.ql != e || r.kv != n;
    return r;
}

}  // namespace q4
