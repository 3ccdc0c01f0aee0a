// C ABI of rotary positions, the paged cache and attention over it
// (gptq_q4_attn_*): argument checks and the handle's memory.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>
#include <type_traits>

#include "q4_cache4.cuh"
#include "q4_handle.h"
#include "q4_serve.h"

struct gptq_q4_attn_s {
    int device = -1;
    int dtype = 0;
    q4::AttnShape shape{};
    int rot = 0, interleaved = 0, max_pos = 0;
    float2 *rope = nullptr;
    q4::Retired retired;
    int *status = nullptr;
    float *ws = nullptr;
    int *tickets = nullptr;
    int ctas = 0;
    uint32_t allowed = 0;
};

namespace {

using q4::api_cuda_fail;
using q4::api_failf;
using q4::api_set_status;

constexpr int kMaxBatch = 4096;

int check(gptq_q4_attn h) {
    if (!h) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "attention handle is NULL");
    int dev = -1;
    if (cudaError_t e = cudaGetDevice(&dev)) return api_cuda_fail(e, "cudaGetDevice");
    if (dev != h->device)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "the attention handle was made on device %d, current device is %d",
                         h->device, dev);
    return GPTQ_Q4_OK;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool aligned4(const void *p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

bool empty(const gptq_q4_batch *b) { return b->batch == 0 || b->tokens == 0; }

int check_batch(const void *c, const gptq_q4_batch *b) {
    if (!c || !b) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "cache and batch must not be NULL");
    if (b->batch < 0 || b->tokens < 0 || b->width < 0 || b->max_q < 0 || b->table_stride < b->width)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "batch=%d, tokens=%d, width=%d and max_q=%d must not be negative, nor table_stride=%lld "
                         "below width",
                         b->batch, b->tokens, b->width, b->max_q, static_cast<long long>(b->table_stride));
    if (b->batch > kMaxBatch)
        return api_failf(GPTQ_Q4_UNSUPPORTED, "batch=%d: at most %d requests in a call", b->batch, kMaxBatch);
    if (empty(b)) return GPTQ_Q4_OK;
    if (!b->cu_q || !b->kv_len || (b->width && !b->table) || !aligned4(b->cu_q) || !aligned4(b->kv_len) ||
        !aligned4(b->table))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "cu_q, kv_len and (unless its width is 0) table must be 4-byte aligned and not NULL");
    return GPTQ_Q4_OK;
}

int check_step(const gptq_q4_attn_s *h, const gptq_q4_cache *c, const gptq_q4_batch *b) {
    if (int r = check_batch(c, b)) return r;
    if (empty(b)) return GPTQ_Q4_OK;
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "the cache's k and v must be 16-byte aligned and not NULL");
    const int64_t page = static_cast<int64_t>(h->shape.hkv) * h->shape.page * h->shape.d;
    if (c->pages < 1 || c->page_stride < page || c->page_stride % 8 || c->page_stride >= int64_t{1} << 39)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "pages=%d must be positive and page_stride=%lld a multiple of 8, at least %lld and below 2^39",
                         c->pages, static_cast<long long>(c->page_stride), static_cast<long long>(page));
    return GPTQ_Q4_OK;
}

int check_step(const gptq_q4_attn_s *h, const gptq_q4_cache4 *c, const gptq_q4_batch *b) {
    if (int r = check_batch(c, b)) return r;
    if (empty(b)) return GPTQ_Q4_OK;
    if (c->group != 32 && c->group != 64)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "group=%d must be 32 or 64", c->group);
    if (!c->kv || !aligned16(c->kv))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "the cache's kv must be 16-byte aligned and not NULL");
    const int64_t page = static_cast<int64_t>(h->shape.hkv) * h->shape.page *
                         q4::record_bytes(h->shape.d, c->group == 32 ? 5 : 6);
    if (c->pages < 1 || c->page_stride < page || c->page_stride % 16 || c->page_stride >= int64_t{1} << 39)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "pages=%d must be positive and page_stride=%lld a multiple of 16, at least %lld and below 2^39",
                         c->pages, static_cast<long long>(c->page_stride), static_cast<long long>(page));
    return GPTQ_Q4_OK;
}

q4::AttnBatch batch_view(const gptq_q4_batch *b) {
    return q4::AttnBatch{b->cu_q, b->kv_len, b->table, b->table_stride, b->width, b->batch, b->tokens};
}
q4::AttnCache cache_view(const gptq_q4_cache *c) {
    return q4::AttnCache{static_cast<uint16_t *>(c->k), static_cast<uint16_t *>(c->v), c->pages, c->page_stride};
}
q4::Cache4 cache_view(const gptq_q4_cache4 *c) {
    return q4::Cache4{static_cast<uint8_t *>(c->kv), c->pages, c->page_stride, c->group == 32 ? 5 : 6};
}

void release(gptq_q4_attn_s *h) {
    if (!h) return;
    const q4::FreeScope scope(h->device);
    cudaFree(h->status);                                  // the first: see FreeScope
    cudaFree(h->rope);
    q4::api_free_retired(h->retired);
    cudaFree(h->ws);
    cudaFree(h->tickets);
    delete h;
}

// For either cache.
template <class Cache>
int append(gptq_q4_attn h, const void *qkv, int64_t qkv_stride, const Cache *cache, const gptq_q4_batch *batch,
           const int32_t *positions, void *q_out, int64_t q_stride, cudaStream_t stream) {
    if (int r = check(h)) return r;
    if (int r = check_step(h, cache, batch)) return r;
    if (empty(batch)) return api_set_status(GPTQ_Q4_OK, nullptr);
    const q4::AttnShape &s = h->shape;
    if (!qkv || !q_out || !aligned16(qkv) || !aligned16(q_out) || !aligned4(positions))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "qkv and q_out must be 16-byte aligned and not NULL, positions 4-byte aligned");
    const int64_t row = static_cast<int64_t>(s.hq + 2 * s.hkv) * s.d, qrow = static_cast<int64_t>(s.hq) * s.d;
    if (qkv_stride < row || qkv_stride % 8 || q_stride < qrow || q_stride % 8)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "row strides (qkv %lld, q %lld) must be multiples of 8 and at least %lld and %lld",
                         static_cast<long long>(qkv_stride), static_cast<long long>(q_stride),
                         static_cast<long long>(row), static_cast<long long>(qrow));
    if (q_out == qkv && q_stride != qkv_stride)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "q_out is qkv but their row strides differ (%lld and %lld)",
                         static_cast<long long>(q_stride), static_cast<long long>(qkv_stride));
    const q4::AppendCall a{static_cast<const uint16_t *>(qkv), static_cast<uint16_t *>(q_out), qkv_stride, q_stride,
                           positions, h->rope, h->rot, h->interleaved, h->max_pos, h->status};
    cudaError_t e;
    if constexpr (std::is_same_v<Cache, gptq_q4_cache>)
        e = q4::launch_attn_append(s, batch_view(batch), cache_view(cache), a, h->dtype == GPTQ_Q4_DTYPE_BF16, stream);
    else
        e = q4::launch_attn_append4(s, batch_view(batch), cache_view(cache), a, h->dtype == GPTQ_Q4_DTYPE_BF16, stream);
    if (e) return api_cuda_fail(e, "append launch");
    q4::api_count_launches(1);
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

template <class Cache>
int read(gptq_q4_attn h, const Cache *cache, const gptq_q4_batch *batch, void *k_out, int64_t k_stride, void *v_out,
         int64_t v_stride, cudaStream_t stream) {
    if (int r = check(h)) return r;
    if (int r = check_step(h, cache, batch)) return r;
    if (empty(batch)) return api_set_status(GPTQ_Q4_OK, nullptr);
    const q4::AttnShape &s = h->shape;
    const int64_t row = static_cast<int64_t>(s.hkv) * s.d;
    if (!k_out || !v_out || !aligned16(k_out) || !aligned16(v_out) || k_stride < row || k_stride % 8 || v_stride < row ||
        v_stride % 8)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "k_out and v_out must be 16-byte aligned and not NULL, their row strides (%lld and %lld) "
                         "multiples of 8 and at least %lld",
                         static_cast<long long>(k_stride), static_cast<long long>(v_stride), static_cast<long long>(row));
    const auto view = cache_view(cache);
    const q4::AttnCache *wide = nullptr;
    const q4::Cache4 *four = nullptr;
    if constexpr (std::is_same_v<Cache, gptq_q4_cache>) wide = &view;
    else four = &view;
    if (cudaError_t e = q4::launch_attn_read(s, batch_view(batch), wide, four, static_cast<uint16_t *>(k_out), k_stride,
                                             static_cast<uint16_t *>(v_out), v_stride, h->dtype == GPTQ_Q4_DTYPE_BF16,
                                             h->status, stream))
        return api_cuda_fail(e, "read launch");
    q4::api_count_launches(1);
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

template <class Cache>
int attend(gptq_q4_attn h, const void *q, int64_t q_stride, const Cache *cache, const gptq_q4_batch *batch, float scale,
           int window, int sinks, void *out, int64_t out_stride, cudaStream_t stream) {
    if (int r = check(h)) return r;
    if (int r = check_step(h, cache, batch)) return r;
    if (!std::isfinite(scale) || window < 0 || sinks < 0)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "scale=%g must be finite, window=%d and sinks=%d not negative",
                         static_cast<double>(scale), window, sinks);
    if (empty(batch)) return api_set_status(GPTQ_Q4_OK, nullptr);
    const q4::AttnShape &s = h->shape;
    if (!q || !out || !aligned16(q) || !aligned16(out))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "q and out must be 16-byte aligned and not NULL");
    const int64_t row = static_cast<int64_t>(s.hq) * s.d;
    if (q_stride < row || q_stride % 8 || out_stride < row || out_stride % 8 ||
        q_stride >= int64_t{1} << 39)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "row strides (q %lld, out %lld) must be multiples of 8, at least %lld and below 2^39",
                         static_cast<long long>(q_stride), static_cast<long long>(out_stride),
                         static_cast<long long>(row));
    // Contexts end at 2^30 tokens, so a longer window hides nothing; differences with a shorter one fit 32 bits.
    const int seen = window < 1 << 30 ? window : 0;
    const q4::AttendCall a{static_cast<const uint16_t *>(q), static_cast<uint16_t *>(out), q_stride, out_stride,
                           scale, seen, seen ? std::min(sinks, 1 << 30) : 0, batch->max_q, h->status, h->ws, h->tickets, h->ctas,
                           &h->allowed};
    // More query rows for each key/value head than the streaming kernel's row tile has: the tensor-core kernel
    // (which takes its maximum before scaling, so a positive scale).  Measured at 64 heads over 8, contexts of up
    // to 4096: 32 requests of 2 tokens (16 rows) 45 us streaming, 53 on tcgen05, one such request 12 and 15; 32 of 4
    // tokens, streaming with row tiles of 32 rows 134, tcgen05 54; one request of 4 tokens 25 and 17.  Over a cache of
    // 4 bits, whose streaming kernel has tiles of 8 rows, the same: 2 tokens 55 streaming and 80, 4 tokens 96 and 82.
    const bool chunk = static_cast<int64_t>(batch->max_q) * s.group > 16 && scale > 0.f;
    const bool bf16 = h->dtype == GPTQ_Q4_DTYPE_BF16;
    cudaError_t e;
    if constexpr (std::is_same_v<Cache, gptq_q4_cache>) {
        const auto tc = a.sinks ? q4::launch_attend_tc_sinks : q4::launch_attend_tc;
        const auto stream_kv = a.sinks ? q4::launch_attend_stream_sinks : q4::launch_attend_stream;
        e = (chunk ? tc : stream_kv)(s, batch_view(batch), cache_view(cache), a, bf16, stream);
    } else {
        const auto tc = s.d == 64 ? q4::launch_attend_tc4_64 : q4::launch_attend_tc4_128;
        e = (chunk ? tc : q4::launch_attend_stream4)(s, batch_view(batch), cache_view(cache), a, bf16, stream);
    }
    if (e) return api_cuda_fail(e, "attention launch");
    q4::api_count_launches(1);
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

}  // namespace

extern "C" {

gptq_q4_attn gptq_q4_attn_make(int q_heads, int kv_heads, int head_dim, int page_size, int dtype) {
    if (q_heads < 1 || kv_heads < 1 || q_heads % kv_heads || q_heads / kv_heads > 128 || q_heads > 65536) {
        api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                  "q_heads=%d must be a positive multiple of kv_heads=%d, at most 128 for each", q_heads, kv_heads);
        return nullptr;
    }
    if (dtype != GPTQ_Q4_DTYPE_FP16 && dtype != GPTQ_Q4_DTYPE_BF16 && dtype != GPTQ_Q4_DTYPE_FP32) {
        api_failf(GPTQ_Q4_INVALID_ARGUMENT, "dtype=%d is neither GPTQ_Q4_DTYPE_FP16 nor GPTQ_Q4_DTYPE_BF16", dtype);
        return nullptr;
    }
    int log2 = 0;
    while (log2 < 10 && (1 << log2) != page_size) ++log2;
    if ((head_dim != 64 && head_dim != 128) || page_size < 8 || (1 << log2) != page_size ||
        dtype == GPTQ_Q4_DTYPE_FP32) {
        api_failf(GPTQ_Q4_UNSUPPORTED,
                  "head_dim=%d must be 64 or 128, page_size=%d a power of two from 8 to 1024, and dtype=%d 16 bits wide",
                  head_dim, page_size, dtype);
        return nullptr;
    }
    int dev = -1;
    if (q4::api_check_device_sm103(&dev)) return nullptr;
    gptq_q4_attn_s *h = new (std::nothrow) gptq_q4_attn_s();
    if (!h) {
        api_failf(GPTQ_Q4_OUT_OF_MEMORY, "host allocation of the attention handle failed");
        return nullptr;
    }
    h->device = dev;
    h->dtype = dtype;
    h->shape = q4::AttnShape{q_heads, kv_heads, q_heads / kv_heads, head_dim, page_size, log2};
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(&h->status), sizeof(int));
    if (!e) e = cudaMemset(h->status, 0, sizeof(int));
    h->ctas = q4::device_sm_count();
    if (!e) e = cudaMalloc(reinterpret_cast<void **>(&h->ws), std::max(q4::attend_stream_ws_bytes(h->ctas), q4::attend_tc_ws_bytes(h->ctas)));
    if (!e) e = cudaMalloc(reinterpret_cast<void **>(&h->tickets), 4 * h->ctas * sizeof(int));
    if (!e) e = cudaMemset(h->tickets, 0, 4 * h->ctas * sizeof(int));
    if (!e) e = cudaDeviceSynchronize();
    if (e) {
        api_cuda_fail(e, "allocating the attention handle");
        release(h);
        return nullptr;
    }
    api_set_status(GPTQ_Q4_OK, nullptr);
    return h;
}

int gptq_q4_rope_freqs(int rotary_dim, double base, int kind, double factor, double low, double high, int original,
                       double *inv_freq, double *length_scale) {
    if (!inv_freq || !length_scale) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "inv_freq and length_scale are NULL");
    if (rotary_dim < 2 || rotary_dim % 2 || !(base > 1.0) || !std::isfinite(base))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "rotary_dim=%d must be positive and even, base=%g above 1",
                         rotary_dim, base);
    if (kind < GPTQ_Q4_ROPE_PLAIN || kind > GPTQ_Q4_ROPE_YARN)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "kind=%d is none of GPTQ_Q4_ROPE_*", kind);
    if (kind != GPTQ_Q4_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "factor=%g must be at least 1", factor);
    if (kind == GPTQ_Q4_ROPE_NTK && rotary_dim == 2)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "GPTQ_Q4_ROPE_NTK needs rotary_dim above 2");
    if (kind >= GPTQ_Q4_ROPE_BANDS &&
        (!(low > 0.0) || !(high > low) || !std::isfinite(high) || original < 1))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "0 < low=%g < high=%g and original=%d >= 1 are wanted", low, high,
                         original);
    const double two_pi = 6.283185307179586476925;
    if (kind == GPTQ_Q4_ROPE_NTK) base *= std::pow(factor, rotary_dim / (rotary_dim - 2.0));
    auto pair_of = [&](double turns) { return rotary_dim * std::log(original / (two_pi * turns)) / (2.0 * std::log(base)); };
    double first = 0, last = 0;
    if (kind == GPTQ_Q4_ROPE_YARN) {
        first = std::fmax(std::floor(pair_of(high)), 0.0);
        last = std::fmin(std::ceil(pair_of(low)), rotary_dim - 1.0);
    }
    for (int i = 0; i < rotary_dim / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / rotary_dim);
        double s = 1.0;                     // share of the unscaled angle
        if (kind == GPTQ_Q4_ROPE_LINEAR) s = 0.0;
        if (kind == GPTQ_Q4_ROPE_BANDS) s = (original * f / two_pi - low) / (high - low);
        if (kind == GPTQ_Q4_ROPE_YARN) s = 1.0 - (i - first) / std::fmax(last - first, 0.001);
        s = std::fmin(std::fmax(s, 0.0), 1.0);
        const bool blends = kind != GPTQ_Q4_ROPE_PLAIN && kind != GPTQ_Q4_ROPE_NTK;
        inv_freq[i] = blends ? s * f + (1.0 - s) * f / factor : f;
    }
    *length_scale = kind == GPTQ_Q4_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

int gptq_q4_attn_set_rope(gptq_q4_attn h, int rotary_dim, int interleaved, const double *inv_freq,
                          double length_scale, int max_pos) {
    if (int r = check(h)) return r;
    if (rotary_dim < 0 || rotary_dim > h->shape.d || rotary_dim % 16)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "rotary_dim=%d must be a multiple of 16, at most head_dim=%d",
                         rotary_dim, h->shape.d);
    if (rotary_dim && (!inv_freq || max_pos < 1 || !std::isfinite(length_scale)))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "inv_freq must not be NULL, max_pos=%d positive and length_scale finite", max_pos);
    for (int i = 0; i < rotary_dim / 2; ++i)
        if (!std::isfinite(inv_freq[i])) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "inv_freq[%d] is not finite", i);
    if (cudaError_t e = cudaDeviceSynchronize()) return api_cuda_fail(e, "set_rope");
    // A captured append holds the table's address, so the table is written anew only where all else that such a call
    // holds stays true, and otherwise kept beside the next one.
    const bool same = h->rope && rotary_dim == h->rot && max_pos == h->max_pos && (interleaved != 0) == (h->interleaved != 0);
    void *table = same ? h->rope : nullptr;
    if (rotary_dim) {
        const size_t bytes = static_cast<size_t>(max_pos) * (rotary_dim / 2) * sizeof(float2);
        if (!same)
            if (cudaError_t e = cudaMalloc(&table, bytes)) return api_cuda_fail(e, "allocating the rotary table");
        cudaError_t e = q4::launch_rope_table(static_cast<float2 *>(table), inv_freq, length_scale, rotary_dim / 2,
                                              max_pos, nullptr);
        if (!e) e = cudaDeviceSynchronize();
        if (e) {
            if (!same) cudaFree(table);
            return api_cuda_fail(e, "building the rotary table");
        }
        q4::api_count_launches(1);
    }
    if (!same && !q4::api_retire(h->retired, h->rope)) {
        cudaFree(table);
        return api_failf(GPTQ_Q4_OUT_OF_MEMORY, "host allocation for the rotary table failed");
    }
    h->rope = static_cast<float2 *>(table);
    h->rot = rotary_dim;
    h->interleaved = interleaved ? 1 : 0;
    h->max_pos = rotary_dim ? max_pos : 0;
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

int gptq_q4_attn_append(gptq_q4_attn h, const void *qkv, int64_t qkv_stride, const gptq_q4_cache *cache,
                        const gptq_q4_batch *batch, const int32_t *positions, void *q_out, int64_t q_stride,
                        cudaStream_t stream) {
    return append(h, qkv, qkv_stride, cache, batch, positions, q_out, q_stride, stream);
}

int gptq_q4_attn_append4(gptq_q4_attn h, const void *qkv, int64_t qkv_stride, const gptq_q4_cache4 *cache,
                         const gptq_q4_batch *batch, const int32_t *positions, void *q_out, int64_t q_stride,
                         cudaStream_t stream) {
    return append(h, qkv, qkv_stride, cache, batch, positions, q_out, q_stride, stream);
}

int gptq_q4_attn_read(gptq_q4_attn h, const gptq_q4_cache *cache, const gptq_q4_batch *batch, void *k_out,
                      int64_t k_stride, void *v_out, int64_t v_stride, cudaStream_t stream) {
    return read(h, cache, batch, k_out, k_stride, v_out, v_stride, stream);
}

int gptq_q4_attn_read4(gptq_q4_attn h, const gptq_q4_cache4 *cache, const gptq_q4_batch *batch, void *k_out,
                       int64_t k_stride, void *v_out, int64_t v_stride, cudaStream_t stream) {
    return read(h, cache, batch, k_out, k_stride, v_out, v_stride, stream);
}

int gptq_q4_attn_attend(gptq_q4_attn h, const void *q, int64_t q_stride, const gptq_q4_cache *cache,
                        const gptq_q4_batch *batch, float scale, int window, void *out, int64_t out_stride,
                        cudaStream_t stream) {
    return attend(h, q, q_stride, cache, batch, scale, window, 0, out, out_stride, stream);
}

int gptq_q4_attn_attend_sinks(gptq_q4_attn h, const void *q, int64_t q_stride, const gptq_q4_cache *cache,
                              const gptq_q4_batch *batch, float scale, int window, int sinks, void *out,
                              int64_t out_stride, cudaStream_t stream) {
    return attend(h, q, q_stride, cache, batch, scale, window, sinks, out, out_stride, stream);
}

int gptq_q4_attn_attend4(gptq_q4_attn h, const void *q, int64_t q_stride, const gptq_q4_cache4 *cache,
                         const gptq_q4_batch *batch, float scale, int window, int sinks, void *out,
                         int64_t out_stride, cudaStream_t stream) {
    return attend(h, q, q_stride, cache, batch, scale, window, sinks, out, out_stride, stream);
}

int gptq_q4_attn_device_error(gptq_q4_attn h) {
    if (int r = check(h)) return r;
    int flag = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (!e) e = cudaMemcpy(&flag, h->status, sizeof(int), cudaMemcpyDeviceToHost);
    if (!e && flag) e = cudaMemset(h->status, 0, sizeof(int));
    // a kernel that gave up may have left pieces uncounted
    if (!e && (flag & q4::kAttnTimeout)) e = cudaMemset(h->tickets, 0, 4 * h->ctas * sizeof(int));
    if (e) return api_cuda_fail(e, "reading the attention handle's status word");
    if (flag)
        return api_failf(GPTQ_Q4_DEVICE_FAULT, "attention kernels reported status 0x%x:%s%s%s%s%s", flag,
                         flag & q4::kAttnBadBatch ? " a length or row range outside its limits;" : "",
                         flag & q4::kAttnBadPage ? " a page index outside the cache;" : "",
                         flag & q4::kAttnBadPosition ? " a position outside the rotary table;" : "",
                         flag & q4::kAttnTimeout ? " a bounded wait ran out;" : "",
                         flag & q4::kAttnTooLong ? " more work than one call can count;" : "");
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

void gptq_q4_attn_free(gptq_q4_attn h) {
    release(h);
    api_set_status(GPTQ_Q4_OK, nullptr);
}

}  // extern "C"
