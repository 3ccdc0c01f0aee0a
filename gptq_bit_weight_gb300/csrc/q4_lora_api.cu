// C ABI of the adapter pool (gptq_q4_lora_*): argument checks, the pool's
// memory and its workspace.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <new>

#include "q4_handle.h"
#include "q4_serve.h"

struct gptq_q4_lora_s {
    int device = -1;
    int K = 0, N = 0, slots = 0, max_rank = 0, dtype = 0;
    uint16_t *a = nullptr, *b = nullptr;
    q4::LoraSlot *slot = nullptr;
    int *status = nullptr;
    void *t = nullptr;           // workspace of t_bytes
    size_t t_bytes = 0;
    q4::Retired retired;
    int sms = 0;
};

namespace {

using q4::api_cuda_fail;
using q4::api_failf;
using q4::api_set_status;

int check(gptq_q4_lora h) {
    if (!h) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "adapter pool is NULL");
    int dev = -1;
    if (cudaError_t e = cudaGetDevice(&dev)) return api_cuda_fail(e, "cudaGetDevice");
    if (dev != h->device)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "the pool was made on device %d, current device is %d", h->device,
                         dev);
    return GPTQ_Q4_OK;
}

void release(gptq_q4_lora_s *h) {
    if (!h) return;
    int cur = -1;
    cudaGetDevice(&cur);
    if (h->device >= 0) cudaSetDevice(h->device);
    cudaDeviceSynchronize();
    cudaFree(h->a);
    cudaFree(h->b);
    cudaFree(h->slot);
    cudaFree(h->status);
    cudaFree(h->t);
    q4::api_free_retired(h->retired);
    if (cur >= 0) cudaSetDevice(cur);
    delete h;
}

q4::LoraView view(const gptq_q4_lora_s *h) {
    return q4::LoraView{h->K, h->N, h->slots, q4::ceil16(h->max_rank), h->a, h->b, h->slot,
                        static_cast<float *>(h->t), h->status};
}

int ensure_rows(gptq_q4_lora_s *h, size_t rows, cudaStream_t s, bool sync_alloc) {
    const size_t need = rows * (q4::ceil16(h->max_rank) + 2) * sizeof(float);
    if (need <= h->t_bytes) return GPTQ_Q4_OK;
    if (cudaError_t e = q4::api_replace(h->retired, &h->t, &h->t_bytes, need, s, sync_alloc))
        return api_cuda_fail(e, "allocating the adapter workspace");
    return GPTQ_Q4_OK;
}

bool aligned16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

extern "C" {

gptq_q4_lora gptq_q4_lora_make(int K, int N, int slots, int max_rank, int dtype) {
    if (K <= 0 || N <= 0 || K % 8 || N % 8) {
        api_failf(GPTQ_Q4_INVALID_ARGUMENT, "K=%d and N=%d must be positive multiples of 8", K, N);
        return nullptr;
    }
    if (slots < 1 || slots > 4096 || max_rank < 1 || max_rank > 256) {
        api_failf(GPTQ_Q4_INVALID_ARGUMENT, "slots=%d must be in [1, 4096] and max_rank=%d in [1, 256]", slots,
                  max_rank);
        return nullptr;
    }
    if (dtype != GPTQ_Q4_DTYPE_FP16 && dtype != GPTQ_Q4_DTYPE_BF16) {
        api_failf(dtype == GPTQ_Q4_DTYPE_FP32 ? GPTQ_Q4_UNSUPPORTED : GPTQ_Q4_INVALID_ARGUMENT,
                  "dtype=%d: adapters are GPTQ_Q4_DTYPE_FP16 or GPTQ_Q4_DTYPE_BF16", dtype);
        return nullptr;
    }
    int dev = -1;
    if (q4::api_check_device_sm103(&dev)) return nullptr;
    gptq_q4_lora_s *h = new (std::nothrow) gptq_q4_lora_s();
    if (!h) {
        api_failf(GPTQ_Q4_OUT_OF_MEMORY, "host allocation of the adapter pool failed");
        return nullptr;
    }
    h->device = dev;
    h->K = K;
    h->N = N;
    h->slots = slots;
    h->max_rank = max_rank;
    h->dtype = dtype;
    h->sms = q4::device_sm_count();
    const size_t each = static_cast<size_t>(slots) * q4::ceil16(max_rank) * 2;
    cudaError_t e = cudaMalloc(reinterpret_cast<void **>(&h->a), each * q4::ceil64(K));
    if (!e) e = cudaMalloc(reinterpret_cast<void **>(&h->b), each * N);
    if (!e) e = cudaMalloc(reinterpret_cast<void **>(&h->slot), slots * sizeof(q4::LoraSlot));
    if (!e) e = cudaMalloc(reinterpret_cast<void **>(&h->status), sizeof(int));
    if (!e) e = cudaMemset(h->slot, 0, slots * sizeof(q4::LoraSlot));
    if (!e) e = cudaMemset(h->status, 0, sizeof(int));
    if (!e) e = cudaDeviceSynchronize();
    if (e) {
        api_cuda_fail(e, "allocating the adapter pool");
        release(h);
        return nullptr;
    }
    if (ensure_rows(h, 64, nullptr, true)) {
        release(h);
        return nullptr;
    }
    api_set_status(GPTQ_Q4_OK, nullptr);
    return h;
}

int gptq_q4_lora_set(gptq_q4_lora h, int slot, const void *a, const void *b, int rank, float scale,
                     cudaStream_t stream) {
    if (int r = check(h)) return r;
    if (slot < 0 || slot >= h->slots || rank < 0 || rank > h->max_rank)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "slot=%d must be in [0, %d) and rank=%d in [0, %d]", slot, h->slots,
                         rank, h->max_rank);
    if (!(rank ? a && b : !a && !b))
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "a and b must be given for a rank above 0, and NULL for rank 0");
    if (!std::isfinite(scale)) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "scale is not finite");
    if (rank) {
        if (int r = q4::api_check_device_ptr(a, h->device, "a")) return r;
        if (int r = q4::api_check_device_ptr(b, h->device, "b")) return r;
        if (reinterpret_cast<uintptr_t>(a) % 2 || reinterpret_cast<uintptr_t>(b) % 2)
            return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "misaligned a or b");
    }
    if (cudaError_t e = q4::launch_lora_set(view(h), h->a, h->b, h->slot, slot, static_cast<const uint16_t *>(a),
                                            static_cast<const uint16_t *>(b), rank, scale,
                                            h->dtype == GPTQ_Q4_DTYPE_BF16, stream))
        return api_cuda_fail(e, "adapter copy launch");
    q4::api_count_launches(rank ? 2 : 1);
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

int gptq_q4_lora_reserve(gptq_q4_lora h, int max_m) {
    if (int r = check(h)) return r;
    if (max_m < 0) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "max_m=%d < 0", max_m);
    if (cudaError_t e = cudaDeviceSynchronize()) return api_cuda_fail(e, "reserve");
    if (int r = ensure_rows(h, static_cast<size_t>(max_m), nullptr, true)) return r;
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

int gptq_q4_lora_add(gptq_q4_lora h, const void *x, int64_t x_stride, const int32_t *row_slot, int M, const void *y,
                     int64_t y_stride, void *out, int64_t out_stride, cudaStream_t stream) {
    if (int r = check(h)) return r;
    if (M < 0) return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "M=%d < 0", M);
    if (M == 0) return api_set_status(GPTQ_Q4_OK, nullptr);
    if (!x || !row_slot || !y || !out)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "x, row_slot, y and out must not be NULL");
    if (!aligned16(x) || !aligned16(y) || !aligned16(out) || reinterpret_cast<uintptr_t>(row_slot) % 4)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "x, y and out must be 16-byte aligned, row_slot 4-byte");
    if (x_stride < h->K || y_stride < h->N || out_stride < h->N || x_stride % 8 || y_stride % 8 || out_stride % 8)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT,
                         "row strides (x %lld, y %lld, out %lld) must be multiples of 8 and at least K=%d, N=%d, N",
                         static_cast<long long>(x_stride), static_cast<long long>(y_stride),
                         static_cast<long long>(out_stride), h->K, h->N);
    if (out == y && out_stride != y_stride)
        return api_failf(GPTQ_Q4_INVALID_ARGUMENT, "out is y but their row strides differ (%lld and %lld)",
                         static_cast<long long>(out_stride), static_cast<long long>(y_stride));
    if (int r = ensure_rows(h, static_cast<size_t>(M), stream, false)) return r;
    const q4::LoraCall c{static_cast<const uint16_t *>(x), static_cast<const uint16_t *>(y),
                         static_cast<uint16_t *>(out), row_slot, x_stride, y_stride, out_stride, M, M, nullptr};
    // Tiles of 128 rows from 321 rows on, for pools whose adapters fit a tile's pass (up to 176 ranks).  Only the GPU
    // knows how the rows lie: this many are taken to be prompts, whose rows come in runs, and rows that do mix their
    // adapters lose by it.  Measured at rank 64, by chunks and by tiles: 8192 x 28672, 128 rows of one adapter 19 us and
    // 20, 256 rows of 4 runs 32 and 27 (below the limit, as rows that mix are the rule there); 1024 rows 96 and 37; 643
    // rows of 6 runs at 28672 x 8192 166 and 42; 8192 x 10240 in 6 runs, 400 rows 31 and 25, 800 rows 65 and 31; rows
    // that mix 32 adapters, 400 rows 36 and 66, 800 rows 59 and 100.
    const bool bf16 = h->dtype == GPTQ_Q4_DTYPE_BF16;
    const q4::LoraTcPlan plan = q4::plan_lora_tc(view(h), M, h->sms);
    int launches = 0;
    cudaError_t e;
    if (M > 320 && plan.ok) e = q4::launch_lora_tc(view(h), c, plan, h->sms, bf16, stream, &launches);
    else e = q4::launch_lora_add(view(h), c, bf16, stream, &launches);
    if (e) return api_cuda_fail(e, "adapter launch");
    q4::api_count_launches(launches);
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

int gptq_q4_lora_device_error(gptq_q4_lora h) {
    if (int r = check(h)) return r;
    int flag = 0;
    cudaError_t e = cudaDeviceSynchronize();
    if (!e) e = cudaMemcpy(&flag, h->status, sizeof(int), cudaMemcpyDeviceToHost);
    if (!e && flag) e = cudaMemset(h->status, 0, sizeof(int));
    if (e) return api_cuda_fail(e, "reading the pool's status word");
    if (flag)
        return api_failf(GPTQ_Q4_DEVICE_FAULT, "adapter kernels reported status 0x%x:%s%s", flag,
                         flag & q4::kLoraBadSlot ? " a row_slot entry is not below the number of slots;" : "",
                         flag & q4::kLoraTimeout ? " a bounded wait ran out;" : "");
    return api_set_status(GPTQ_Q4_OK, nullptr);
}

void gptq_q4_lora_free(gptq_q4_lora h) {
    release(h);
    api_set_status(GPTQ_Q4_OK, nullptr);
}

}  // extern "C"
