// The handle behind gptq_q4_handle, shared by the C-ABI translation units.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/gptq_q4.h"
#include "q4_internal.cuh"

namespace q4 {
// Device buffers that a handle has replaced.  A captured graph holds the
// addresses that its calls were given, so they stay until the handle is freed.
struct Retired {
    struct Node {
        void *p;
        Node *next;
    } *head = nullptr;
};

// For a scope that frees a handle, which may be in a thread that captures a stream, or beside one that does.  In the
// relaxed mode a capture goes on past cudaFree; cudaDeviceSynchronize would end any capture of the device, in every mode.
// cudaFree of memory from cudaMalloc waits for all kernels in flight, of memory from cudaMallocAsync it does not: the
// status word, which every handle has from cudaMalloc, goes first.
class FreeScope {
    cudaStreamCaptureMode mode_ = cudaStreamCaptureModeRelaxed;
    int device_ = -1;

public:
    explicit FreeScope(int device) {
        cudaThreadExchangeStreamCaptureMode(&mode_);
        cudaGetDevice(&device_);
        if (device >= 0) cudaSetDevice(device);
    }
    ~FreeScope() {
        if (device_ >= 0) cudaSetDevice(device_);
        cudaThreadExchangeStreamCaptureMode(&mode_);
    }
    FreeScope(const FreeScope &) = delete;
    FreeScope &operator=(const FreeScope &) = delete;
};
}  // namespace q4

struct gptq_q4_s {
    int device = -1;
    int K = 0, N = 0, groupsize = 0, geff = 0, G = 0;   // K, geff: rows and rows per group of the private layout
    int Kx = 0;             // the caller's K (columns of x); K > Kx when groups are padded
    int act_order = 0;
    uint32_t *wp = nullptr;
    uint32_t *s2 = nullptr;
    uint32_t *zeros = nullptr;
    int32_t *perm = nullptr;
    int32_t *inv8 = nullptr;    // 8-bit: private row of each split row (2 Kx entries)
    uint16_t *bias = nullptr;   // bias_store, or NULL without a bias
    uint16_t *bias_store = nullptr;
    int *status = nullptr;
    float *ws = nullptr;
    size_t ws_bytes = 0;
    int *tickets = nullptr;
    size_t tickets_bytes = 0;
    uint16_t *temp_state = nullptr;
    size_t temp_state_bytes = 0;
    int path = GPTQ_Q4_PATH_AUTO;
    int prefill_min_m = 0;
    int zero_offset = 1;    // GPTQ_Q4_FORMAT_GPTQ: effective zero = stored + 1
    int bits = 4;           // 8: the handle holds an 8-bit layer as two 4-bit halves along K
    int zsplit = 0;         // groups [0, zsplit) take zero offset 0 (8-bit: the high-nibble half)
    int act_bf16 = 0;       // x and out are bf16 (GPTQ_Q4_DTYPE_BF16)
    int act_f32 = 0;        // x and out are fp32 (GPTQ_Q4_DTYPE_FP32)
    float *rowscale = nullptr;  // bf16 / fp32: 2^e per row of the current call
    size_t rowscale_bytes = 0;
    float *part = nullptr;      // fp32: the raw sums of the hi and lo rows, [2M][N]
    size_t part_bytes = 0;
    q4::Retired retired;        // replaced ones of these work buffers
    size_t device_bytes = 0;    // the replaced ones among them
};

namespace q4 {
// Status reporting and argument checks of the C ABI (q4_api.cu).
int api_set_status(int code, const char *msg);
int api_cuda_fail(cudaError_t e, const char *what);
int api_check_matmul_args(gptq_q4_handle h, const void *x, int M, const void *out);
HandleView api_view(const gptq_q4_s *h);
void api_count_launches(int n);
// Puts a buffer of at least `need` bytes in the place of *buf (*bytes large), which is retired; the contents are not
// kept.  sync: exactly `need`, at once; else by stream order, and twice the old size where there is room, so that
// the retired ones add up to no more than the present one.  zero: filled with zeros.  On an error nothing has changed.
cudaError_t api_replace(Retired &old, void **buf, size_t *bytes, size_t need, cudaStream_t s, bool sync,
                        bool zero = false);
// Keeps p until the handle is freed; false if there is no host memory for that.
bool api_retire(Retired &old, void *p);
void api_free_retired(Retired &old);
int api_check_device_ptr(const void *p, int dev, const char *name);
int api_check_device_sm103(int *dev_out);
int api_failf(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
}  // namespace q4
