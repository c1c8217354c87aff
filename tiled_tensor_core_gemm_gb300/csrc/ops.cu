// Argument checks shared by the expert-layer operators' C entries.
#include "ops.h"

#include <mutex>

namespace tcgemm {

cudaError_t op_malloc(void **p, size_t bytes, int dev, cudaStream_t stream) {
    static std::mutex mu;
    static cudaMemPool_t pools[64];
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    cudaMemPool_t pool;
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!pools[dev]) {
            cudaMemPoolProps props = {};
            props.allocType = cudaMemAllocationTypePinned;
            props.location.type = cudaMemLocationTypeDevice;
            props.location.id = dev;
            // The first call may come while this or another thread captures a graph.
            // Creating a pool is not a stream's work, so the capture need not forbid it.
            cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
            cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
            if (e != cudaSuccess) return e;
            cudaMemPool_t made = nullptr;
            e = cudaMemPoolCreate(&made, &props);
            if (e == cudaSuccess) {
                uint64_t keep = 256ull << 20;
                e = cudaMemPoolSetAttribute(made, cudaMemPoolAttrReleaseThreshold, &keep);
                if (e != cudaSuccess) cudaMemPoolDestroy(made);
            }
            const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
            if (e == cudaSuccess) pools[dev] = made;
            if (e == cudaSuccess) e = back;
            if (e != cudaSuccess) return e;
        }
        pool = pools[dev];
    }
    return cudaMallocFromPoolAsync(p, bytes, pool, stream);
}

int op_check(OpSpan *spans, int count, int *sms) {
    char msg[256];
    for (int i = 0; i < count; ++i) {
        const OpSpan &s = spans[i];
        if (s.bytes == 0) continue;
        if (!s.p) {
            std::snprintf(msg, sizeof msg, "%s is NULL", s.name);
            return api_error(GEMM_ERR_INVALID_ARG, msg);
        }
        if ((uintptr_t)s.p % (uintptr_t)s.align != 0) {
            std::snprintf(msg, sizeof msg, "%s is not aligned to its %d-byte element", s.name, s.align);
            return api_error(GEMM_ERR_INVALID_ARG, msg);
        }
        if (s.bytes > (1ull << 62) || (uint64_t)(uintptr_t)s.p + s.bytes < (uint64_t)(uintptr_t)s.p) {
            std::snprintf(msg, sizeof msg, "%s: extent out of range", s.name);
            return api_error(GEMM_ERR_INVALID_ARG, msg);
        }
    }
    for (int i = 0; i < count; ++i)
        for (int j = i + 1; j < count; ++j) {
            const OpSpan &a = spans[i], &b = spans[j];
            if (!(a.written || b.written) || a.bytes == 0 || b.bytes == 0) continue;
            const uint64_t a0 = (uint64_t)(uintptr_t)a.p, b0 = (uint64_t)(uintptr_t)b.p;
            if (a0 < b0 + b.bytes && b0 < a0 + a.bytes) {
                std::snprintf(msg, sizeof msg, "%s and %s overlap", a.name, b.name);
                return api_error(GEMM_ERR_INVALID_ARG, msg);
            }
        }
    int dev = 0, n = 0, major = 0, minor = 0, clusters = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return op_launched("cudaGetDevice", e);
    int rc = api_device_info(dev, &n, &major, &minor, &clusters);
    if (rc) return rc;
    if (!(major == 10 && minor == 3)) {
        std::snprintf(msg, sizeof msg, "this library is built for sm_103a only (device is sm_%d%d)", major, minor);
        return api_error(GEMM_ERR_UNSUPPORTED, msg);
    }
    uint64_t begin;
    for (int i = 0; i < count; ++i)
        if (spans[i].bytes && (rc = api_check_device_span_range(spans[i].name, spans[i].p, spans[i].bytes, dev, &begin,
                                                                &spans[i].memory_end)))
            return rc;
    if (sms) *sms = n;
    return GEMM_OK;
}

}  // namespace tcgemm
