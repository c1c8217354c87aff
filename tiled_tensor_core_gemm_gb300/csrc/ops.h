// What the expert-layer operators' translation units share: the argument checks
// of their C entries, and loads and stores of FP32 / BF16 / FP16 vectors.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cstdio>
#include <initializer_list>
#include <type_traits>

#include "gemm_ops.h"
#include "internal.h"

namespace tcgemm {

// --------------------------------------------------------------- C entries ---
// A span of device memory an entry point reads or writes.
struct OpSpan {
    const char *name;
    const void *p;
    uint64_t bytes;   // 0: nothing is touched, the pointer is not looked at
    int align;        // its element's size
    bool written;
    uint64_t memory_end = 0;   // op_check: where the allocation that holds it ends
};

// Steps along one dimension of a strided array.
struct OpDim {
    int64_t count, stride;
};

// Elements from the first of a strided array to behind its last (0: it has none).
// What does not fit 64 bits (sizes and strides may be 2^31 and 2^46) is the largest
// value: no extent wraps round to a small one.
inline uint64_t op_reach(std::initializer_list<OpDim> dims) {
    unsigned __int128 n = 1;
    for (const OpDim &d : dims) {
        if (d.count <= 0) return 0;
        n += (unsigned __int128)(d.count - 1) * (unsigned __int128)d.stride;
    }
    return n > UINT64_MAX ? UINT64_MAX : (uint64_t)n;
}

// The same in bytes.
inline uint64_t op_bytes(std::initializer_list<OpDim> dims, int elem) {
    const uint64_t n = op_reach(dims);
    return n > UINT64_MAX / (uint64_t)elem ? UINT64_MAX : n * (uint64_t)elem;
}

// The last byte touched + 1 of `rows` rows of `cols` elements, `ld` apart.
inline uint64_t op_extent(int64_t rows, int64_t cols, int64_t ld, int elem) {
    return op_bytes({{rows, ld}, {cols, 1}}, elem);
}

// The pitch of a matrix that is only read, row by row: 0 (one row stands for
// all) or at least a row.
inline bool op_read_pitch_ok(int64_t ld, int64_t cols) { return (ld == 0 || ld >= cols) && ld <= (1LL << 36); }

// Checks the spans (NULL, alignment, a written span overlapping another) before
// any CUDA call, then that the current device is one this library serves and
// that every span is its memory, and notes where that memory ends.  Returns a
// gemm_status_t; *sms as asked.
int op_check(OpSpan *spans, int count, int *sms);

// How a kernel reads eight neighbouring elements of a row (op_load8):
//   kOpWide     rows start on 16 bytes and are whole vectors
//   kOpShifted  the aligned 16-byte blocks that hold at least one of the elements,
//               shifted into place: as many bytes a load as the aligned case
//   kOpExact    element by element
// A shifted load touches up to 14 bytes on either side of a row.  Before it they
// belong to the allocation (which starts on 16 bytes or more); behind the last
// row's end they may not, and only then, rarely, elements are loaded one by one
// (GB300, 8191 x 4095 BF16 quantised by rows: 35.5 us instead of 27.5).
enum OpAccess { kOpWide, kOpShifted, kOpExact };

inline int op_access(bool wide, const OpSpan *read, int count) {
    if (wide) return kOpWide;
    for (int i = 0; i < count; ++i)
        if (read[i].bytes && (((uint64_t)(uintptr_t)read[i].p + read[i].bytes + 15) & ~15ull) > read[i].memory_end)
            return kOpExact;
    return kOpShifted;
}

// Workspace on `stream` (cudaFreeAsync returns it), from a pool of the library's
// own that keeps up to 256 MiB over a synchronisation: the default pool gives
// its memory back there, and the next call then waits for the driver (200 us
// and more for a workspace of a megabyte).
cudaError_t op_malloc(void **p, size_t bytes, int dev, cudaStream_t stream);

inline int op_type_bytes(int type) { return type == GEMM_OUT_F32 ? 4 : 2; }
inline bool op_type_ok(int type) { return type == GEMM_OUT_F32 || type == GEMM_OUT_BF16 || type == GEMM_OUT_F16; }
inline int op_launched(const char *what, cudaError_t e) {
    if (e == cudaSuccess) return GEMM_OK;
    char msg[192];
    std::snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
    return api_error(GEMM_ERR_CUDA, msg);
}

// Reads and clears the status word of the block-scaled product's kernel.
cudaError_t scaled_read_and_clear_status(uint32_t words[4]);
// The same of the 16-bit product's (project.cu).
cudaError_t project_read_and_clear_status(uint32_t words[4]);

#ifdef __CUDACC__
// ----------------------------------------------------------------- vectors ---
template <typename T> struct OpType;
template <> struct OpType<float> {
    static __device__ __forceinline__ float up(float x) { return x; }
    static __device__ __forceinline__ float down(float x) { return x; }
};
template <> struct OpType<__nv_bfloat16> {
    static __device__ __forceinline__ float up(__nv_bfloat16 x) { return __bfloat162float(x); }
    static __device__ __forceinline__ __nv_bfloat16 down(float x) { return __float2bfloat16_rn(x); }
};
template <> struct OpType<__half> {
    static __device__ __forceinline__ float up(__half x) { return __half2float(x); }
    static __device__ __forceinline__ __half down(float x) { return __float2half_rn(x); }
};

// Eight elements as they sit in memory: 32 bytes of FP32, 16 of the 16-bit types.
template <typename T> struct alignas(16) OpVec8 {
    T v[8];
};

// Eight elements from p, of which the first `have` exist; the rest are 0.
// kOpWide: p is on a 16-byte boundary and have is 0 or 8.
template <int ACCESS, typename T>
__device__ __forceinline__ OpVec8<T> op_load8(const T *p, int have) {
    constexpr int W = (int)sizeof(T) * 2;            // 32-bit words of the eight
    OpVec8<T> r;
    uint32_t *d = reinterpret_cast<uint32_t *>(r.v);
    if (ACCESS == kOpWide) {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 w = have > 0 ? __ldg(reinterpret_cast<const uint4 *>(p) + i / 4) : make_uint4(0, 0, 0, 0);
            d[i] = w.x;
            d[i + 1] = w.y;
            d[i + 2] = w.z;
            d[i + 3] = w.w;
        }
        return r;
    }
    if (ACCESS == kOpExact) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r.v[i] = i < have ? __ldg(p + i) : OpType<T>::down(0.f);
        return r;
    }
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint32_t off = (uint32_t)(at & 15u);
    const uint4 *blocks = reinterpret_cast<const uint4 *>(at - off);
    const uint32_t end = have > 0 ? off + (uint32_t)have * (uint32_t)sizeof(T) : 0u;   // bytes from the first block
    uint32_t w[W + 4];
#pragma unroll
    for (int i = 0; i < W + 4; i += 4) {
        const uint4 v = (uint32_t)i * 4u < end ? __ldg(blocks + i / 4) : make_uint4(0, 0, 0, 0);
        w[i] = v.x;
        w[i + 1] = v.y;
        w[i + 2] = v.z;
        w[i + 3] = v.w;
    }
    if (off & 8u) {
#pragma unroll
        for (int i = 0; i < W + 2; ++i) w[i] = w[i + 2];
    }
    if (off & 4u) {
#pragma unroll
        for (int i = 0; i < W + 1; ++i) w[i] = w[i + 1];
    }
#pragma unroll
    for (int i = 0; i < W; ++i) d[i] = sizeof(T) == 2 ? __funnelshift_r(w[i], w[i + 1], 8u * (off & 3u)) : w[i];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i >= have) r.v[i] = OpType<T>::down(0.f);
    return r;
}

// Stores the first `have` of eight elements; WIDE as kOpWide.
template <bool WIDE, typename T>
__device__ __forceinline__ void op_store8(T *p, const OpVec8<T> &r, int have) {
    if (WIDE) {
        if (have > 0) {
#pragma unroll
            for (int i = 0; i < (int)(sizeof(T) * 8 / 16); ++i)
                reinterpret_cast<uint4 *>(p)[i] = reinterpret_cast<const uint4 *>(r.v)[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < have) p[i] = r.v[i];
    }
}
#endif

// Calls f with an OpAccess as a compile-time constant.
template <typename F> auto op_by_access(int access, F &&f) {
    if (access == kOpWide) return f(std::integral_constant<int, kOpWide>());
    if (access == kOpShifted) return f(std::integral_constant<int, kOpShifted>());
    return f(std::integral_constant<int, kOpExact>());
}

// Rows of a pitched array all start on 16 bytes.
inline bool op_wide(const void *p, int64_t ld, int elem) {
    return (uintptr_t)p % 16 == 0 && ((uint64_t)ld * (uint64_t)elem) % 16 == 0;
}

// Calls f with a value of the C++ type of `type` (gemm_out_t).
template <typename F> auto op_by_type(int type, F &&f) {
    if (type == GEMM_OUT_BF16) return f(__nv_bfloat16());
    if (type == GEMM_OUT_F16) return f(__half());
    return f(float());
}

}  // namespace tcgemm
