// Quantisation to FP8 with a scale for each block of 128:
//
//   s = max(max |x| / top, 2^-126),  q = rne(x * (1 / s)),  top = 448 or 57344.
//
// The lower bound keeps 1 / s finite for blocks of zeros and denormals.  Both
// divisions are IEEE; the only rounding to fewer bits is q's.
//
// One block of 256 threads takes a 128 x 128 tile of X: 16 threads across, each
// with 8 neighbouring columns, and 16 row groups, each thread holding 8 rows
// (16 apart) in registers.  X is read once, 16 bytes a thread and eight loads
// in flight; the largest magnitudes meet in a half-warp (rows), in shared
// memory over the row groups (columns), or both (tiles); the values are then
// rounded from the registers.  It is bound by HBM: one read of X, one write of
// q (one per copy when a row goes to its experts' rows) and of the scales.
//
// Measured on GB300, BF16 to E4M3: 8192 x 4096 by rows 19 to 20 us and by tiles
// 21 (101 MB, 5.3 and 4.8 TB/s; 15 us at a plain copy's rate: about five go to
// filling and draining the launch's 4.5 rounds of blocks, for eight FP32 matrices
// of 4096 x 2048 by tiles take 51 us, 336 MB at 6.5 TB/s); 8191 x 5120 by columns
// 23.5 us (127 MB, 5.4 TB/s); 8192 x 4096 by rows to eight rows each 67 us (344 MB,
// 5.1 TB/s: four fifths of it writes, in 128-byte pieces).
#include <cuda_fp8.h>

#include "ops.h"

namespace tcgemm {
namespace {

constexpr int kTile = 128;
constexpr int kQThreads = 256;
constexpr int kRows = 8;      // rows a thread holds

struct QuantParams {
    const void *X;
    int64_t ldx, x_stride;
    uint8_t *Q;
    int64_t ldq, q_stride;
    float *S;
    int64_t s_row, s_col, s_batch;
    const int32_t *slots;
    int64_t rows, cols, out_rows;
    int copies;
    int tiles_c;
    float top;
    int e5m2;
    int q_wide;               // rows of Q start on 8 bytes (16 when rows are scattered)
};

__device__ __forceinline__ uint2 to_fp8x8(const float (&f)[8], int e5m2) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t lo, hi;
        if (e5m2) {
            lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * h], f[4 * h + 1]), __NV_SATFINITE, __NV_E5M2);
            hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * h + 2], f[4 * h + 3]), __NV_SATFINITE, __NV_E5M2);
        } else {
            lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * h], f[4 * h + 1]), __NV_SATFINITE, __NV_E4M3);
            hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * h + 2], f[4 * h + 3]), __NV_SATFINITE, __NV_E4M3);
        }
        w[h] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void put8(uint8_t *p, uint2 q, int have, bool wide) {
    if (wide && have >= 8) {
        *reinterpret_cast<uint2 *>(p) = q;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < have) p[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
}

template <typename T>
__device__ __forceinline__ uint2 scaled8(const OpVec8<T> &x, float inv, int e5m2) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = OpType<T>::up(x.v[k]) * inv;
    return to_fp8x8(f, e5m2);
}

template <typename T, int BLOCK, int ACCESS, bool SCATTER = false>
__global__ void __launch_bounds__(kQThreads, sizeof(T) == 4 ? 2 : 3) quantize_kernel(const QuantParams p) {
    pdl_enter();
    __shared__ float s_max[16][kTile];   // [row group][column]; tiles use one value a warp
    __shared__ float s_scale[kTile];
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int64_t tile = blockIdx.x;
    const int64_t r0 = tile / p.tiles_c * kTile;
    const int64_t cb = tile % p.tiles_c, c = cb * kTile + tx * 8;
    const int64_t b = blockIdx.y;
    const T *X = static_cast<const T *>(p.X) + b * p.x_stride;
    uint8_t *Q = p.Q + b * p.q_stride;
    float *S = p.S + b * p.s_batch;
    const int have = c < p.cols ? (int)(p.cols - c < 8 ? p.cols - c : 8) : 0;

    OpVec8<T> x[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + ty + 16 * i;
        x[i] = op_load8<ACCESS, T>(X + r * p.ldx + c, r < p.rows ? have : 0);
    }

    float inv8[8];           // 1 / scale of its rows (row blocks) or columns (column blocks)
    float inv = 0.f;         // of the tile
    if (BLOCK == GEMM_BLOCK_ROW) {
        // Lane i (mod 8) of a row's half-warp divides for the thread's i-th row.
        float mine = 0.f;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            float m = 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(OpType<T>::up(x[i].v[k])));
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((tx & 7) == i) mine = m;
        }
        const float s = fmaxf(mine / p.top, 0x1p-126f), s_inv = 1.f / s;
        if (tx < kRows) s_scale[ty + 16 * tx] = s;
#pragma unroll
        for (int i = 0; i < kRows; ++i) inv8[i] = __shfl_sync(0xffffffffu, s_inv, (threadIdx.x & 16) | i);
        if (!SCATTER) {
            __syncthreads();
            if (threadIdx.x < kTile && r0 + threadIdx.x < p.rows)
                S[(r0 + threadIdx.x) * p.s_row + cb * p.s_col] = s_scale[threadIdx.x];
        }
    } else {
        float m[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            m[k] = 0.f;
#pragma unroll
            for (int i = 0; i < kRows; ++i) m[k] = fmaxf(m[k], fabsf(OpType<T>::up(x[i].v[k])));
        }
        if (BLOCK == GEMM_BLOCK_TILE) {
            float t = m[0];
#pragma unroll
            for (int k = 1; k < 8; ++k) t = fmaxf(t, m[k]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
            if ((threadIdx.x & 31) == 0) s_scale[threadIdx.x >> 5] = t;
            __syncthreads();
            t = s_scale[0];
#pragma unroll
            for (int w = 1; w < kQThreads / 32; ++w) t = fmaxf(t, s_scale[w]);
            const float s = fmaxf(t / p.top, 0x1p-126f);
            inv = 1.f / s;
            if (threadIdx.x == 0) S[tile / p.tiles_c * p.s_row + cb * p.s_col] = s;
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) s_max[ty][tx * 8 + k] = m[k];
            __syncthreads();
            if (threadIdx.x < kTile) {
                float t = s_max[0][threadIdx.x];
#pragma unroll
                for (int g = 1; g < 16; ++g) t = fmaxf(t, s_max[g][threadIdx.x]);
                const float s = fmaxf(t / p.top, 0x1p-126f);
                s_scale[threadIdx.x] = 1.f / s;
                const int64_t col = cb * kTile + threadIdx.x;
                if (col < p.cols) S[tile / p.tiles_c * p.s_row + col * p.s_col] = s;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < 8; ++k) inv8[k] = s_scale[tx * 8 + k];
        }
    }

    // The rows stay packed: without this the compiler keeps their 64 widened
    // values from the search above, and an SM holds a block less.
    if (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) asm volatile("" : "+r"(reinterpret_cast<uint32_t *>(x[i].v)[k]));
    }
    if (SCATTER) {
        // The tile's rows meet in shared memory; eight lanes then write a row to each
        // of its places, 16 bytes a lane, and its scale.
        __shared__ __align__(16) uint8_t s_q[kTile][kTile];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            *reinterpret_cast<uint2 *>(&s_q[ty + 16 * i][tx * 8]) = scaled8(x[i], inv8[i], p.e5m2);
        __syncthreads();
        const int lane8 = threadIdx.x & 7;
        const int64_t at = cb * kTile + lane8 * 16;
        const int left = at < p.cols ? (int)(p.cols - at < 16 ? p.cols - at : 16) : 0;
        for (int g = threadIdx.x >> 3; g < kTile && r0 + g < p.rows; g += kQThreads / 8) {
            const int32_t *slots = p.slots + (r0 + g) * p.copies;
            const uint4 v = *reinterpret_cast<const uint4 *>(&s_q[g][lane8 * 16]);
#pragma unroll 4
            for (int j = 0; j < p.copies; ++j) {
                const int32_t to = __ldg(slots + j);
                if (to < 0 || to >= p.out_rows) continue;
                uint8_t *d = Q + (int64_t)to * p.ldq + at;
                if (p.q_wide && left == 16) *reinterpret_cast<uint4 *>(d) = v;
                else
                    for (int k = 0; k < left; ++k) d[k] = s_q[g][lane8 * 16 + k];
                if (lane8 == 0) S[(int64_t)to * p.s_row + cb * p.s_col] = s_scale[g];
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = r0 + ty + 16 * i;
        if (r >= p.rows || have == 0) continue;
        if (BLOCK == GEMM_BLOCK_COL) {
            float f[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] = OpType<T>::up(x[i].v[k]) * inv8[k];
            put8(Q + r * p.ldq + c, to_fp8x8(f, p.e5m2), have, p.q_wide);
        } else {
            put8(Q + r * p.ldq + c, scaled8(x[i], BLOCK == GEMM_BLOCK_ROW ? inv8[i] : inv, p.e5m2), have, p.q_wide);
        }
    }
}

}  // namespace
}  // namespace tcgemm

using namespace tcgemm;

extern "C" int gemm_quantize_block(int64_t batch, int64_t rows, int64_t cols, int type, const void *X, int64_t ldx,
                                   int64_t x_stride, int block, int to, void *Q, int64_t ldq, int64_t q_stride,
                                   float *S, int64_t s_row, int64_t s_col, int64_t s_batch, const int32_t *slots,
                                   int64_t copies, int64_t out_rows, struct CUstream_st *stream_) {
    api_clear_error();
    if (!op_type_ok(type)) return api_error(GEMM_ERR_INVALID_ARG, "unknown element type");
    if (to != GEMM_E4M3 && to != GEMM_E5M2) return api_error(GEMM_ERR_INVALID_ARG, "dtype must be E4M3 or E5M2");
    if (block < GEMM_BLOCK_ROW || block > GEMM_BLOCK_TILE) return api_error(GEMM_ERR_INVALID_ARG, "unknown block");
    const int64_t kMax = 0x7fffffffLL, kLdMax = 1LL << 36;
    if (batch < 0 || rows < 0 || cols < 0 || batch > 65535 || rows > kMax || cols > kMax)
        return api_error(GEMM_ERR_INVALID_ARG, "size out of range (0 <= rows, cols < 2^31, batch <= 65535)");
    const int64_t mb = block == GEMM_BLOCK_ROW ? rows : (rows + 127) / 128;
    const int64_t nb = block == GEMM_BLOCK_COL ? cols : (cols + 127) / 128;
    if (!op_read_pitch_ok(ldx, cols) || ldq < cols || ldq > kLdMax)
        return api_error(GEMM_ERR_INVALID_ARG, "leading dimension out of range");
    if (x_stride < 0 || q_stride < 0 || s_row < 0 || s_col < 0 || s_batch < 0 || x_stride > (1LL << 46) ||
        q_stride > (1LL << 46) || s_row > kLdMax || s_col > kLdMax || s_batch > (1LL << 46))
        return api_error(GEMM_ERR_INVALID_ARG, "stride out of range");
    if (slots) {
        if (block != GEMM_BLOCK_ROW || batch != 1)
            return api_error(GEMM_ERR_INVALID_ARG, "slots need row blocks and one matrix");
        if (copies < 1 || copies > 1024 || out_rows < 0 || out_rows > kMax || rows * copies > kMax)
            return api_error(GEMM_ERR_INVALID_ARG, "copies or out_rows out of range");
    }
    if (batch == 0 || rows == 0 || cols == 0 || (slots && out_rows == 0)) return GEMM_OK;
    const int64_t q_rows = slots ? out_rows : rows, s_rows = slots ? out_rows : mb;
    if (batch > 1 && ((uint64_t)q_stride < op_reach({{rows, ldq}, {cols, 1}}) ||
                      (uint64_t)s_batch < op_reach({{s_rows, s_row}, {nb, s_col}})))
        return api_error(GEMM_ERR_INVALID_ARG, "matrices of Q or S overlap");
    // distinct scales: one stride must step over the whole of the other
    if ((s_rows > 1 && nb > 1 && (uint64_t)s_row < op_reach({{nb, s_col}}) &&
         (uint64_t)s_col < op_reach({{s_rows, s_row}})) ||
        (s_rows > 1 && s_row == 0) || (nb > 1 && s_col == 0))
        return api_error(GEMM_ERR_INVALID_ARG, "scales overlap (s_row, s_col)");
    const int eb = op_type_bytes(type);
    OpSpan spans[] = {
        {"X", X, op_bytes({{batch, x_stride}, {rows, ldx}, {cols, 1}}, eb), eb, false},
        {"Q", Q, op_bytes({{batch, q_stride}, {q_rows, ldq}, {cols, 1}}, 1), 1, true},
        {"S", S, op_bytes({{batch, s_batch}, {s_rows, s_row}, {nb, s_col}}, 4), 4, true},
        {"slots", slots, slots ? (uint64_t)(rows * copies) * 4 : 0, 4, false}};
    const int rc = op_check(spans, 4, nullptr);
    if (rc) return rc;

    QuantParams p;
    p.X = X;
    p.ldx = ldx;
    p.x_stride = x_stride;
    p.Q = static_cast<uint8_t *>(Q);
    p.ldq = ldq;
    p.q_stride = q_stride;
    p.S = S;
    p.s_row = s_row;
    p.s_col = s_col;
    p.s_batch = s_batch;
    p.slots = slots;
    p.rows = rows;
    p.cols = cols;
    p.out_rows = out_rows;
    p.copies = (int)copies;
    p.tiles_c = (int)((cols + kTile - 1) / kTile);
    p.top = to == GEMM_E4M3 ? 448.f : 57344.f;
    p.e5m2 = to == GEMM_E5M2;
    const bool wide = cols % 8 == 0 && op_wide(X, ldx, eb) && (batch == 1 || ((uint64_t)x_stride * eb) % 16 == 0);
    const int q_align = slots ? 16 : 8;
    p.q_wide = (uintptr_t)Q % q_align == 0 && ldq % q_align == 0 && (batch == 1 || q_stride % 8 == 0);
    const int64_t tiles = (rows + kTile - 1) / kTile * p.tiles_c;
    if (tiles > kMax) return api_error(GEMM_ERR_INVALID_ARG, "too many blocks");
    const dim3 grid((unsigned)tiles, (unsigned)batch, 1);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const cudaError_t e = op_by_type(type, [&](auto t) {
        return op_by_access(op_access(wide, spans, 1), [&](auto w) {
            using T = decltype(t);
            constexpr int W = decltype(w)::value;
            if (slots)
                return launch_pdl(quantize_kernel<T, GEMM_BLOCK_ROW, W, true>, grid, dim3(kQThreads), 0, stream, p);
            if (block == GEMM_BLOCK_ROW)
                return launch_pdl(quantize_kernel<T, GEMM_BLOCK_ROW, W>, grid, dim3(kQThreads), 0, stream, p);
            if (block == GEMM_BLOCK_COL)
                return launch_pdl(quantize_kernel<T, GEMM_BLOCK_COL, W>, grid, dim3(kQThreads), 0, stream, p);
            return launch_pdl(quantize_kernel<T, GEMM_BLOCK_TILE, W>, grid, dim3(kQThreads), 0, stream, p);
        });
    });
    return op_launched("quantize launch", e);
}
