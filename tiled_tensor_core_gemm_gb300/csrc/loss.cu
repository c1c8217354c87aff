// The output projection's loss and its gradients: the C entries, and the kernels
// around the products of project.cu.
//
// Forward: one product H . W^T whose epilogue keeps, for each token and part of 128
// (64 in single-CTA tiles) columns, the maximum and the sum of the exponentials;
// loss_finish joins the parts.  What bounds it is the product: 2 T V D flops, or W
// once from memory where the tokens are few.  The parts are 8 bytes for each 128
// logits, 1/32 of what keeping them in 16 bits would write.
//
// Backward, the vocabulary in pieces: the piece's logits again with the gradient of
// the softmax as epilogue (16 bits, to a workspace), then dH += d W and dW = d^T H,
// the latter reading d and H as they lie (both MN-major).  6 T V D flops; dH's sums
// are read and written once a piece in FP32 (or kept as K ranges, where it has few
// tiles).  What rounding d took from its label entries is added back in FP32
// (project.h: ProductRests).
#include <algorithm>

#include "gemm_project.h"
#include "project.h"

namespace tcgemm {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kFinishWarps = 16;
// Up to here loss_rows orders the tokens by their labels in T^2 comparisons, beyond order_place
// does in passes over the labels' bits.  A whole dW of 8 columns over 8000 labels (two passes),
// comparing and in passes: 2048 tokens 54 and 64 us, 4096 80 and 81, 8192 137 and 128, 65536
// 2641 and 1605; over 131072 labels (three) 4096 take 711 and 712.
constexpr int64_t kCountTokens = 4096;
constexpr int kOrderBlocks = 128;
constexpr int kRestWarps = 16;   // of loss_rests, at most
constexpr int kWalk = 32;        // places in the order of the labels that each of them takes: one a thread to look up
constexpr int kJoinBlocks = 8;   // blocks of loss_rests that one of loss_rests_join looks at

// Token t's label, V for one that does not count.
__device__ __forceinline__ int label_key(const void *labels, int label_bytes, int64_t t, int64_t V) {
    const int64_t y = label_bytes == 8 ? __ldg(static_cast<const long long *>(labels) + t)
                                       : (int64_t)__ldg(static_cast<const int32_t *>(labels) + t);
    return y >= 0 && y < V ? (int)y : (int)V;
}

__device__ __forceinline__ bool counted(const void *labels, int label_bytes, int64_t t, int64_t V) {
    return label_key(labels, label_bytes, t, V) < (int)V;
}

// Joins a row's (maximum, sum) with another's.
__device__ __forceinline__ void join(float2 &a, float2 b) {
    const float top = fmaxf(a.x, b.x), base = top == -INFINITY ? 0.f : top;
    a.y = a.y * exp2f(a.x - base) + b.y * exp2f(b.x - base);
    a.x = top;
}

// TOKENS tokens a block (fewer where there are few, so that blocks fill the SMs), the
// threads of a token sharing its parts: joined within a warp by a butterfly, then over
// the warps in their order, so the result does not depend on timing.
template <int TOKENS>
__global__ void __launch_bounds__(32 * kFinishWarps)
loss_finish(int64_t T, int64_t V, int parts, const float2 *__restrict__ part, const float *__restrict__ sums,
            const float *__restrict__ hits, const void *labels, int label_bytes, gemm_loss_t how, float *loss, float *lse) {
    pdl_enter();
    __shared__ float2 soft[kFinishWarps][TOKENS];
    __shared__ float plain[kFinishWarps][TOKENS];
    constexpr int kWorkers = 32 * kFinishWarps / TOKENS;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = threadIdx.x % TOKENS;
    const int64_t t = (int64_t)blockIdx.x * TOKENS + mine;
    float2 m = make_float2(-INFINITY, 0.f);
    float s = 0.f;
    if (t < T) {
#pragma unroll 4
        for (int i = threadIdx.x / TOKENS; i < parts; i += kWorkers) {
            join(m, __ldg(part + (int64_t)i * T + t));
            if (sums) s += __ldg(sums + (int64_t)i * T + t);
        }
    }
#pragma unroll
    for (int d = TOKENS; d < 32; d <<= 1) {
        join(m, make_float2(__shfl_xor_sync(0xffffffffu, m.x, d), __shfl_xor_sync(0xffffffffu, m.y, d)));
        s += __shfl_xor_sync(0xffffffffu, s, d);
    }
    if (lane < TOKENS) {
        soft[warp][mine] = m;
        plain[warp][mine] = s;
    }
    __syncthreads();
    if (threadIdx.x >= TOKENS || t >= T) return;
    for (int w = 1; w < kFinishWarps; ++w) {
        join(m, soft[w][mine]);
        s += plain[w][mine];
    }
    const float total = kLn2 * (m.x + log2f(m.y));
    lse[t] = total;
    if (!loss) return;
    float l = 0.f;
    if (counted(labels, label_bytes, t, V)) {
        l = total - (1.f - how.smoothing) * __ldg(hits + t) + how.z_loss * total * total;
        if (how.smoothing != 0.f) l -= how.smoothing / (float)V * s;
    }
    loss[t] = l;
}

// FP16: the power of two that brings the largest |d| just below 2^15, and its
// inverse.  |d| is at most |grad| (1 + 2 a |lse|) (p and the target are in [0, 1],
// the cap's slope too).
__global__ void __launch_bounds__(1024)
loss_scale(int64_t T, int64_t V, const float *__restrict__ grad, int64_t grad_stride, const float *__restrict__ lse,
           const void *labels, int label_bytes, float z_loss, float *scale) {
    pdl_enter();
    __shared__ float most[32];
    float m = 0.f;
    for (int64_t t = threadIdx.x; t < T; t += 1024)
        if (counted(labels, label_bytes, t, V))
            m = fmaxf(m, fabsf(__ldg(grad + t * grad_stride)) * (1.f + 2.f * z_loss * fabsf(__ldg(lse + t))));
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    m = most[threadIdx.x];
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (threadIdx.x == 0) {
        int e = 0;
        if (m > 0.f && m < INFINITY) e = 14 - ilogbf(m);
        e = max(-100, min(100, e));
        scale[0] = ldexpf(1.f, e);
        scale[1] = ldexpf(1.f, -e);
    }
}

// The tokens in the order of their labels, where counting takes too many comparisons: eight
// bits of the labels at a time from the lowest, each pass stable.  A block takes `per`
// neighbouring tokens.  order_count: how many of them have each digit.
struct OrderKeys {
    const void *labels;            // the first pass: the labels themselves
    int label_bytes;
    int64_t V;
    const int32_t *keys, *tokens;  // or what the last pass left
    __device__ __forceinline__ int key(int64_t k) const { return keys ? __ldg(keys + k) : label_key(labels, label_bytes, k, V); }
};

__global__ void __launch_bounds__(256)
order_count(int64_t T, int64_t per, int shift, OrderKeys in, int32_t *counts) {
    pdl_enter();
    __shared__ int count[256];
    count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t end = min(T, (blockIdx.x + 1) * per);
    for (int64_t k = blockIdx.x * per + threadIdx.x; k < end; k += 256) atomicAdd(&count[in.key(k) >> shift & 255], 1);
    __syncthreads();
    counts[blockIdx.x * 256 + threadIdx.x] = count[threadIdx.x];
}

// A token's place: behind those of lower digits, those of its digit in blocks before, and
// those before it in its own block, 256 tokens at a time.
__global__ void __launch_bounds__(256)
order_place(int64_t T, int64_t per, int shift, OrderKeys in, const int32_t *__restrict__ counts, int32_t *keys_out, int32_t *tokens_out) {
    pdl_enter();
    __shared__ int seen[8][256], sums[8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int all = 0, next = 0;                       // with this thread's digit: everywhere; then the place of the next
#pragma unroll 16
    for (int b = 0; b < (int)gridDim.x; ++b) {
        const int n = __ldg(counts + b * 256 + (int)threadIdx.x);
        all += n;
        next += b < (int)blockIdx.x ? n : 0;
    }
    int up = all;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, up, d);
        if (lane >= d) up += x;
    }
    if (lane == 31) sums[warp] = up;
    __syncthreads();
    next += up - all;
    for (int w = 0; w < warp; ++w) next += sums[w];
    const int64_t end = min(T, (blockIdx.x + 1) * per);
    for (int64_t k0 = blockIdx.x * per; k0 < end; k0 += 256) {
        const int64_t k = k0 + threadIdx.x;
        const bool live = k < end;
        const int key = live ? in.key(k) : 0, digit = live ? key >> shift & 255 : -1;
        const uint32_t same = __match_any_sync(0xffffffffu, digit);
        const int rank = __popc(same & ((1u << lane) - 1u));
        for (int d = lane; d < 256; d += 32) seen[warp][d] = 0;
        __syncwarp();
        if (live && rank == 0) seen[warp][digit] = __popc(same);
        __syncthreads();
        for (int w = 0; w < 8; ++w) {
            const int n = seen[w][threadIdx.x];
            seen[w][threadIdx.x] = next;
            next += n;
        }
        __syncthreads();
        if (live) {
            const int at = seen[warp][digit] + rank;
            keys_out[at] = key;
            tokens_out[at] = in.tokens ? __ldg(in.tokens + k) : (int)k;
        }
        __syncwarp();
    }
}

// Per token: what the logits' gradient takes (project.cu: take_gradient): lse in base 2,
// grad (1 + 2 a lse), grad, and whether the token counts; with `sorted` the tokens in the
// order of the labels (ties in the order of the tokens, tokens that do not count last), each
// by counting the labels before its own; `index` cleared; and H's row, at a pitch TMA can
// address, zero for a token that does not count, so that nothing it holds (padding may be
// anything) reaches dW as 0 x NaN.  With W (held D x V): its label's column of it, as a row.
// A block takes EACH tokens, so that a label read is compared with as many.
template <int ACCESS, int EACH, typename E>
__global__ void __launch_bounds__(256)
loss_rows(int T, int64_t V, int D, const E *__restrict__ H, int64_t ldh, E *__restrict__ out, int64_t ldo,
          const float *__restrict__ grad, int64_t grad_stride, const float *__restrict__ lse, const void *labels,
          int label_bytes, float z_loss, const float *scale, float4 *rows, int32_t *sorted, int32_t *tokens, int32_t *index,
          const E *__restrict__ W, int64_t ldw, E *__restrict__ mine_of_w) {
    pdl_enter();
    __shared__ int count[EACH];
    const int per = (D + 7) / 8;
    if (index)
        for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < V; v += (int64_t)gridDim.x * 256) index[v] = -1;
    const float f = scale ? __ldg(scale) : 1.f;
    auto key = [&](int t) { return label_key(labels, label_bytes, t, V); };
    for (int64_t t0 = (int64_t)blockIdx.x * EACH; t0 < T; t0 += (int64_t)gridDim.x * EACH) {
        int mine[EACH];
#pragma unroll
        for (int k = 0; k < EACH; ++k) mine[k] = t0 + k < T ? key((int)t0 + k) : -1;
        if (sorted) {
            int before[EACH];
#pragma unroll
            for (int k = 0; k < EACH; ++k) before[k] = 0;
            __syncthreads();
            if (threadIdx.x < EACH) count[threadIdx.x] = 0;
            __syncthreads();
#pragma unroll 4
            for (int s = threadIdx.x; s < T; s += 256) {
                const int y = key(s);
#pragma unroll
                for (int k = 0; k < EACH; ++k) before[k] += y < mine[k] || (y == mine[k] && s < (int)t0 + k);
            }
#pragma unroll
            for (int k = 0; k < EACH; ++k) {
                const int n = __reduce_add_sync(0xffffffffu, before[k]);
                if ((threadIdx.x & 31) == 0) atomicAdd(&count[k], n);
            }
            __syncthreads();
        }
#pragma unroll
        for (int k = 0; k < EACH; ++k) {
            const int64_t t = t0 + k;
            if (t >= T) break;
            const bool has = mine[k] < (int)V;
            if (threadIdx.x == 0) {
                if (sorted) {
                    sorted[count[k]] = mine[k];
                    tokens[count[k]] = (int)t;
                }
                const float l = __ldg(lse + t), g = f * __ldg(grad + t * grad_stride);
                rows[t] = has ? make_float4(l * kLog2e, g * fmaf(2.f * z_loss, l, 1.f), g, 1.f)
                              : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            if (W && has)
                for (int c = threadIdx.x; c < D; c += 256) mine_of_w[t * ldo + c] = W[c * ldw + mine[k]];
            for (int c = threadIdx.x; c < per; c += 256)
                op_store8<true>(out + t * ldo + 8 * c, op_load8<ACCESS>(H + t * ldh + 8 * c, has ? min(8, D - 8 * c) : 0), 8);
        }
    }
}

// For each label in [first, first + cols) that a token has: the sum of the rests times
// the rows of H over its tokens, in their order.  A warp takes kWalk places in the order of
// the labels for 64 columns, whatever labels they have.  What it sums of a label that begins
// there goes to the label's row of `sums`, which `index` then names (by_label: the label's
// own, else that of its first place), together with what the warps behind sum of the same
// label; and what a block sums of a label that began before it to its row of `heads`, for
// loss_rests_join.  So a label that all tokens have takes no longer than many: the gradients
// of 65536 x 8000 x 512 take 2.3 ms with one label for all and 2.5 with labels at random; a
// block a label took 17.5 and 3.9.
template <typename E>
__global__ void __launch_bounds__(32 * kRestWarps)
loss_rests(int T, int64_t first, int64_t cols, int D, int col_blocks, const int32_t *__restrict__ sorted,
           const int32_t *__restrict__ tokens, const float *__restrict__ rests, const E *__restrict__ H, int64_t ldh,
           int by_label, int32_t *index, float *__restrict__ sums, float *__restrict__ heads) {
    pdl_enter();
    constexpr int kPlaces = kRestWarps * kWalk;
    __shared__ int label[kPlaces + 1];           // of the place before and of the block's, in the piece (-1: elsewhere)
    __shared__ int token[kPlaces];
    __shared__ float rest[kPlaces];
    __shared__ float2 head[kRestWarps][32];      // what a warp sums of a label that began before it
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5, places = warps * kWalk;
    const int block = blockIdx.x / col_blocks, c = ((int)(blockIdx.x - (unsigned)block * col_blocks) * 32 + lane) * 2;
    const int64_t k0 = (int64_t)block * places;
    auto in_piece = [&](int64_t k) {
        const int64_t y = k >= 0 && k < T ? __ldg(sorted + k) - first : -1;
        return y >= 0 && y < cols ? (int)y : -1;
    };
    const int64_t k = k0 + threadIdx.x;          // (a place a thread)
    const int before = threadIdx.x == 0 ? in_piece(k0 - 1) : -1, mine = in_piece(k), t = k < T ? __ldg(tokens + k) : 0;
    if (threadIdx.x == 0) label[0] = before;
    label[threadIdx.x + 1] = mine;
    token[threadIdx.x] = t;
    rest[threadIdx.x] = mine >= 0 ? __ldg(rests + t) : 0.f;
    if (!__syncthreads_or(mine >= 0)) return;
    const E *column = H + c;                     // (rows are padded to eight, with zeros)
    const int q0 = warp * kWalk;
    float a = 0.f, b = 0.f;
    bool began = false;                          // the label did in this warp's places
    int64_t row = 0;                             // its row of `sums`
    auto store = [&](float *to, int64_t r) {
        if (c < D) *reinterpret_cast<float2 *>(to + r * ldh + c) = make_float2(a, b);
    };
    for (int q1 = q0; q1 < q0 + kWalk; q1 += 16) {
        uint32_t w[16];
#pragma unroll
        for (int q = 0; q < 16; ++q)
            w[q] = label[q1 + q + 1] >= 0 && c < D ? __ldg(reinterpret_cast<const uint32_t *>(column + token[q1 + q] * ldh)) : 0u;
#pragma unroll
        for (int q = 0; q < 16; ++q) {
            const int y = label[q1 + q + 1], was = label[q1 + q];
            if (y != was) {
                if (q1 + q > q0 && was >= 0) {
                    if (began) store(sums, row);
                    else head[warp][lane] = make_float2(a, b);
                }
                a = b = 0.f;
                began = true;
                row = by_label ? y : k0 + q1 + q;
                if (y >= 0 && c == 0) index[first + y] = (int32_t)row;
            }
            const E *pair = reinterpret_cast<const E *>(&w[q]);
            a = fmaf(rest[q1 + q], OpType<E>::up(pair[0]), a);
            b = fmaf(rest[q1 + q], OpType<E>::up(pair[1]), b);
        }
    }
    const int last = label[q0 + kWalk];
    if (!began) head[warp][lane] = make_float2(a, b);
    __syncthreads();
    auto add_heads = [&](int from, int y) {      // of the warps that go on with the label
        for (int w = from; w < warps && label[w * kWalk + 1] == y; ++w) {
            a += head[w][lane].x;
            b += head[w][lane].y;
        }
    };
    if (began && last >= 0) {
        add_heads(warp + 1, last);
        store(sums, row);
    }
    if (warp == 0 && label[0] >= 0 && label[1] == label[0]) {
        a = head[0][lane].x;
        b = head[0][lane].y;
        if (label[kWalk] == label[0]) add_heads(1, label[0]);
        store(heads, block);
    }
}

// What the labels that go on from one block of loss_rests (`places` places) into the next have
// in `heads`, added to their rows of `sums`.  A block looks at kJoinBlocks of them, for 64
// columns; a label's heads are shared out to its warps 16 at a time, and the warps' sums added
// in their order.
__global__ void __launch_bounds__(256)
loss_rests_join(int T, int64_t first, int64_t cols, int D, int col_blocks, int places, const int32_t *__restrict__ sorted,
                const int32_t *__restrict__ index, const float *__restrict__ heads, int64_t ld, float *__restrict__ sums) {
    pdl_enter();
    __shared__ float2 part[8][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = blockIdx.x / col_blocks, c = ((int)(blockIdx.x - (unsigned)group * col_blocks) * 32 + lane) * 2;
    const int64_t s0 = 1 + (int64_t)group * kJoinBlocks;
    // the first of a label's heads: the label went on into this block, but not into the one before
    bool starts = false;
    int y = -1;
    if (lane < kJoinBlocks && (s0 + lane) * places < T) {
        const int64_t k = (s0 + lane) * places;
        y = __ldg(sorted + k);
        starts = y >= first && y < first + cols && __ldg(sorted + k - 1) == y && (k == places || __ldg(sorted + k - places - 1) != y);
    }
    for (uint32_t todo = __ballot_sync(0xffffffffu, starts); todo; todo &= todo - 1) {       // (the same in every warp)
        const int u = __ffs(todo) - 1, label = __shfl_sync(0xffffffffu, y, u);
        float a = 0.f, b = 0.f;
        for (int64_t s = s0 + u + warp * 16;; s += 8 * 16) {
            const bool has = lane < 16 && (s + lane) * places < T && __ldg(sorted + (s + lane) * places) == label;
            const int n = __popc(__ballot_sync(0xffffffffu, has));
            float2 x[16];
#pragma unroll
            for (int q = 0; q < 16; ++q)
                x[q] = q < n && c < D ? *reinterpret_cast<const float2 *>(heads + (s + q) * ld + c) : make_float2(0.f, 0.f);
#pragma unroll
            for (int q = 0; q < 16; ++q) {
                a += x[q].x;
                b += x[q].y;
            }
            if (n < 16) break;
        }
        part[warp][lane] = make_float2(a, b);
        __syncthreads();
        if (warp == 0 && c < D) {
            float2 *const at = reinterpret_cast<float2 *>(sums + (int64_t)__ldg(index + label) * ld + c);
            float2 sum = *at;
            for (int w = 0; w < 8; ++w) sum = make_float2(sum.x + part[w][lane].x, sum.y + part[w][lane].y);
            *at = sum;
        }
        __syncthreads();
    }
}

// dH from the FP32 sums of its K ranges, in their order: four columns a thread.
template <typename E>
__global__ void __launch_bounds__(256)
loss_join(int64_t T, int D, int parts, int64_t part_rows, const float *__restrict__ sums, int64_t pitch, E *__restrict__ out,
          int64_t ldo) {
    pdl_enter();
    const int quads = (D + 3) / 4;
    for (int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x; n < T * quads; n += (int64_t)gridDim.x * 256) {
        const int64_t t = n / quads;
        const int c = (int)(n - t * quads) * 4;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int s = 0; s < parts; ++s) {
            const float4 x = __ldcs(reinterpret_cast<const float4 *>(sums + (s * part_rows + t) * pitch + c));
            a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
        }
        const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (c + k < D) out[t * ldo + c + k] = OpType<E>::down(v[k]);
    }
}

int no_memory(uint64_t bytes, cudaError_t e) {
    cudaGetLastError();
    char msg[128];
    std::snprintf(msg, sizeof msg, "workspace of %llu bytes: %s", (unsigned long long)bytes, cudaGetErrorString(e));
    return api_error(GEMM_ERR_NO_MEMORY, msg);
}

// Parts of one stream-ordered allocation, each on 256 bytes.
struct Workspace {
    uint64_t bytes = 0;
    uint8_t *base = nullptr;
    uint64_t add(uint64_t n) {
        const uint64_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    }
    int make(cudaStream_t stream) {
        int dev = 0;
        cudaGetDevice(&dev);
        void *p = nullptr;
        const cudaError_t e = op_malloc(&p, bytes ? bytes : 256, dev, stream);
        if (e != cudaSuccess) return no_memory(bytes, e);
        base = static_cast<uint8_t *>(p);
        return GEMM_OK;
    }
    int done(int rc, cudaStream_t stream) {
        const cudaError_t e = cudaFreeAsync(base, stream);
        return rc ? rc : op_launched("cudaFreeAsync", e);
    }
};

struct LossArgs {
    int64_t T, V, D;
    int type;
    const void *H;
    int64_t ldh;
    const void *W;
    int64_t ldw;
    int w_major;
    const void *labels;
    int label_bytes;
    gemm_loss_t how;
    bool pack_h, pack_w;       // TMA cannot address them
    uint64_t h_lo, h_hi, w_lo, w_hi;
};

int check_args(LossArgs *a, int dtype, const gemm_loss_t *how) {
    const int64_t kMax = 0x7fffffffLL - 512, kLdMax = 1LL << 36;
    if (dtype != GEMM_BF16 && dtype != GEMM_FP16) return api_error(GEMM_ERR_INVALID_ARG, "dtype must be BF16 or FP16");
    a->type = dtype == GEMM_BF16 ? GEMM_OUT_BF16 : GEMM_OUT_F16;
    if (a->T < 0 || a->V < 1 || a->D < 0 || a->T > kMax || a->V > kMax || a->D > kMax)
        return api_error(GEMM_ERR_INVALID_ARG, "size negative or out of range (V must be at least 1)");
    if (a->w_major != 0 && a->w_major != 1) return api_error(GEMM_ERR_INVALID_ARG, "w_major is 0 or 1");
    if (a->label_bytes != 4 && a->label_bytes != 8) return api_error(GEMM_ERR_INVALID_ARG, "label_bytes is 4 or 8");
    const int64_t w_cols = a->w_major ? a->V : a->D;
    if (a->ldh < std::max<int64_t>(a->D, 1) || a->ldw < std::max<int64_t>(w_cols, 1) || a->ldh > kLdMax || a->ldw > kLdMax)
        return api_error(GEMM_ERR_INVALID_ARG, "leading dimension out of range");
    a->how = how ? *how : gemm_loss_t{0.f, 0.f, 0.f};
    if (!(a->how.softcap >= 0.f) || a->how.softcap > 1e30f || (a->how.softcap > 0.f && a->how.softcap < 1e-30f) ||
        !(a->how.smoothing >= 0.f && a->how.smoothing < 1.f) || !(a->how.z_loss >= 0.f) || a->how.z_loss > 1e30f)
        return api_error(GEMM_ERR_INVALID_ARG, "softcap, smoothing or z_loss out of range");
    return GEMM_OK;
}

OpSpan h_span(const LossArgs &a) { return OpSpan{"H", a.H, op_extent(a.T, a.D, a.ldh, 2), 2, false}; }
OpSpan w_span(const LossArgs &a) {
    return OpSpan{"W", a.W, a.w_major ? op_extent(a.D, a.V, a.ldw, 2) : op_extent(a.V, a.D, a.ldw, 2), 2, false};
}
OpSpan label_span(const LossArgs &a) {
    return OpSpan{"labels", a.labels, (uint64_t)a.T * (uint64_t)a.label_bytes, a.label_bytes, false};
}

// Which operands have to be copied, and the allocations they lie in.
int plan_packs(LossArgs *a) {
    if (a->T <= 1) a->ldh = op_round_up(std::max<int64_t>(a->D, 1), 8);
    const int64_t w_rows = a->w_major ? a->D : a->V, w_cols = a->w_major ? a->V : a->D;
    if (w_rows <= 1) a->ldw = op_round_up(std::max<int64_t>(w_cols, 1), 8);
    a->pack_h = !op_wide(a->H, a->ldh, 2) && a->D > 0;
    a->pack_w = !op_wide(a->W, a->ldw, 2) && a->D > 0;
    int dev = 0;
    cudaGetDevice(&dev);
    int rc = GEMM_OK;
    const OpSpan h = h_span(*a), w = w_span(*a);
    if (a->pack_h) rc = api_check_device_span_range("H", a->H, h.bytes, dev, &a->h_lo, &a->h_hi);
    if (rc == GEMM_OK && a->pack_w) rc = api_check_device_span_range("W", a->W, w.bytes, dev, &a->w_lo, &a->w_hi);
    return rc;
}

// Vocabulary entries a piece takes: equal pieces of at most `most`, multiples of 256.
int64_t piece_columns(int64_t V, int64_t most) {
    const int64_t forced = options_snapshot().loss_columns;
    if (forced) return std::min(forced, op_round_up(V, 64));
    most = std::max<int64_t>(256, most / 256 * 256);
    return std::min(most, op_round_up(op_cdiv(V, op_cdiv(V, most)), 256));
}

int64_t packed_w_bytes(const LossArgs &a, int64_t piece) {
    if (!a.pack_w) return 0;
    return 2 * (a.w_major ? a.D * op_round_up(piece, 8) : piece * op_round_up(a.D, 8));
}

// Entries [v0, v0 + n) of W as TMA can read them (copied to `to` where it cannot).
int piece_of_w(const LossArgs &a, int64_t v0, int64_t n, void *to, ProductOperand *out, cudaStream_t stream) {
    const uint16_t *src = static_cast<const uint16_t *>(a.W) + (a.w_major ? v0 : v0 * a.ldw);
    out->p = src;
    out->rows = n;
    out->ld = a.ldw;
    out->mn = a.w_major;
    if (!a.pack_w) return GEMM_OK;
    out->p = to;
    out->ld = op_round_up(a.w_major ? n : a.D, 8);
    return op_launched("operand pack", pack_rows_launch(src, a.ldw, to, out->ld, a.w_major ? a.D : n, a.w_major ? n : a.D, 2,
                                                        a.w_lo, a.w_hi, stream));
}

ProductLoss loss_of(const LossArgs &a) {
    ProductLoss l;
    l.labels = a.labels;
    l.label_bytes = a.label_bytes;
    l.softcap = a.how.softcap;
    l.eps_v = a.how.smoothing / (float)a.V;
    l.one_eps = 1.f - a.how.smoothing;
    l.want_sum = a.how.smoothing != 0.f;
    return l;
}

}  // namespace
}  // namespace tcgemm

using namespace tcgemm;

extern "C" {

int gemm_project_loss(int64_t T, int64_t V, int64_t D, int dtype, const void *H, int64_t ldh, const void *W, int64_t ldw,
                      int w_major, const void *labels, int label_bytes, const gemm_loss_t *how, float *loss, float *lse,
                      struct CUstream_st *stream_) {
    api_clear_error();
    LossArgs a = {T, V, D, 0, H, ldh, W, ldw, w_major, labels, label_bytes, {}, false, false, 0, 0, 0, 0};
    int rc = check_args(&a, dtype, how);
    if (rc) return rc;
    OpSpan spans[5] = {h_span(a), w_span(a), label_span(a), {"loss", loss, loss ? (uint64_t)T * 4 : 0, 4, true},
                       {"lse", lse, (uint64_t)T * 4, 4, true}};
    if (T == 0) return GEMM_OK;
    int sms = 0;
    if ((rc = op_check(spans, 5, &sms))) return rc;
    if ((rc = plan_packs(&a))) return rc;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    // in one piece, unless W has to be copied (256 MB at a time)
    const int64_t piece = piece_columns(V, a.pack_w ? (1LL << 27) / std::max<int64_t>(D, 1) : V + 256);
    // the tokens 65536 at a time, which bounds the memory of their parts (half a GB at V = 131072)
    const int64_t most = std::min<int64_t>(T, 65536);
    const ProductPlan plan = product_plan_stats(most, std::min(piece, V), D, !a.w_major, sms);
    int64_t parts = 0;
    for (int64_t v = 0; v < V; v += piece) parts += product_parts(plan, std::min(piece, V - v));
    if (parts > 0x7fffffffLL) return api_error(GEMM_ERR_INVALID_ARG, "too many tiles");
    const int64_t h_pitch = a.pack_h ? op_round_up(D, 8) : a.ldh;
    const bool smooth = a.how.smoothing != 0.f;
    Workspace ws;
    const uint64_t at_parts = ws.add((uint64_t)parts * most * 8), at_sums = ws.add(smooth ? (uint64_t)parts * most * 4 : 0),
                   at_hits = ws.add((uint64_t)most * 4), at_h = ws.add(a.pack_h ? (uint64_t)T * h_pitch * 2 : 0),
                   at_w = ws.add((uint64_t)packed_w_bytes(a, piece));
    if ((rc = ws.make(stream))) return rc;
    const void *h = H;
    if (a.pack_h) {
        h = ws.base + at_h;
        rc = op_launched("operand pack", pack_rows_launch(H, a.ldh, ws.base + at_h, h_pitch, T, D, 2, a.h_lo, a.h_hi, stream));
    }
    float2 *const part_of = reinterpret_cast<float2 *>(ws.base + at_parts);
    float *const sum_of = reinterpret_cast<float *>(ws.base + at_sums), *const hits = reinterpret_cast<float *>(ws.base + at_hits);
    for (int64_t t = 0; rc == GEMM_OK && t < T; t += most) {
        const int64_t n = std::min(most, T - t);
        const void *mine = static_cast<const uint8_t *>(labels) + t * label_bytes;
        ProductCall c;
        c.epilogue = kEpiStats;
        c.type = a.type;
        c.I = n;
        c.K = D;
        c.plan = plan;
        c.p = {static_cast<const uint16_t *>(h) + t * h_pitch, n, h_pitch, 0};
        c.loss = loss_of(a);
        c.loss.labels = mine;
        c.loss.hits = hits;
        int64_t part = 0;
        for (int64_t v = 0; v < V; v += piece) {
            c.J = std::min(piece, V - v);
            if ((rc = piece_of_w(a, v, c.J, ws.base + at_w, &c.q, stream))) break;
            c.loss.first = v;
            c.loss.parts = part_of + part * n;
            c.loss.sums = sum_of + part * n;
            part += product_parts(plan, c.J);
            if ((rc = product_launch(c, sms, stream))) break;
        }
        if (rc) break;
        auto finish = [&](auto tokens) {
            constexpr int kTokens = decltype(tokens)::value;
            return op_launched("loss", launch_pdl(loss_finish<kTokens>, dim3((unsigned)op_cdiv(n, kTokens)), dim3(32 * kFinishWarps), 0,
                                                  stream, n, V, (int)parts, (const float2 *)part_of,
                                                  (const float *)(smooth ? sum_of : nullptr), (const float *)hits, mine, label_bytes,
                                                  a.how, loss ? loss + t : nullptr, lse + t));
        };
        if (n <= 256) rc = finish(std::integral_constant<int, 1>());
        else if (n <= 2048) rc = finish(std::integral_constant<int, 8>());
        else rc = finish(std::integral_constant<int, 32>());
    }
    return ws.done(rc, stream);
}

int gemm_project_loss_backward(int64_t T, int64_t V, int64_t D, int dtype, const float *grad, int64_t grad_stride,
                               const void *H, int64_t ldh, const void *W, int64_t ldw, int w_major, const void *labels,
                               int label_bytes, const gemm_loss_t *how, const float *lse, void *dH, int64_t lddh, void *dW,
                               int64_t lddw, struct CUstream_st *stream_) {
    api_clear_error();
    LossArgs a = {T, V, D, 0, H, ldh, W, ldw, w_major, labels, label_bytes, {}, false, false, 0, 0, 0, 0};
    int rc = check_args(&a, dtype, how);
    if (rc) return rc;
    const int64_t kLdMax = 1LL << 36, dw_rows = w_major ? D : V, dw_cols = w_major ? V : D;
    if (grad_stride != 0 && grad_stride != 1) return api_error(GEMM_ERR_INVALID_ARG, "grad_stride is 0 or 1");
    if ((dH && (lddh < std::max<int64_t>(D, 1) || lddh > kLdMax)) || (dW && (lddw < std::max<int64_t>(dw_cols, 1) || lddw > kLdMax)))
        return api_error(GEMM_ERR_INVALID_ARG, "leading dimension out of range");
    OpSpan spans[7] = {h_span(a),
                       w_span(a),
                       label_span(a),
                       {"grad", grad, T ? (uint64_t)((T - 1) * grad_stride + 1) * 4 : 0, 4, false},
                       {"lse", lse, (uint64_t)T * 4, 4, false},
                       {"dH", dH, dH ? op_extent(T, D, lddh, 2) : 0, 2, true},
                       {"dW", dW, dW ? op_extent(dw_rows, dw_cols, lddw, 2) : 0, 2, true}};
    if (D == 0 || (!dH && !dW)) return GEMM_OK;
    int sms = 0;
    if ((rc = op_check(spans, 7, &sms))) return rc;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (T == 0) {
        if (!dW) return GEMM_OK;
        return op_launched("cudaMemset2DAsync",
                           cudaMemset2DAsync(dW, (size_t)lddw * 2, 0, (size_t)dw_cols * 2, (size_t)dw_rows, stream));
    }
    if ((rc = plan_packs(&a))) return rc;
    const int et = a.type;
    const bool f16 = et == GEMM_OUT_F16;
    // A piece's d is at most 256 MB, or 256 columns: 512 bytes a token beyond 524288 tokens
    const int64_t piece = piece_columns(V, (1LL << 27) / T);
    const int64_t pieces = op_cdiv(V, piece), d_pitch = op_round_up(piece, 64), h_pitch = op_round_up(D, 8),
                  acc_pitch = op_round_up(D, 64);
    // dH = d . W sums over a long piece of the vocabulary into few tiles
    const ProductPlan h_plan = product_plan_rows(T, D, std::min(piece, V), sms, 16);
    const int64_t part_rows = op_round_up(T, 256);
    const bool join = h_plan.parts > 1;
    Workspace ws;
    // dW takes the label entries' rests by label, so the tokens are put in the order of their labels.
    const bool order = dW != nullptr, passes = order && T > kCountTokens;
    const bool by_label = piece < T;
    const int rest_warps = (int)std::min<int64_t>(kRestWarps, op_cdiv(T, kWalk));
    const int64_t blocks = op_cdiv(T, rest_warps * kWalk);          // of loss_rests
    const uint64_t at_index = ws.add(order ? (uint64_t)V * 4 : 0),
                   at_sums = ws.add(order ? (uint64_t)std::min(T, piece) * h_pitch * 4 : 0),
                   at_heads = ws.add(order ? (uint64_t)blocks * h_pitch * 4 : 0);
    const uint64_t at_rests = ws.add((uint64_t)T * 4),
                   at_label_w = ws.add(dH && w_major ? (uint64_t)T * h_pitch * 2 : 0),
                   at_sorted = ws.add((uint64_t)T * 4), at_tokens = ws.add((uint64_t)T * 4),
                   at_keys = ws.add(passes ? (uint64_t)T * 4 : 0), at_places = ws.add(passes ? (uint64_t)T * 4 : 0),
                   at_counts = ws.add(passes ? kOrderBlocks * 256 * 4 : 0);
    const uint64_t at_rows = ws.add((uint64_t)T * 16), at_scale = ws.add(8), at_h = ws.add((uint64_t)T * h_pitch * 2),
                   at_d = ws.add((uint64_t)T * d_pitch * 2), at_w = ws.add((uint64_t)packed_w_bytes(a, piece)),
                   at_acc = ws.add(!dH ? 0 : join ? (uint64_t)h_plan.parts * part_rows * acc_pitch * 4 : pieces > 1 ? (uint64_t)T * acc_pitch * 4 : 0);
    if ((rc = ws.make(stream))) return rc;
    float4 *rows = reinterpret_cast<float4 *>(ws.base + at_rows);
    int32_t *index = reinterpret_cast<int32_t *>(ws.base + at_index);
    float *sums = reinterpret_cast<float *>(ws.base + at_sums);
    int32_t *sorted = reinterpret_cast<int32_t *>(ws.base + at_sorted), *tokens = reinterpret_cast<int32_t *>(ws.base + at_tokens);
    float *rests = reinterpret_cast<float *>(ws.base + at_rests), *heads = reinterpret_cast<float *>(ws.base + at_heads);
    float *scale = reinterpret_cast<float *>(ws.base + at_scale), *acc = reinterpret_cast<float *>(ws.base + at_acc);
    if (f16 && rc == GEMM_OK)
        rc = op_launched("loss scale", launch_pdl(loss_scale, dim3(1), dim3(1024), 0, stream, T, V, grad, grad_stride, lse, labels,
                                                  label_bytes, a.how.z_loss, scale));
    if (passes) {
        const int64_t per = op_round_up(op_cdiv(T, kOrderBlocks), 256);
        const dim3 grid((unsigned)op_cdiv(T, per));
        int32_t *keys = reinterpret_cast<int32_t *>(ws.base + at_keys), *places = reinterpret_cast<int32_t *>(ws.base + at_places),
                *counts = reinterpret_cast<int32_t *>(ws.base + at_counts);
        OrderKeys in = {labels, label_bytes, V, nullptr, nullptr};
        for (int shift = 0; rc == GEMM_OK && (V >> shift) > 0; shift += 8) {          // (keys are at most V)
            rc = op_launched("label counts", launch_pdl(order_count, grid, dim3(256), 0, stream, T, per, shift, in, counts));
            if (rc) break;
            rc = op_launched("label order", launch_pdl(order_place, grid, dim3(256), 0, stream, T, per, shift, in,
                                                       (const int32_t *)counts, keys, places));
            std::swap(keys, sorted);
            std::swap(places, tokens);
            in.keys = sorted;
            in.tokens = tokens;
        }
    }
    const bool wide = op_wide(H, a.ldh, 2) && D % 8 == 0;
    const int access = op_access(wide, &spans[0], 1);
    if (rc == GEMM_OK)
        rc = op_by_access(access, [&](auto acc_kind) {
            auto go = [&](auto e, auto each) {
                using E = decltype(e);
                constexpr int kEach = decltype(each)::value;
                // Where it gathers W's columns its blocks start together, after the kernel before: they then
                // read the same rows of W at the same time (the gradients of 4096 x 32000 x 2048 with W held
                // dim x vocabulary 1395 us, as a programmatic dependent 1475).
                const dim3 grid((unsigned)std::max(op_cdiv(T, kEach), order ? op_cdiv(V, 16384) : 0));
                return op_launched("loss rows",
                                   launch_kernel(dH == nullptr || !w_major, loss_rows<decltype(acc_kind)::value, kEach, E>, grid, dim3(256),
                                                 0, stream, (int)T, V, (int)D, static_cast<const E *>(H), a.ldh,
                                                 reinterpret_cast<E *>(ws.base + at_h), h_pitch, grad, grad_stride, lse, labels,
                                                 label_bytes, a.how.z_loss, (const float *)(f16 ? scale : nullptr), rows,
                                                 order && !passes ? sorted : nullptr, tokens, order ? index : nullptr,
                                                 static_cast<const E *>(dH && w_major ? W : nullptr), a.ldw,
                                                 reinterpret_cast<E *>(ws.base + at_label_w)));
            };
            using One = std::integral_constant<int, 1>;
            using Eight = std::integral_constant<int, 8>;
            if (f16) return T <= 2048 ? go(__half(), One()) : go(__half(), Eight());
            return T <= 2048 ? go(__nv_bfloat16(), One()) : go(__nv_bfloat16(), Eight());
        });
    const ProductOperand h_rows = {ws.base + at_h, T, h_pitch, 0}, h_cols = {ws.base + at_h, D, h_pitch, 1};
    int64_t n = 0;
    for (int64_t v = 0; rc == GEMM_OK && v < V; v += piece, ++n) {
        const int64_t cols = std::min(piece, V - v);
        ProductOperand w;
        if ((rc = piece_of_w(a, v, cols, ws.base + at_w, &w, stream))) break;
        ProductCall d;
        d.epilogue = kEpiDlogits;
        d.type = et;
        d.I = T;
        d.J = cols;
        d.K = D;
        d.plan = product_plan_rows(T, cols, D, sms);
        d.p = h_rows;
        d.q = w;
        d.C = ws.base + at_d;
        d.ldc = d_pitch;
        d.epi.active = 1;
        d.epi.out = et;
        d.padded = true;
        d.loss = loss_of(a);
        d.loss.first = v;
        d.loss.rows = rows;
        d.loss.rests = rests;
        if ((rc = product_launch(d, sms, stream))) break;
        if (dH) {
            ProductCall c;
            c.epilogue = kEpiRests;
            c.loss = loss_of(a);
            c.loss.first = v;
            c.rests.kind = 1;
            c.rests.rests = rests;
            c.rests.w = w_major ? ws.base + at_label_w : w.p;
            c.rests.ld = w_major ? h_pitch : w.ld;
            c.rests.by_token = w_major;
            c.rests.cols = cols;
            c.type = et;
            c.I = T;
            c.J = D;
            c.K = cols;
            c.plan = h_plan;
            c.part_rows = part_rows;
            c.p = {ws.base + at_d, T, d_pitch, 0};
            c.q = {w.p, D, w.ld, w.mn ^ 1};       // (W's entries are the sum now)
            c.old = n > 0 ? acc : nullptr;
            c.ld_old = acc_pitch;
            const bool last = n + 1 == pieces && !join;
            c.padded = !last;
            c.C = last ? dH : acc;
            c.ldc = last ? lddh : acc_pitch;
            c.epi.active = 1;
            c.epi.out = last ? et : GEMM_OUT_F32;
            c.alpha = f16 ? scale + 1 : nullptr;
            if ((rc = product_launch(c, sms, stream))) break;
        }
        if (dW) {
            const ProductOperand d_cols = {ws.base + at_d, cols, d_pitch, 1};
            ProductCall c;
            if (order) {
                auto go = [&](auto e) {
                    using E = decltype(e);
                    const int64_t wide = op_cdiv(D, 64);
                    return op_launched("loss rests",
                                       launch_pdl(loss_rests<E>, dim3((unsigned)(blocks * wide)), dim3(32 * rest_warps), 0, stream,
                                                  (int)T, v, cols, (int)D, (int)wide, (const int32_t *)sorted, (const int32_t *)tokens,
                                                  (const float *)rests, reinterpret_cast<const E *>(ws.base + at_h), h_pitch,
                                                  by_label ? 1 : 0, index, sums, heads));
                };
                if ((rc = f16 ? go(__half()) : go(__nv_bfloat16()))) break;
                if (blocks > 1) {
                    const int64_t wide = op_cdiv(D, 64);
                    rc = op_launched("loss rests join",
                                     launch_pdl(loss_rests_join, dim3((unsigned)(op_cdiv(blocks - 1, kJoinBlocks) * wide)), dim3(256), 0,
                                                stream, (int)T, v, cols, (int)D, (int)wide, rest_warps * kWalk, (const int32_t *)sorted,
                                                (const int32_t *)index, (const float *)heads, h_pitch, sums));
                    if (rc) break;
                }
            }
            c.epilogue = order ? kEpiRests : kEpiRows;
            c.loss.first = v;
            c.rests.kind = w_major ? 3 : 2;
            c.rests.index = index;
            c.rests.sums = sums;
            c.rests.ld = h_pitch;
            c.type = et;
            c.I = w_major ? D : cols;
            c.J = w_major ? cols : D;
            c.K = T;
            c.plan = product_plan_rows(c.I, c.J, T, sms);
            c.p = w_major ? h_cols : d_cols;
            c.q = w_major ? d_cols : h_cols;
            c.C = static_cast<uint16_t *>(dW) + (w_major ? v : v * lddw);
            c.ldc = lddw;
            c.epi.active = 1;
            c.epi.out = et;
            c.alpha = f16 ? scale + 1 : nullptr;
            if ((rc = product_launch(c, sms, stream))) break;
        }
    }
    if (rc == GEMM_OK && dH && join) {
        auto go = [&](auto e) {
            using E = decltype(e);
            return op_launched("loss join",
                               launch_pdl(loss_join<E>, dim3((unsigned)std::min<int64_t>(op_cdiv(T * op_cdiv(D, 4), 256), sms * 8)),
                                          dim3(256), 0, stream, T, (int)D, h_plan.parts, part_rows, (const float *)acc, acc_pitch,
                                          static_cast<E *>(dH), lddh));
        };
        rc = f16 ? go(__half()) : go(__nv_bfloat16());
    }
    return ws.done(rc, stream);
}

}  // extern "C"
