// Products of 16-bit matrices whose operands are gathered or whose result is used
// where it is made, for the output projection's loss and the low-rank adapters:
//
//   D[i][j] = sum_k P[i][k] * Q[j][k]
//
// P is the operand whose rows become Tensor Memory lanes, Q the one whose rows
// become its columns.  Four uses, by `mode`:
//
//   plain      D as it is.
//   add        D += low x adapters: the adapters' part is further K-blocks of the
//              same accumulator.  `low` holds, for each token, the rank-wide
//              activations in the columns of its adapter's slot and zeros in the
//              other slots of its granule of tokens, so one pass over a tile's
//              slots adds every token's own adapter and nothing else.
//   low        makes it: tokens x the adapters of the granule's slots, all of them
//              for every token of the tile (the adapters' matrices are read once a
//              tile, and those bytes are what this costs), then masked.
//   gradient   for one adapter, sums over the tokens that may take it: the K-blocks
//              are 64 tokens each of the granules on the adapter's list, and the
//              zeros in `low` drop the other tokens.
//
// `low` in 16 bits would be most of the gradients' error, and of a result of few tokens,
// so what its rounding took is kept in 16 bits too and multiplied along there: it rides
// in the ring slot of the first (more MMAs, no more slots).
//
// and four epilogues: C written with its columns on the lanes ("swapped": few
// tokens, so that the lanes carry the weights' rows and a tile is only as wide as
// the tokens are), C row by row, the statistics of a softmax over the columns, and
// the gradient of its logits.
//
// What bounds it (GB300): with many tokens the tensor cores, which a 256 x 256 pair keeps
// 86% busy with the loss statistics of 2048 x 16384 x 4096 (91% of active cycles; 543 to
// 573 us for 65536 columns = 1.92 to 2.0 PFLOP/s) and 71 to 78% with its gradients'
// products (few rounds); over a step of 8192 x 131072 x 4096 the power cap does, at 0.97 to
// 1.0 of the sustained rate.  With few, the stream of the weights: 5 x 50021 x 2048 at
// 5.4 TB/s; 64 x 4096 x 12288 at 4.3 from 96 of 152 SMs.  In between, a K-block's 0.18 us
// in small tiles (of which the MMAs' issue is about half) and 8 us around them.
//
// Roles as in scaled.cu: warp 0 issues the TMA loads into a ring, warp 1 the MMAs
// (two K-blocks of 64 a ring slot, one 128-byte swizzle row each), and from warp 4 on the epilogue
// warps, which read one of two accumulators while the MMAs fill the other.  Either
// operand in either major: K-major as rows of 64 values, MN-major in chunks of 64
// rows of K by 64 values.  Every wait is bounded; a role that gives up waits,
// again bounded, for what it started.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <mutex>

#include "epilogue.cuh"
#include "gelu.cuh"
#include "project.h"
#include "ptx.cuh"
#include "ptx_ops.cuh"

namespace tcgemm {

__device__ uint32_t g_project_status[4];

namespace {

constexpr int kLanes = 128;
constexpr int kBlockK = 64;
constexpr int kSmemMax = 232448;
constexpr int kCtrlBytes = 1024;
constexpr int kSlotBlocks = 2;             // K-blocks of a ring slot
constexpr int kChunkBytes = 64 * 128;      // an MN-major chunk: 64 rows of K x 64 values
constexpr int kBoxBytes = 4096;            // 32 rows x 128 bytes of C
constexpr float kLog2e = 1.4426950408889634f;

enum Role : uint32_t { kRoleProducer = 1, kRoleMma = 2, kRoleEpilogue = 3, kRoleDrain = 4 };

struct ProductParams {
    int mode;
    int I, J, num_kb;
    int tiles_i, tiles_j, num_tiles;
    int width;                 // columns of a tile: BN, or (statistics) fewer
    int group_i;               // raster: lane tiles taken together
    int splits;                // CTAs of a cluster that share a tile's K
    int k_parts, part_rows;    // K ranges whose sums go to C one below the other, part_rows apart
    int p_mn, q_mn;
    uint32_t idesc, idesc_add; // of the operands, and of low x adapters
    void *C;
    int64_t ldc, c_stride;
    // a second product (low, gradient): tiles from tiles_first on
    int tiles_first, I2, num_kb2, tiles_i2;
    void *C2;
    int64_t ldc2, c_stride2;
    int wide2;
    int wide, tma_store;       // C's rows start on 16 bytes; and end on them
    EpiParams epi;
    const float *alpha;
    const float *old;
    int64_t ld_old;
    // adapters
    int pitch_log2, granule, granule_blocks, max_slots, adapters;
    const int32_t *slots, *counts, *slot_of, *lists, *list_counts;
    int64_t granules;
    const float *scales;
    int64_t rest;              // elements from low to what its rounding took (0: not kept)
    // loss
    const void *labels;
    int label_bytes;
    int64_t first;
    float softcap, inv_softcap, eps_v, one_eps;
    int want_sum;
    float2 *parts;
    float *sums, *hits;
    const float4 *rows;
    float *rests_out;
    ProductRests rests;
    int f16;                   // the operands' type
    int early, debug_stall;
    unsigned long long timeout_ns;
};

template <int BN, int CG, int EPI, int PROWS>
struct Cfg {
    static constexpr bool SWAPPED = EPI == kEpiSwapped || EPI == kEpiGradient;
    static constexpr int EW = BN <= 32 ? 4 : 8;            // epilogue warps
    static constexpr int ROWS = kLanes * CG;
    static constexpr int COLS = BN / (EW / 4);             // columns of a thread
    static constexpr int THREADS = 128 + EW * 32;
    // K-blocks an accumulator sums (0: all).  The tensor cores' long FP32 sums lose a
    // little at every step (a loss over 4096 values off by 1.9e-6, against 4e-7 of an
    // FP32 product); the statistics add accumulators of 8 x 64 in registers.
    static constexpr int SEG = EPI == kEpiStats ? 8 : 0;
    // Registers a thread after the first warpgroup has given some up (0: as launched).
    static constexpr int GIVE = EPI == kEpiStats && COLS > 64 ? 56 : 0, TAKE = GIVE ? 224 : 0;
    static_assert(GIVE == 0 || 128 * GIVE + EW * 32 * TAKE <= THREADS * 168, "the shares exceed the launch's registers");
    // Rows of P a CTA loads.  With 32 the MMAs read what follows as further lanes,
    // which nobody looks at: few tokens stream W through a ring that is nearly all W's.
    static constexpr int P_BYTES = PROWS * 128;
    static constexpr int Q_ROWS = BN / CG;                 // each CTA of a pair loads half of Q's rows
    // (an N-major chunk has at least 64 columns; the gradient has as much again for low's
    // rests, and few tokens have room for theirs)
    static constexpr int Q_ONE = (Q_ROWS < 64 ? 64 : Q_ROWS) * 128;
    static constexpr int Q_BYTES = EPI == kEpiGradient ? 2 * Q_ONE : Q_ONE;
    static constexpr bool ADD_RESTS = EPI == kEpiSwapped && Q_ROWS <= 32;
    static constexpr int Q_CHUNKS = Q_ROWS < 64 ? 1 : Q_ROWS / 64;
    static constexpr int BLOCK = P_BYTES + Q_BYTES;
    static_assert(PROWS == kLanes || (EPI == kEpiStats && Q_BYTES + P_BYTES >= kLanes * 128), "P's rows");
    // A ring slot is two K-blocks: what a slot costs its producer and its MMA warp to
    // wait for, announce and hand on (about 500 cycles each, whatever the tile) is as
    // much as a 256 x 256 pair's MMAs of one K-block take, and twice a smaller tile's.
    static constexpr int STAGE = kSlotBlocks * BLOCK;
    static constexpr int TMEM_COLS = 2 * BN < 32 ? 32 : 2 * BN;
    static constexpr int OUT_BYTES = SWAPPED ? 2048 : EPI == kEpiStats ? 0 : kBoxBytes;
    static constexpr int FIXED = 1024 + kCtrlBytes + EW * OUT_BYTES;
    static constexpr int FIT = (kSmemMax - FIXED) / STAGE;
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static_assert(STAGES >= 2 && SMEM <= kSmemMax, "ring");
    static_assert((2 * STAGES + 4) * 8 + 16 <= kCtrlBytes, "barrier area");
    static_assert(2 * BN <= 512, "two accumulators");
    static_assert(!SWAPPED || kLanes * BN * 4 <= STAGES * STAGE, "a tile's partial sums fit in the ring");
};

__device__ __noinline__ void record_failure(uint32_t role, int tile, volatile int *abort_flag) {
    *abort_flag = 1;
    if (atomicCAS(&g_project_status[0], 0u, (uint32_t)GEMM_ERR_TIMEOUT) == 0u) {
        g_project_status[1] = role;
        g_project_status[2] = (uint32_t)tile;
        g_project_status[3] = blockIdx.x;
        __threadfence();
    }
}

struct Bounds {
    volatile int *abort_flag;
    unsigned long long timeout_ns;
};

// A whole warp waits for a phase of a barrier.  False once the time is up or
// another role has given up.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, const Bounds &b, uint32_t role, int tile) {
    uint64_t t0 = 0;
#pragma unroll 1
    while (!__all_sync(0xffffffffu, ptx::mbar_try_wait<false>(bar, parity))) {
        const uint64_t now = ptx::globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, now - t0 > b.timeout_ns || *b.abort_flag != 0)) {
            if ((threadIdx.x & 31) == 0) record_failure(role, tile, b.abort_flag);
            __syncwarp();
            return false;
        }
    }
    return true;
}

// The wait of a role that has given up, for what it started itself.
__device__ __noinline__ void wait_landed(uint32_t bar, uint32_t parity, unsigned long long timeout_ns) {
    const uint64_t t0 = ptx::globaltimer_ns();
    while (!ptx::mbar_try_wait<false>(bar, parity))
        if (ptx::globaltimer_ns() - t0 > timeout_ns) return;
}

// A position in a ring of N slots.
template <int N> struct Ring {
    int slot = 0;
    uint32_t lap = 0;          // its parity
    __device__ __forceinline__ void step() {
        if (++slot == N) {
            slot = 0;
            lap ^= 1u;
        }
    }
};

// One output tile and this CTA's K-blocks of it.  K-blocks from num_kb on are the
// adapters' (kModeAdd).
struct Tile {
    int i0, i1, j0, j1;
    int e, g, slots;           // the adapter; the granule and its slots
    int down;                  // rows of C above this K range's
    int kb0, kb1;
    int own;                   // where the operands' own K-blocks end and the adapters' begin
    bool none;                 // nothing to do: no slot reaches these lanes
    bool second;               // of the launch's second product
    // K-blocks of the ring slot that begins with kb (never of both kinds).
    __device__ __forceinline__ int slot_blocks(int kb) const { return min(kSlotBlocks, (kb < own ? own : kb1) - kb); }
};

// The slots of a granule (within what a plan can hold, whatever the buffer given as one does).
__device__ __forceinline__ int slots_of(const ProductParams &p, int g) { return min(max(__ldg(p.counts + g), 0), p.max_slots); }

template <int BN, int ROWS, bool SWAPPED>
__device__ __forceinline__ Tile tile_at(const ProductParams &p, int t, int crank) {
    Tile T;
    T.e = T.g = T.slots = T.down = 0;
    T.none = false;
    T.second = SWAPPED && t >= p.tiles_first;
    if (T.second) t -= p.tiles_first;
    T.i1 = T.second ? p.I2 : p.I;
    T.j1 = p.J;
    int total = T.second ? p.num_kb2 : p.num_kb, ranges = p.splits, range = crank;
    if (p.mode == kModeLow) {
        // (the first lanes of every token tile first: most granules have few slots)
        const int ti = t / p.tiles_j;
        T.i0 = ti * ROWS;
        T.j0 = (t - ti * p.tiles_j) * BN;
        T.g = T.j0 / p.granule;
        T.slots = slots_of(p, T.g);
        T.i1 = T.slots << p.pitch_log2;
        T.none = T.i0 >= T.i1;
    } else if (p.mode == kModeGradient) {
        const int tiles_i = T.second ? p.tiles_i2 : p.tiles_i;
        T.e = t / tiles_i;
        T.i0 = (t - T.e * tiles_i) * ROWS;
        T.j0 = 0;
        total = min(max(__ldg(p.list_counts + T.e), 0), (int)p.granules) * p.granule_blocks;
    } else {
        if (!SWAPPED && p.k_parts > 1) {
            const int tiles = p.tiles_i * p.tiles_j;
            ranges = p.k_parts;
            range = t / tiles;
            t -= range * tiles;
            T.down = range * p.part_rows;
        }
        const int per = p.group_i * p.tiles_j, grp = t / per, first = grp * p.group_i;
        const int gi = min(p.group_i, p.tiles_i - first);
        const int in = t - grp * per;
        T.i0 = (first + in % gi) * ROWS;
        T.j0 = in / gi * p.width;
        T.j1 = min(p.J, T.j0 + p.width);
        if (p.mode == kModeAdd) {
            T.g = (SWAPPED ? T.j0 : T.i0) / p.granule;
            T.slots = slots_of(p, T.g);
            total += ((T.slots << p.pitch_log2) + kBlockK - 1) / kBlockK;
        }
    }
    const int each = (total + ranges - 1) / ranges;
    T.kb0 = min(total, range * each);
    T.kb1 = min(total, T.kb0 + each);
    T.own = p.mode == kModeAdd ? min(T.kb1, p.num_kb) : T.kb1;
    return T;
}

// A list in memory, 32 entries of it in a warp's registers at a time.
struct WarpList {
    const int32_t *p;
    int count, base = -32, held = 0;
    __device__ __forceinline__ int at(int i) {        // warp-uniform
        if (i < base || i >= base + 32) {
            base = i & ~31;
            const int k = base + (int)(threadIdx.x & 31);
            held = k < count ? __ldg(p + k) : 0;
        }
        return __shfl_sync(0xffffffffu, held, i & 31);
    }
};

// The epilogue's value from a whole sum.
__device__ __forceinline__ float finish(const EpiParams &e, float acc, float bias) {
    float y = fmaf(e.alpha, acc, bias);
    if (e.act == GEMM_ACT_RELU) y = ptx::relu_nan(y);
    else if (e.act == GEMM_ACT_GELU) y = gelu2(make_float2(y, y)).x;
    return y;
}

// What rounding x to the operands' type takes from it; nothing where the rounded value is
// not finite (an infinity has no rest: inf - inf would make its row NaN).
__device__ __forceinline__ float rest_of(const ProductParams &p, float x) {
    const float r = x - (p.f16 ? __half2float(__float2half_rn(x)) : __bfloat162float(__float2bfloat16_rn(x)));
    return fabsf(r) < INFINITY ? r : 0.f;
}

// Four neighbouring columns of row cr of C.  `side`: the bias of each, or (low)
// the factor of their slot's adapter; `slot`: (low) the token's.
__device__ __forceinline__ void write_four(const ProductParams &p, const Tile &T, int64_t cr, int64_t cc, float4 v,
                                           const float (&side)[4], int slot) {
    float y[4] = {v.x, v.y, v.z, v.w};
    void *const C = T.second ? p.C2 : p.C;
    const int64_t ldc = T.second ? p.ldc2 : p.ldc;
    if (p.mode == kModeLow) {
        // a token keeps the columns of its own slot (selected, not multiplied: what
        // another slot's product held, a NaN included, goes)
        const bool mine = slot == (int)(cc >> p.pitch_log2);
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = mine ? y[k] * side[k] : 0.f;
        if (p.rest) {
            float z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) z[k] = rest_of(p, y[k]);
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(C) + p.rest + cr * ldc + cc) =
                make_uint2(epi_pack2(p.epi.out, z[0], z[1]), epi_pack2(p.epi.out, z[2], z[3]));
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = finish(p.epi, y[k], side[k]);
    }
    const int64_t at = T.e * (T.second ? p.c_stride2 : p.c_stride) + cr * ldc + cc;
    if ((T.second ? p.wide2 : p.wide) && cc + 4 <= T.i1) {
        if (p.epi.out != GEMM_OUT_F32)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(C) + at) =
                make_uint2(epi_pack2(p.epi.out, y[0], y[1]), epi_pack2(p.epi.out, y[2], y[3]));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(C) + at) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (cc + k < T.i1) epi_store(C, at + k, p.epi.out, y[k]);
    }
}

// What write_four takes beside the four columns from cc on.
__device__ __forceinline__ void side_of(const ProductParams &p, const Tile &T, int64_t cc, float (&side)[4]) {
    if (p.mode == kModeLow) {
        const int s = (int)(cc >> p.pitch_log2);
        const int ad = p.scales && cc < T.i1 ? __ldg(p.slots + (int64_t)T.g * p.max_slots + s) : -1;
        const float f = (unsigned)ad < (unsigned)p.adapters ? __ldg(p.scales + ad) : 1.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) side[k] = f;
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) side[k] = p.epi.bias && cc + k < T.i1 ? __ldg(p.epi.bias + cc + k) : 0.f;
    }
}

// A warp's 32 lanes x COLS columns of D as COLS rows of C of 32 neighbouring
// columns, through 2 KB of shared memory, 16 rows of C at a time: eight lanes
// then hold 32 neighbouring elements of a row.
template <int COLS>
__device__ __forceinline__ void write_swapped(const ProductParams &p, const Tile &T, int row0, int col0, float (&acc)[COLS],
                                              const float (&side)[4], int (&own)[COLS / 4], uint32_t buf, int lane) {
    const int u = lane & 7;
    const int64_t cc = (int64_t)T.i0 + row0 + 4 * u;
#pragma unroll 1
    for (int c0 = 0; c0 < COLS; c0 += 16) {
        const int64_t r0 = (int64_t)T.j0 + col0 + c0;
        if (r0 >= T.j1) break;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 16; ++c) ptx::st_shared_f(buf + 4u * (uint32_t)(c * 32 + lane), acc[c]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int r = (lane >> 3) + 4 * k;
            const float4 v = ptx::ld_shared_v4f(buf + 128u * (uint32_t)r + 16u * (uint32_t)u);
            if (cc < T.i1 && r0 + r < T.j1) write_four(p, T, r0 + r, cc, v, side, own[k]);
        }
#pragma unroll
        for (int c = 0; c + 16 < COLS; ++c) acc[c] = acc[c + 16];
#pragma unroll
        for (int k = 0; k + 4 < COLS / 4; ++k) own[k] = own[k + 4];
    }
}

// The slots (low) of the rows of C that a lane writes in write_swapped, looked up while
// the MMAs run (with the factors likewise: one token's two launches 21 -> 17 us by graph).
template <int COLS>
__device__ __forceinline__ void slots_of_rows(const ProductParams &p, const Tile &T, int col0, int lane, int (&own)[COLS / 4]) {
#pragma unroll
    for (int k = 0; k < COLS / 4; ++k) {
        const int r = T.j0 + col0 + 4 * k + (lane >> 3);
        own[k] = p.mode == kModeLow && r < T.j1 ? __ldg(p.slot_of + r) : -1;
    }
}

// 64 columns of a thread's row: from Tensor Memory, as floats.
__device__ __forceinline__ void load_64(uint32_t src, float (&v)[64]) {
    uint32_t a[32], b[32];
    ptx::tmem_ld_32x32b_x32(src, a);
    ptx::tmem_ld_32x32b_x32(src + 32u, b);
    ptx::tmem_wait_ld(a);
    ptx::tmem_landed(b);
#pragma unroll
    for (int c = 0; c < 32; ++c) {
        v[c] = __uint_as_float(a[c]);
        v[32 + c] = __uint_as_float(b[c]);
    }
}

// v += COLS columns of a thread's row, 32 at a time (one load in flight: the MMAs of
// the next K-blocks take ten times as long, and a second would cost registers).
template <int COLS>
__device__ __forceinline__ void add_columns(uint32_t src, float (&v)[COLS]) {
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += 32) {
        uint32_t a[32];
        ptx::tmem_ld_32x32b_x32(src + (uint32_t)c0, a);
        ptx::tmem_wait_ld(a);
#pragma unroll
        for (int c = 0; c < 32; ++c) v[c0 + c] += __uint_as_float(a[c]);
    }
}

// Rows of a box of 32 rows x 128 bytes in shared memory to C with ordinary stores.
__device__ __forceinline__ void store_box_plain(const ProductParams &p, const Tile &T, uint32_t buf, int64_t i0,
                                                int64_t jb, bool half, int lane) {
    const int rows = T.i1 - i0 < 32 ? (int)(T.i1 - i0) : 32;
    const int64_t row0 = i0 + T.down;
    const int most = half ? 64 : 32;
    const int cols = (int)(T.j1 - jb < most ? T.j1 - jb : most);
#pragma unroll 2
    for (int r = 0; r < rows; ++r) {
        const uint32_t from = buf + 128u * (uint32_t)r;
        const int64_t at = (row0 + r) * p.ldc + jb + lane;
        const uint32_t sw = (uint32_t)(r & 7) << 4;
        if (half) {
            uint16_t *d = static_cast<uint16_t *>(p.C) + at;
            if (lane < cols) d[0] = ptx::ld_shared_u16(from + ((2u * (uint32_t)lane) ^ sw));
            if (lane + 32 < cols) d[32] = ptx::ld_shared_u16(from + ((2u * (uint32_t)lane + 64u) ^ sw));
        } else if (lane < cols) {
            static_cast<float *>(p.C)[at] = ptx::ld_shared_f(from + ((4u * (uint32_t)lane) ^ sw));
        }
    }
}

// 64 columns of 32 rows, one row a thread, to C: through a box (16-bit) or two
// (FP32) of 32 rows x 128 bytes of shared memory with TMA's 128-byte swizzle,
// which leaves by a TMA store where C's layout allows it.
__device__ __forceinline__ void store_64(const ProductParams &p, const CUtensorMap *tmC, const Tile &T, int64_t i0,
                                         int64_t j, const float (&v)[64], uint32_t buf, int lane) {
    const bool half = p.epi.out != GEMM_OUT_F32;
    const uint32_t row = buf + 128u * (uint32_t)lane;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int64_t jb = j + 32 * b;
        if (b == 1 && (half || jb >= T.j1)) break;
        // the box's last store must have read it
        if (lane == 0) ptx::bulk_wait_group_read<0>();
        __syncwarp();
        if (half) {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                ptx::st_shared_v4(row + 16u * (uint32_t)(u ^ (lane & 7)),
                                  make_uint4(epi_pack2(p.epi.out, v[8 * u], v[8 * u + 1]),
                                             epi_pack2(p.epi.out, v[8 * u + 2], v[8 * u + 3]),
                                             epi_pack2(p.epi.out, v[8 * u + 4], v[8 * u + 5]),
                                             epi_pack2(p.epi.out, v[8 * u + 6], v[8 * u + 7])));
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                ptx::st_shared_v4f(row + 16u * (uint32_t)(u ^ (lane & 7)),
                                   make_float4(v[32 * b + 4 * u], v[32 * b + 4 * u + 1], v[32 * b + 4 * u + 2],
                                               v[32 * b + 4 * u + 3]));
        }
        if (p.tma_store) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                ptx::tma_store_2d(tmC, buf, (int)jb, (int)i0 + T.down);
                ptx::bulk_commit_group();
            }
        } else {
            __syncwarp();
            store_box_plain(p, T, buf, i0, jb, half, lane);
            __syncwarp();
        }
    }
}

// The row-wise epilogue on 64 columns from j on of row i.
__device__ __forceinline__ void finish_row(const ProductParams &p, const Tile &T, int64_t i, int64_t j, float alpha,
                                           float (&v)[64]) {
    if (alpha != 1.f) {
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] *= alpha;
    }
    if (p.old && i < T.i1) {
        const float *o = p.old + (i + T.down) * p.ld_old + j;          // (rows start on 16 bytes, pitch a multiple of 64)
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
            if (j + c >= T.j1) break;
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(o + c));
            v[c] += x.x;
            v[c + 1] += x.y;
            v[c + 2] += x.z;
            v[c + 3] += x.w;
        }
    }
    if (p.epi.bias) {
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] += j + c < T.j1 ? __ldg(p.epi.bias + j + c) : 0.f;
    }
    if (p.epi.act == GEMM_ACT_RELU) {
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] = ptx::relu_nan(v[c]);
    } else if (p.epi.act == GEMM_ACT_GELU) {
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
            const float2 g = gelu2(make_float2(v[c], v[c + 1]));
            v[c] = g.x;
            v[c + 1] = g.y;
        }
    }
}

// tanh of the first 64 of v.  Logits mostly lie well inside their cap: while all of a
// warp's are at most 1/2 the Taylor series up to x^15 is within a unit in the last place
// (at 1/2 the next term is 4.5e-9, a seventh of one) and takes 8 multiply-adds, where tanhf
// takes about 25 instructions with two special-function calls.
template <int N>
__device__ __forceinline__ void tanh_64(float (&v)[N]) {
    float most = 0.f;
#pragma unroll
    for (int c = 0; c < 64; ++c) most = fmaxf(most, fabsf(v[c]));
    if (__all_sync(0xffffffffu, most <= 0.5f)) {
        auto both = [](float c) { return make_float2(c, c); };
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
            const float2 x = make_float2(v[c], v[c + 1]), q = __fmul2_rn(x, x);
            float2 r = both(-929569.f / 638512875.f);
            r = __ffma2_rn(r, q, both(21844.f / 6081075.f));
            r = __ffma2_rn(r, q, both(-1382.f / 155925.f));
            r = __ffma2_rn(r, q, both(62.f / 2835.f));
            r = __ffma2_rn(r, q, both(-17.f / 315.f));
            r = __ffma2_rn(r, q, both(2.f / 15.f));
            r = __ffma2_rn(r, q, both(-1.f / 3.f));
            r = __ffma2_rn(__fmul2_rn(r, q), x, x);
            v[c] = r.x;
            v[c + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] = tanhf(v[c]);
    }
}

// The label of token i as a column of this call's D (far outside it if it has none here).
__device__ __forceinline__ int64_t label_column(const ProductParams &p, int64_t i) {
    const int64_t y = p.label_bytes == 8 ? __ldg(static_cast<const long long *>(p.labels) + i)
                                         : (int64_t)__ldg(static_cast<const int32_t *>(p.labels) + i);
    return y < 0 ? -(1LL << 40) : y - p.first;
}

// v += f * eight neighbouring 16-bit values (on 16 bytes).
__device__ __forceinline__ void add_eight(const ProductParams &p, const uint4 &w, float f, float *v) {
    const uint32_t q[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float lo, hi;
        epi_unpack2(p.f16 ? GEMM_OUT_F16 : GEMM_OUT_BF16, q[k], lo, hi);
        v[2 * k] = fmaf(f, lo, v[2 * k]);
        v[2 * k + 1] = fmaf(f, hi, v[2 * k + 1]);
    }
}

// What rounding took from the label entries of d (ProductRests), on 64 columns from j
// on of row i.
__device__ __forceinline__ void add_rests(const ProductParams &p, const Tile &T, int64_t i, int64_t j, int lane, float (&v)[64]) {
    const ProductRests &r = p.rests;
    const int have = (int)(T.j1 - j < 64 ? T.j1 - j : 64), type = p.f16 ? GEMM_OUT_F16 : GEMM_OUT_BF16;
    if (r.kind == 1) {
        const int64_t y = i < T.i1 ? label_column(p, i) : -1;
        if (y < 0 || y >= r.cols) return;
        const float f = __ldg(r.rests + i);
        const uint16_t *at = static_cast<const uint16_t *>(r.w) + (r.by_token ? i : y) * r.ld + j;
        // eight columns at a time (rows start on 16 bytes); what is left one by one
#pragma unroll
        for (int c = 0; c < 64; c += 8) {
            if (c + 8 <= have) {
                add_eight(p, __ldg(reinterpret_cast<const uint4 *>(at + c)), f, v + c);
            } else if (c < have) {
#pragma unroll
                for (int k = 0; k < 7; ++k) {
                    float lo = 0.f, hi;
                    if (c + k < have) epi_unpack2(type, __ldg(at + c + k), lo, hi);
                    v[c + k] = fmaf(f, lo, v[c + k]);
                }
            }
        }
    } else if (r.kind == 2) {
        const int k = i < T.i1 ? __ldg(r.index + p.first + i) : -1;
        if (k < 0) return;
        const float *at = r.sums + k * r.ld + j;             // (on 16 bytes, with room for the row's last four)
#pragma unroll
        for (int c = 0; c < 64; c += 4) {
            if (c >= have) break;
            const float4 x = __ldg(reinterpret_cast<const float4 *>(at + c));
            v[c] += x.x;
            v[c + 1] += x.y;
            v[c + 2] += x.z;
            v[c + 3] += x.w;
        }
    } else {
        int k[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) k[h] = 32 * h + lane < have ? __ldg(r.index + p.first + j + 32 * h + lane) : -1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!__any_sync(0xffffffffu, k[h] >= 0)) continue;
            // (all loads before the first sum: one after the other the 60 labels among the
            // first 64 entries cost a tile 40 us)
            float x[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const int64_t row = __shfl_sync(0xffffffffu, k[h], c);
                x[c] = row >= 0 && i < T.i1 ? __ldg(r.sums + row * r.ld + i) : 0.f;
            }
#pragma unroll
            for (int c = 0; c < 32; ++c) v[32 * h + c] += x[c];
        }
    }
}

// Running maximum (in base 2) and sum of a row's exponentials.
struct Softmax {
    float top = -INFINITY, sum = 0.f, plain = 0.f;
};

// Takes the first 64 of v, logits of neighbouring columns, of which the first `have`
// exist (and changes them).  `at`: the label's place among them, or outside [0, 64).
template <int N>
__device__ __forceinline__ void take_logits(const ProductParams &p, float (&v)[N], int have, int at, Softmax &s,
                                            float &hit) {
    if (p.softcap != 0.f) {
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] *= p.inv_softcap;
        tanh_64(v);
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] *= p.softcap;
    }
    if (p.want_sum) {
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
            a += c < have ? v[c] : 0.f;
            b += c + 1 < have ? v[c + 1] : 0.f;
        }
        s.plain += a + b;
    }
    if (__any_sync(0xffffffffu, at >= 0 && at < have)) {
#pragma unroll
        for (int c = 0; c < 64; ++c) hit = c == at && c < have ? v[c] : hit;
    }
    if (have < 64) {
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] = c < have ? v[c] : -INFINITY;
    }
    float m0 = v[0], m1 = v[1], m2 = v[2], m3 = v[3];
#pragma unroll
    for (int c = 4; c < 64; c += 4) {
        m0 = fmaxf(m0, v[c]);
        m1 = fmaxf(m1, v[c + 1]);
        m2 = fmaxf(m2, v[c + 2]);
        m3 = fmaxf(m3, v[c + 3]);
    }
    const float top = fmaxf(s.top, fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * kLog2e);
    const float base = top == -INFINITY ? 0.f : top;        // (nothing but -inf so far: the sum stays 0)
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int c = 0; c < 64; c += 2) {
        a += ptx::exp2_approx(fmaf(v[c], kLog2e, -base));
        b += ptx::exp2_approx(fmaf(v[c + 1], kLog2e, -base));
    }
    s.sum = fmaf(s.sum, ptx::exp2_approx(s.top - base), a + b);
    s.top = top;
}

// 64 logits to their gradient times the row's factors (loss.cu: rows).
__device__ __forceinline__ void take_gradient(const ProductParams &p, float (&v)[64], const float4 &row, int at) {
    const float lse = row.x, a = row.y, flat = row.z * p.eps_v;
    if (p.softcap != 0.f) {
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] *= p.inv_softcap;
        tanh_64(v);
#pragma unroll
        for (int c = 0; c < 64; ++c) {
            const float u = v[c];
            const float d = fmaf(ptx::exp2_approx(fmaf(p.softcap * u, kLog2e, -lse)), a, -flat);
            v[c] = (c == at ? d - row.z * p.one_eps : d) * fmaf(-u, u, 1.f);
        }
        return;
    }
#pragma unroll
    for (int c = 0; c < 64; ++c) v[c] = fmaf(ptx::exp2_approx(fmaf(v[c], kLog2e, -lse)), a, -flat);
    if (__any_sync(0xffffffffu, at >= 0 && at < 64)) {
#pragma unroll
        for (int c = 0; c < 64; ++c) v[c] = c == at ? v[c] - row.z * p.one_eps : v[c];
    }
}

template <int BN, int CG, int EPI, int PROWS>
__global__ void __launch_bounds__((Cfg<BN, CG, EPI, PROWS>::THREADS), 1)
product_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
               const __grid_constant__ CUtensorMap tmLow, const __grid_constant__ CUtensorMap tmAd,
               const __grid_constant__ CUtensorMap tmC, const ProductParams p) {
    using Cf = Cfg<BN, CG, EPI, PROWS>;
    constexpr bool kPair = CG == 2, kSwapped = Cf::SWAPPED, kGradient = EPI == kEpiGradient;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    uint8_t *ring = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *out_bufs = ring + Cf::STAGES * Cf::STAGE;
    uint64_t *bars = reinterpret_cast<uint64_t *>(out_bufs + Cf::EW * Cf::OUT_BYTES);
    constexpr int kBars = 2 * Cf::STAGES + 4;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const Bounds bounds = {abort_flag, p.timeout_ns};

    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto empty = [&](int s) { return bar0 + 8u * (uint32_t)(Cf::STAGES + s); };
    auto accf = [&](int b) { return bar0 + 8u * (uint32_t)(2 * Cf::STAGES + b); };
    auto acce = [&](int b) { return bar0 + 8u * (uint32_t)(2 * Cf::STAGES + 2 + b); };
    const uint32_t ring0 = ptx::smem_addr(ring), out0 = ptx::smem_addr(out_bufs);

    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int crank = kSwapped && p.splits > 1 ? (int)ptx::cluster_ctarank() : 0;   // its K range
    const uint32_t rank = kPair ? ptx::cluster_ctarank() : 0u;                      // its half of the pair's tile

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cf::STAGES; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(empty(s), 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(accf(b), 1);
            ptx::mbar_init(acce(b), Cf::EW * CG);
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
        if (p.num_kb > 0) {
            if (p.mode != kModeLow) ptx::prefetch_tensormap(&tmP);
            if (!kGradient) ptx::prefetch_tensormap(&tmQ);
        }
        if (p.tma_store) ptx::prefetch_tensormap(&tmC);
    }
    if (warp == 1) {
        ptx::tmem_alloc<CG>(ptx::smem_addr(tmem_slot), Cf::TMEM_COLS);
        ptx::tmem_relinquish<CG>();
    }
    // Global memory from here on: the previous kernel on the stream is done.  With
    // `early` that kernel makes `low` and nothing else this one reads, and let this
    // one start only once it had itself waited for everything before it: the
    // operands may be read at once, `low` after a wait, and nothing is written
    // before one.
    if (!p.early) {
        ptx::pdl_wait();
        if (threadIdx.x == 0) ptx::pdl_launch_dependents();
    }
    ptx::tc_fence_before();
    if (kPair) {
        __syncwarp();
        ptx::cluster_sync();      // the peer's barriers are ready before any arrival on them
    } else {
        __syncthreads();
    }
    ptx::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int share = kPair ? 2 : kSwapped ? p.splits : 1;      // CTAs of a tile
    const int unit = (int)blockIdx.x / share, units = (int)gridDim.x / share;

    if (warp == 0) {
        if constexpr (Cf::GIVE != 0) ptx::regs_give_back<Cf::GIVE>();
        // ---------------------------------------------------------- TMA producer
        // (the whole warp, one elected thread issuing)
        Ring<Cf::STAGES> at;
        int issued = 0;
        bool ok = true, waited = !p.early;
        for (int t = unit; ok && t < p.num_tiles; t += units) {
            const Tile T = tile_at<BN, Cf::ROWS, kSwapped>(p, t, crank);
            if (T.none) continue;
            const int i0 = T.i0 + (int)rank * kLanes, j0 = T.j0 + (int)rank * (p.width / CG);
            uint32_t fb = 0, sp = 0, sq = 0, to = 0;
            // The next ring slot: its barrier, where its operands go, and (of a pair the
            // leader's) the barrier their bytes count on.
            auto next_slot = [&]() {
                if (!wait_warp(empty(at.slot), at.lap ^ 1u, bounds, kRoleProducer, t)) return ok = false;
                fb = full(at.slot);
                sp = ring0 + (uint32_t)(at.slot * Cf::STAGE);
                sq = sp + Cf::P_BYTES;
                to = kPair ? ptx::mapa_shared(fb, 0) : fb;
                at.step();
                ++issued;
                return true;
            };
            if (EPI == kEpiSwapped && p.mode == kModeLow) {
                // the adapters of the tile's lanes: at most eight boxes of `pitch` rows
                const int pitch = 1 << p.pitch_log2, boxes = min(kLanes, T.i1 - T.i0) >> p.pitch_log2;
                const int s = (T.i0 >> p.pitch_log2) + (int)lane;
                const int mine = (int)lane < boxes ? __ldg(p.slots + (int64_t)T.g * p.max_slots + s) : 0;
                int ad[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) ad[u] = __shfl_sync(0xffffffffu, mine, u);
                const uint32_t bytes = (uint32_t)((boxes << p.pitch_log2) * 128 + Cf::Q_ROWS * 128);
                // (the second product's maps are where this mode has no other use for them)
                const CUtensorMap *const mq = T.second ? &tmP : &tmQ, *const ma = T.second ? &tmC : &tmAd;
                for (int kb = T.kb0; kb < T.kb1 && next_slot(); kb += kSlotBlocks) {
                    const int n = T.slot_blocks(kb);
                    if (ptx::elect_one()) {
                        ptx::mbar_arrive_expect_tx(fb, bytes * n);
#pragma unroll
                        for (int s = 0; s < kSlotBlocks; ++s) {
                            if (s >= n) break;
                            const int k0 = (kb + s) * kBlockK;
                            ptx::tma_load_2d(sq + s * Cf::BLOCK, mq, fb, k0, j0);
#pragma unroll
                            for (int u = 0; u < 8; ++u)
                                if (u < boxes) ptx::tma_load_3d<1>(sp + (uint32_t)(s * Cf::BLOCK + u * pitch * 128), ma, fb, k0, 0, ad[u]);
                        }
                    }
                    __syncwarp();
                }
                continue;
            }
            if constexpr (kGradient) {
                // 64 tokens of a granule on the list at a time, and the adapter's slot in it
                const int log2_blocks = 31 - __clz(p.granule_blocks);
                const CUtensorMap *const mp = T.second ? &tmQ : &tmP, *const ml = T.second ? &tmAd : &tmLow;
                WarpList list = {p.lists + T.e * p.granules, (T.kb1 + p.granule_blocks - 1) >> log2_blocks};
                for (int kb = T.kb0; kb < T.kb1; kb += kSlotBlocks) {
                    const int n = T.slot_blocks(kb);
                    int k0[kSlotBlocks], jx[kSlotBlocks];
#pragma unroll
                    for (int s = 0; s < kSlotBlocks; ++s) {
                        const int k = min(kb + s, T.kb1 - 1), entry = list.at(k >> log2_blocks);
                        k0[s] = (entry >> 8) * p.granule + (k & (p.granule_blocks - 1)) * kBlockK;
                        jx[s] = (entry & 255) << p.pitch_log2;
                    }
                    if (!next_slot()) break;
                    if (ptx::elect_one()) {
                        ptx::mbar_arrive_expect_tx(fb, (uint32_t)(Cf::BLOCK * n));
#pragma unroll
                        for (int s = 0; s < kSlotBlocks; ++s) {
                            if (s >= n) break;
                            ptx::tma_load_2d(sp + s * Cf::BLOCK, mp, fb, i0, k0[s]);
                            ptx::tma_load_2d(sp + s * Cf::BLOCK + kChunkBytes, mp, fb, i0 + 64, k0[s]);
#pragma unroll
                            for (int c = 0; c < Cf::Q_CHUNKS; ++c) {
                                const uint32_t to_q = sq + (uint32_t)(s * Cf::BLOCK + c * kChunkBytes);
                                ptx::tma_load_3d<1>(to_q, ml, fb, jx[s] + 64 * c, k0[s], 0);
                                ptx::tma_load_3d<1>(to_q + Cf::Q_ONE, ml, fb, jx[s] + 64 * c, k0[s], 1);
                            }
                        }
                    }
                    __syncwarp();
                }
                continue;
            }
            const uint32_t bytes = (uint32_t)(Cf::P_BYTES + (p.q_mn ? Cf::Q_BYTES : p.width / CG * 128)) * CG;
            for (int kb = T.kb0; kb < T.own && next_slot(); kb += kSlotBlocks) {
                const int n = T.slot_blocks(kb);
                if (ptx::elect_one()) {
                    if (rank == 0) ptx::mbar_arrive_expect_tx(fb, bytes * n);
#pragma unroll
                    for (int s = 0; s < kSlotBlocks; ++s) {
                        if (s >= n) break;
                        const int k0 = (kb + s) * kBlockK;
                        const uint32_t dp = sp + s * Cf::BLOCK, dq = sq + s * Cf::BLOCK;
                        if (p.p_mn) {
                            ptx::tma_load_2d_cg<CG>(dp, &tmP, to, i0, k0);
                            ptx::tma_load_2d_cg<CG>(dp + kChunkBytes, &tmP, to, i0 + 64, k0);
                        } else {
                            ptx::tma_load_2d_cg<CG>(dp, &tmP, to, k0, i0);
                        }
                        if (p.q_mn) {
#pragma unroll
                            for (int c = 0; c < Cf::Q_CHUNKS; ++c)
                                ptx::tma_load_2d_cg<CG>(dq + (uint32_t)(c * kChunkBytes), &tmQ, to, j0 + 64 * c, k0);
                        } else {
                            ptx::tma_load_2d_cg<CG>(dq, &tmQ, to, k0, j0);
                        }
                    }
                }
                __syncwarp();
            }
            if constexpr (EPI == kEpiSwapped || EPI == kEpiRows) {   // (the others have no adapters)
                if (!ok || p.mode != kModeAdd || T.kb1 <= p.num_kb) continue;
                if (!waited) ptx::pdl_wait();
                waited = true;
                // low, and up to four boxes of `box` rows of the adapters' (a slot's, or half
                // of one of 128) in N-major chunks of 64 columns
                constexpr int kAddChunks = kSwapped ? kLanes / 64 : Cf::Q_CHUNKS;
                const int box = min(1 << p.pitch_log2, kBlockK), log2_box = min(p.pitch_log2, 6);
                WarpList list = {p.slots + (int64_t)T.g * p.max_slots, T.slots};
                for (int kb = max(T.kb0, p.num_kb); kb < T.kb1; kb += kSlotBlocks) {
                    const int n = T.slot_blocks(kb);
                    int boxes[kSlotBlocks], ad[kSlotBlocks][4], all = 0;
#pragma unroll
                    for (int s = 0; s < kSlotBlocks; ++s) {
                        const int row0 = (kb + s - p.num_kb) * kBlockK;
                        boxes[s] = s < n ? min(kBlockK, (T.slots << p.pitch_log2) - row0) >> log2_box : 0;
                        all += boxes[s];
#pragma unroll
                        for (int u = 0; u < 4; ++u) ad[s][u] = u < boxes[s] ? list.at((row0 + u * box) >> p.pitch_log2) : 0;
                    }
                    if (!next_slot()) break;
                    if (ptx::elect_one()) {
                        constexpr int kLow = !kSwapped ? Cf::P_BYTES : Cf::ADD_RESTS ? 2 * Cf::Q_ROWS * 128 : Cf::Q_ROWS * 128;
                        if (rank == 0) ptx::mbar_arrive_expect_tx(fb, (uint32_t)(all * box * 128 * kAddChunks + n * kLow) * CG);
#pragma unroll
                        for (int s = 0; s < kSlotBlocks; ++s) {
                            if (s >= n) break;
                            const int row0 = (kb + s - p.num_kb) * kBlockK;
                            ptx::tma_load_3d<CG>((kSwapped ? sq : sp) + s * Cf::BLOCK, &tmLow, to, row0, kSwapped ? j0 : i0, 0);
                            if (Cf::ADD_RESTS)
                                ptx::tma_load_3d<CG>(sq + s * Cf::BLOCK + Cf::Q_ROWS * 128, &tmLow, to, row0, j0, 1);
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                if (u < boxes[s]) {
#pragma unroll
                                    for (int c = 0; c < kAddChunks; ++c)
                                        ptx::tma_load_3d<CG>(
                                            (kSwapped ? sp : sq) + (uint32_t)(s * Cf::BLOCK + c * kChunkBytes + u * box * 128), &tmAd,
                                            to, (kSwapped ? i0 : j0) + 64 * c, row0 & ((1 << p.pitch_log2) - 1), ad[s][u]);
                                }
                        }
                    }
                    __syncwarp();
                }
            }
        }
        if (!waited) ptx::pdl_wait();      // (this grid ends after the one it depends on)
        // Until the MMAs have released every slot no read of this shared memory and
        // no arrival on its barriers is outstanding.
        Ring<Cf::STAGES> end = at;
        for (int i = 0; ok && i < Cf::STAGES; ++i, at.step()) ok = wait_warp(empty(at.slot), at.lap ^ 1u, bounds, kRoleDrain, -1);
        // Given up: the copies already issued still land in this shared memory
        // (those of a pair are counted in the leader).
        if (!ok && rank == 0) {
            const int n = issued < Cf::STAGES ? issued : Cf::STAGES;
            for (int i = 0; i < n; ++i) {
                // the i-th slot before `end`
                int slot = end.slot - 1 - i;
                uint32_t lap = end.lap;
                if (slot < 0) {
                    slot += Cf::STAGES;
                    lap ^= 1u;
                }
                wait_landed(full(slot), lap, p.timeout_ns);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if constexpr (Cf::GIVE != 0) ptx::regs_give_back<Cf::GIVE>();
        // ------------------------------------------------------------ MMA issuer
        if (rank == 0) {
            Ring<Cf::STAGES> at;
            Ring<2> acc;
            bool ok = true;
            uint32_t last_bar = 0, last_parity = 0;      // of the MMAs issued last
            // descriptors in 16-byte units: leading offset, and the step of one MMA's K = 16.
            // K-major: 32 bytes inside a 128-byte row, 8-row groups 1024 bytes apart.
            // MN-major: 16 rows of K further, chunks of 64 values 8 KB apart.
            const uint32_t p_lead = (p.p_mn ? 512u : 1u) << 16, q_lead = (p.q_mn ? 512u : 1u) << 16;
            const uint32_t p_step = p.p_mn ? 128u : 2u, q_step = p.q_mn ? 128u : 2u;
            // (no accumulator is handed back before the first has been written; half
            // the limit, so that this wait and not one behind it runs out first)
            if (p.debug_stall) ok = wait_warp(acce(0), 0u, Bounds{abort_flag, p.timeout_ns / 2}, kRoleMma, unit);
            for (int t = unit; ok && t < p.num_tiles; t += units) {
                const Tile T = tile_at<BN, Cf::ROWS, kSwapped>(p, t, crank);
                if (T.none) continue;
                int start = T.kb0;                 // of the accumulator's K-blocks
                for (int kb = T.kb0, next; kb < T.kb1; kb = next) {
                    next = kb + T.slot_blocks(kb);
                    const bool end = next == T.kb1 || (Cf::SEG && next == start + Cf::SEG);
                    if ((kb == start && !wait_warp(acce(acc.slot), acc.lap ^ 1u, bounds, kRoleMma, t)) ||
                        !wait_warp(full(at.slot), at.lap, bounds, kRoleMma, t)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    if (ptx::elect_one()) {
                        // (in a cluster the address has the CTA's rank above its 18 bits)
                        const uint32_t sp = ((ring0 + (uint32_t)(at.slot * Cf::STAGE)) & 0x3FFFFu) >> 4,
                                       sq = sp + Cf::P_BYTES / 16;
                        const uint32_t d = tmem + (uint32_t)(acc.slot * BN), first = kb == start ? 0u : 1u;
                        if (kb >= T.own) {
                            // low is K-major, the adapters' rows are N-major; 16 values of K for
                            // each 16 rows of the slots there are
                            const uint32_t pd = sp | ((kSwapped ? 512u : 1u) << 16), qd = sq | ((kSwapped ? 1u : 512u) << 16);
                            constexpr uint32_t ps = kSwapped ? 128u : 2u, qs = kSwapped ? 2u : 128u;
                            for (int k = kb; k < next; ++k) {
                                const int steps = min(4, ((T.slots << p.pitch_log2) - (k - p.num_kb) * kBlockK) / 16);
                                const uint32_t at_block = (uint32_t)((k - kb) * (Cf::BLOCK / 16));
                                for (int kk = 0; kk < steps; ++kk) {
                                    ptx::mma_f16_sw128<CG>(d, pd + at_block + ps * (uint32_t)kk, qd + at_block + qs * (uint32_t)kk,
                                                           p.idesc_add, kk != 0 || k != kb ? 1u : first);
                                    if (Cf::ADD_RESTS)
                                        ptx::mma_f16_sw128<CG>(d, pd + at_block + ps * (uint32_t)kk,
                                                               qd + at_block + qs * (uint32_t)kk + Cf::Q_ROWS * 128 / 16, p.idesc_add, 1u);
                                }
                            }
                        } else {
                            const uint32_t pd = sp | p_lead, qd = sq | q_lead;
#pragma unroll
                            for (int s = 0; s < kSlotBlocks; ++s) {
                                if (kb + s >= next) break;
                                const uint32_t at_block = (uint32_t)(s * (Cf::BLOCK / 16));
#pragma unroll
                                for (int kk = 0; kk < 4; ++kk)
                                    ptx::mma_f16_sw128<CG>(d, pd + at_block + p_step * kk, qd + at_block + q_step * kk, p.idesc,
                                                           kk != 0 || s != 0 ? 1u : first);
                                if constexpr (kGradient) {
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        ptx::mma_f16_sw128<CG>(d, pd + at_block + p_step * kk, qd + at_block + q_step * kk + Cf::Q_ONE / 16,
                                                               p.idesc, 1u);
                                }
                            }
                        }
                        if (kPair) ptx::mma_commit_pair(empty(at.slot), 0x3);
                        else ptx::mma_commit(empty(at.slot));
                        if (end) {
                            if (kPair) ptx::mma_commit_pair(accf(acc.slot), 0x3);
                            else ptx::mma_commit(accf(acc.slot));
                        }
                    }
                    __syncwarp();
                    last_bar = empty(at.slot);
                    last_parity = at.lap;
                    at.step();
                    if (end) {
                        acc.step();
                        start = next;
                    }
                }
            }
            if (*abort_flag && last_bar) wait_landed(last_bar, last_parity, p.timeout_ns);
        }
        __syncwarp();
    } else if (warp >= 4) {
        if constexpr (Cf::TAKE != 0) ptx::regs_take<Cf::TAKE>();
        // -------------------------------------------------------------- epilogue
        if (p.early) {
            ptx::pdl_wait();
            if (threadIdx.x == 128) ptx::pdl_launch_dependents();
        }
        const uint32_t quarter = warp & 3, half = (warp - 4) >> 2;     // lanes it may read; its columns
        const int row = (int)(quarter * 32 + lane), col0 = (int)half * Cf::COLS;
        const uint32_t tbase = tmem + (quarter << 21) + (uint32_t)col0;    // lane field: quarter * 32 << 16
        const uint32_t out_buf = out0 + (warp - 4) * (uint32_t)Cf::OUT_BYTES;
        const uint32_t acce_to = kPair ? ptx::mapa_shared(acce(0), 0) : acce(0);   // where accumulators are handed back
        Ring<2> acc;
        const float alpha = p.epi.alpha * (p.alpha ? __ldg(p.alpha) : 1.f);
        for (int t = unit; t < p.num_tiles; t += units) {
            const Tile T = tile_at<BN, Cf::ROWS, kSwapped>(p, t, crank);
            if (T.none) continue;
            const bool have = T.kb0 < T.kb1;         // (an empty sum is zero)
            if constexpr (EPI == kEpiStats) {
                const int64_t i0 = (int64_t)T.i0 + (int)(rank * kLanes + quarter * 32), i = i0 + lane;
                const int64_t j0 = (int64_t)T.j0 + col0;
                const bool live = i0 < T.i1 && j0 < T.j1;
                float v[Cf::COLS];
#pragma unroll
                for (int c = 0; c < Cf::COLS; ++c) v[c] = 0.f;
                bool ok = true;
                for (int kb = T.kb0; kb < T.kb1; kb += Cf::SEG) {
                    if (!(ok = wait_warp(accf(acc.slot), acc.lap, bounds, kRoleEpilogue, t))) break;
                    ptx::tc_fence_after();
                    const uint32_t src = tbase + (uint32_t)(acc.slot * BN), back = acce_to + 8u * (uint32_t)acc.slot;
                    if (live) add_columns<Cf::COLS>(src, v);
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (kPair) ptx::mbar_arrive_peer_if(back, lane == 0);
                    else ptx::mbar_arrive_if(back, lane == 0);
                    acc.step();
                }
                if (!ok) break;
                const int64_t part = (T.j0 / p.width * (BN / Cf::COLS) + (int)half) * (int64_t)p.I + i;
                if (!live) {
                    if (i < T.i1) {              // a last tile of few columns: nothing in this half
                        p.parts[part] = make_float2(-INFINITY, 0.f);
                        if (p.want_sum) p.sums[part] = 0.f;
                    }
                    continue;
                }
                Softmax soft;
                const int64_t label = i < T.i1 ? label_column(p, i) : -(1LL << 40);
#pragma unroll 1
                for (int s = 0; s < Cf::COLS / 64; ++s) {
                    const int64_t j = j0 + 64 * s;
                    if (j >= T.j1) break;
                    const int64_t rel = label - j;
                    const int place = rel >= 0 && rel < 64 && rel < T.j1 - j ? (int)rel : -1;
                    float hit = 0.f;
                    take_logits(p, v, T.j1 - j < 64 ? (int)(T.j1 - j) : 64, place, soft, hit);
                    if (place >= 0) p.hits[i] = hit;
#pragma unroll
                    for (int c = 0; c + 64 < Cf::COLS; ++c) v[c] = v[c + 64];
                }
                if (i < T.i1) {
                    p.parts[part] = make_float2(soft.top, soft.sum);
                    if (p.want_sum) p.sums[part] = soft.plain;
                }
                continue;
            }
            float side[4] = {0.f, 0.f, 0.f, 0.f};
            int own[kSwapped ? Cf::COLS / 4 : 1] = {};
            if constexpr (kSwapped) {
                if (p.splits == 1) {
                    side_of(p, T, (int64_t)T.i0 + (int)(quarter * 32) + 4 * (int)(lane & 7), side);
                    slots_of_rows<Cf::COLS>(p, T, col0, (int)lane, own);
                }
            }
            if (have && !wait_warp(accf(acc.slot), acc.lap, bounds, kRoleEpilogue, t)) break;
            ptx::tc_fence_after();
            const uint32_t src = tbase + (uint32_t)(acc.slot * BN), back = acce_to + 8u * (uint32_t)acc.slot;
            auto release = [&]() {
                ptx::tc_fence_before();
                __syncwarp();
                if (kPair) ptx::mbar_arrive_peer_if(back, lane == 0);
                else ptx::mbar_arrive_if(back, lane == 0);
            };
            if constexpr (kSwapped) {
                float v[Cf::COLS];
                if (have) {
                    constexpr int kPart = Cf::COLS < 32 ? 16 : 32;
                    uint32_t r[Cf::COLS / kPart][kPart];
#pragma unroll
                    for (int c = 0; c < Cf::COLS / kPart; ++c) ptx::tmem_load(src + (uint32_t)(c * kPart), r[c]);
#pragma unroll
                    for (int c = 0; c < Cf::COLS / kPart; ++c) {
                        ptx::tmem_wait(r[c]);
#pragma unroll
                        for (int k = 0; k < kPart; ++k) v[c * kPart + k] = __uint_as_float(r[c][k]);
                    }
                    release();
                    acc.step();
                } else {
#pragma unroll
                    for (int c = 0; c < Cf::COLS; ++c) v[c] = 0.f;
                }
                if (p.splits > 1) {
                    // this CTA's K range of the tile, for the cluster to read: [column][lane]
                    float *part = reinterpret_cast<float *>(ring);
#pragma unroll
                    for (int c = 0; c < Cf::COLS; ++c) part[(col0 + c) * kLanes + row] = v[c];
                    break;                                   // one tile a cluster
                }
                write_swapped<Cf::COLS>(p, T, (int)(quarter * 32), col0, v, side, own, out_buf, (int)lane);
            } else {
                const int64_t i0 = (int64_t)T.i0 + (int)(rank * kLanes + quarter * 32), i = i0 + lane;
                const int64_t j0 = (int64_t)T.j0 + col0;
                // steps of 64 columns that hold anything of C
                int steps = i0 < T.i1 && j0 < T.j1 ? (int)((T.j1 - j0 + 63) / 64 < Cf::COLS / 64 ? (T.j1 - j0 + 63) / 64 : Cf::COLS / 64) : 0;
                if (steps == 0 && have) release();
                float4 info = make_float4(0.f, 0.f, 0.f, 0.f);
                int64_t label = -(1LL << 40);
                if constexpr (EPI == kEpiDlogits) {
                    if (steps && i < T.i1) {
                        info = __ldg(p.rows + i);
                        if (info.w != 0.f) label = label_column(p, i);
                    }
                }
#pragma unroll 1
                for (int s = 0; s < steps; ++s) {
                    const int64_t j = j0 + 64 * s;
                    float v[64];
                    if (have) {
                        load_64(src + (uint32_t)(64 * s), v);
                        if (s + 1 == steps) release();
                    } else {
#pragma unroll
                        for (int c = 0; c < 64; ++c) v[c] = 0.f;
                    }
                    if constexpr (EPI == kEpiDlogits) {
                        const int64_t rel = label - j;
                        // (a row without a label gives nothing, whatever its logits are)
                        if (__any_sync(0xffffffffu, info.w != 0.f))
                            take_gradient(p, v, info, rel >= 0 && rel < 64 ? (int)rel : -1);
                        if (info.w == 0.f) {
#pragma unroll
                            for (int c = 0; c < 64; ++c) v[c] = 0.f;
                        }
                        if (rel >= 0 && rel < 64) {
                            float d = 0.f;
#pragma unroll
                            for (int c = 0; c < 64; ++c) d = c == (int)rel ? v[c] : d;
                            d = rest_of(p, d);
                            p.rests_out[i] = d;
                        }
                    } else {
                        if constexpr (EPI == kEpiRests) {
                            if (T.down == 0) add_rests(p, T, i, j, (int)lane, v);
                        }
                        finish_row(p, T, i, j, alpha, v);
                    }
                    store_64(p, &tmC, T, i0, j, v, out_buf, (int)lane);
                }
                if (have) acc.step();
            }
        }
    } else {
        if constexpr (Cf::GIVE != 0) ptx::regs_give_back<Cf::GIVE>();
        if (p.early) ptx::pdl_wait();
    }

    // Before the CTA's shared memory goes, its TMA stores must have read it.
    if (warp >= 4 && lane == 0) ptx::bulk_wait_group_read<0>();
    // K ranges: every CTA of the cluster sums its share of the columns over all
    // of them, in their order, and writes it: rows of C, four neighbouring
    // elements a thread and step, two steps' loads in flight.
    if (kSwapped && p.splits > 1) {
        const bool writes = warp >= 4 && unit < p.num_tiles;
        Tile T = {};
        float side[4] = {0.f, 0.f, 0.f, 0.f};
        int64_t cc = 0;                                  // (a warp's lanes take a whole row of the tile)
        if (writes) {
            T = tile_at<BN, Cf::ROWS, kSwapped>(p, unit, crank);
            cc = (int64_t)T.i0 + 4 * (int)lane;
            side_of(p, T, cc, side);
        }
        __syncwarp();
        ptx::cluster_sync();
        if (writes && !T.none && *abort_flag == 0) {
            const int c0 = BN * crank / p.splits, quads = (BN * (crank + 1) / p.splits - c0) * (kLanes / 4);
            constexpr int kStep = Cf::EW * 32;
            for (int q = (int)threadIdx.x - 128; q < quads; q += 2 * kStep) {
                const int c = c0 + q / 32, d = c0 + min(q + kStep, quads - 1) / 32;
                const bool first = T.j0 + c < T.j1 && cc < T.i1, second = q + kStep < quads && T.j0 + d < T.j1 && cc < T.i1;
                const int own_c = p.mode == kModeLow && first ? __ldg(p.slot_of + T.j0 + c) : -1;
                const int own_d = p.mode == kModeLow && second ? __ldg(p.slot_of + T.j0 + d) : -1;
                const uint32_t at0 = ring0 + 4u * (uint32_t)(c * kLanes + 4 * (int)lane);
                const uint32_t at1 = ring0 + 4u * (uint32_t)(d * kLanes + 4 * (int)lane);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
                for (int s = 0; s < p.splits; ++s) {
                    const float4 x = ptx::ld_cluster_v4f(ptx::mapa_shared(at0, (uint32_t)s));
                    const float4 y = ptx::ld_cluster_v4f(ptx::mapa_shared(at1, (uint32_t)s));
                    v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
                    w = make_float4(w.x + y.x, w.y + y.y, w.z + y.z, w.w + y.w);
                }
                if (first) write_four(p, T, (int64_t)T.j0 + c, cc, v, side, own_c);
                if (second) write_four(p, T, (int64_t)T.j0 + d, cc, w, side, own_d);
            }
        }
        __syncwarp();
        ptx::cluster_sync();
    }
    ptx::tc_fence_before();
    if (kPair) {
        __syncwarp();
        ptx::cluster_sync();      // neither CTA of a pair leaves while the other may still signal it
    } else {
        __syncthreads();
    }
    ptx::tc_fence_after();
    if (warp == 1) ptx::tmem_dealloc<CG>(tmem, Cf::TMEM_COLS);
}

// ------------------------------------------------------------------- host ---
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// `count` matrices of rows x cols elements, in boxes of box_rows x 128 bytes.
int encode(CUtensorMap *map, const void *base, int type, int64_t rows, int64_t cols, int64_t ld, int box_rows,
           int64_t count = 0, int64_t stride = 0) {
    auto enc = tensor_map_encoder();
    if (!enc) return api_error(GEMM_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const int eb = op_type_bytes(type);
    // (the pitch of a single row, or the stride of a single matrix, is nobody's)
    if (rows <= 1) ld = op_round_up(cols, 16);
    if (count <= 1) stride = ld;
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)(count ? count : 1)};
    const cuuint64_t strides[2] = {(cuuint64_t)(ld * eb), (cuuint64_t)(stride * eb)};
    const cuuint32_t box[3] = {(cuuint32_t)(128 / eb), (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, type == GEMM_OUT_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : type == GEMM_OUT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                        : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           count ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return GEMM_OK;
    char msg[96];
    std::snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return api_error(GEMM_ERR_CUDA, msg);
}

struct Maps {
    CUtensorMap p, q, low, ad, c;
};

template <int BN, int CG, int EPI, int PROWS = kLanes>
int launch(const Maps &m, const ProductParams &p, int grid, cudaStream_t stream) {
    using Cf = Cfg<BN, CG, EPI, PROWS>;
    auto kern = product_kernel<BN, CG, EPI, PROWS>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3(Cf::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cf::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (CG == 2 || p.splits > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = CG == 2 ? 2u : (unsigned)p.splits;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (options_snapshot().pdl != 1) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    // The shared memory a kernel may have is set once a device, and again should a launch
    // find it unset (after a device reset): setting it takes 0.5 us of a 25 us call.
    static std::atomic<uint64_t> set{0};
    int dev = 0;
    cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    for (int again = 0;; ++again) {
        if (again || !(set.load(std::memory_order_relaxed) & bit)) {
            const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM);
            if (e != cudaSuccess) return op_launched("cudaFuncSetAttribute", e);
            set.fetch_or(bit, std::memory_order_relaxed);
            again = 1;
        }
        const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, m.p, m.q, m.low, m.ad, m.c, p);
        if (e == cudaErrorInvalidValue && !again) {
            cudaGetLastError();
            continue;
        }
        return op_launched("product launch", e);
    }
}

int launch_plan(const ProductPlan &pl, int epilogue, const Maps &m, const ProductParams &p, int grid, cudaStream_t stream) {
    if (epilogue == kEpiGradient) {
        if (pl.bn == 16) return launch<16, 1, kEpiGradient>(m, p, grid, stream);
        if (pl.bn == 32) return launch<32, 1, kEpiGradient>(m, p, grid, stream);
        if (pl.bn == 64) return launch<64, 1, kEpiGradient>(m, p, grid, stream);
        return launch<128, 1, kEpiGradient>(m, p, grid, stream);
    }
    if (epilogue == kEpiSwapped) {
        if (pl.bn == 16) return launch<16, 1, kEpiSwapped>(m, p, grid, stream);
        if (pl.bn == 32) return launch<32, 1, kEpiSwapped>(m, p, grid, stream);
        if (pl.bn == 64) return launch<64, 1, kEpiSwapped>(m, p, grid, stream);
        return launch<128, 1, kEpiSwapped>(m, p, grid, stream);
    }
    const bool pair = pl.cg == 2;
    if (epilogue == kEpiStats && pair && pl.p_rows == 32) return launch<256, 2, kEpiStats, 32>(m, p, grid, stream);
    if (epilogue == kEpiStats)
        return pair ? launch<256, 2, kEpiStats>(m, p, grid, stream) : launch<128, 1, kEpiStats>(m, p, grid, stream);
    if (epilogue == kEpiDlogits)
        return pair ? launch<256, 2, kEpiDlogits>(m, p, grid, stream) : launch<128, 1, kEpiDlogits>(m, p, grid, stream);
    if (epilogue == kEpiRests)
        return pair ? launch<256, 2, kEpiRests>(m, p, grid, stream) : launch<128, 1, kEpiRests>(m, p, grid, stream);
    return pair ? launch<256, 2, kEpiRows>(m, p, grid, stream) : launch<128, 1, kEpiRows>(m, p, grid, stream);
}

// D f32 (bit 4), A/B format (bits 7-9, 10-12: f16 0, bf16 1), A / B MN-major
// (bits 15, 16), N >> 3 (bits 17-22), M >> 4 (bits 24-28).
uint32_t idesc_of(int type, int bn, int cg, int p_mn, int q_mn) {
    const uint32_t fmt = type == GEMM_OUT_BF16 ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)p_mn << 15) | ((uint32_t)q_mn << 16) |
           ((uint32_t)(bn >> 3) << 17) | ((uint32_t)((kLanes * cg) >> 4) << 24);
}

int encode_operand(CUtensorMap *m, const ProductOperand &o, int type, int64_t K, int box_rows) {
    return o.mn ? encode(m, o.p, type, K, o.rows, o.ld, 64) : encode(m, o.p, type, o.rows, K, o.ld, box_rows);
}

}  // namespace

int64_t product_parts(const ProductPlan &plan, int64_t cols) {
    // (both kernels have two halves of epilogue warps)
    return 2 * op_cdiv(cols, plan.width ? plan.width : plan.bn);
}

// Tile of a product with the tokens (or whatever else there is much of) on the
// lanes, and (most_parts > 1) into how many K ranges its tiles go, by the rounds of
// tiles and a tile's pace, in us: 0.27 a K-block of a 256 x 256 pair (its MMAs) and
// 0.3 of 128 x 128 (its operands from L2), and 7 and 4 around the first and last tile
// (1000 x 1016 x 2056: 20.4 us in 16 pair tiles, 64 of 128 x 128 finish earlier).  K ranges are for few tiles over a long K; their FP32 sums are written and
// read again.
ProductPlan product_plan_rows(int64_t I, int64_t J, int64_t K, int sms, int most_parts) {
    const int64_t kb = op_cdiv(K, kBlockK);
    const Options opt = options_snapshot();
    ProductPlan best;
    double least = 0.;
    for (int cg = 2; cg >= 1; --cg) {
        if (opt.product_bn && opt.product_bn != 128 * cg) continue;
        const int64_t tiles = op_cdiv(I, 128 * cg) * op_cdiv(J, 128 * cg);
        for (int parts = 1; parts <= most_parts; ++parts) {
            if (parts > 1 && (kb < 8 * parts || (double)parts * I * J > 3.2e7)) break;
            const double rounds = (double)op_cdiv(tiles * parts, sms / cg);
            const double cost = rounds * (op_cdiv(kb, parts) * (cg == 2 ? 0.27 : 0.3) + 0.4) + (cg == 2 ? 7. : 4.) +
                                (parts > 1 ? 4. + (double)parts * I * J * 8. / 5e6 : 0.);
            if (best.bn && cost >= least) continue;
            least = cost;
            best.bn = 128 * cg;
            best.cg = cg;
            best.parts = parts;
        }
    }
    return best;
}

// Few tokens stream the weights: the widest tiles that still take as few rounds
// leave the last round no emptier than it must be (50021 x 2048: 196 tiles of 256
// columns on 76 pairs are 2.6 rounds run as 3; of 224 columns 2.9).
ProductPlan product_plan_stats(int64_t tokens, int64_t vocab, int64_t K, bool any, int sms) {
    ProductPlan pl = product_plan_rows(tokens, vocab, K, sms);
    const int forced = options_snapshot().product_bn;
    if (tokens <= 32 && forced != 128) {
        // (their ring holds nearly nothing but W: 5 x 50021 x 2048 42 us, in 128 columns 58)
        pl.bn = 256;
        pl.cg = 2;
        pl.p_rows = 32;
    }
    if (!any || tokens > 256) return pl;
    const int64_t units = sms / pl.cg, rounds = op_cdiv(op_cdiv(vocab, pl.bn), units);
    const int64_t width = op_round_up(op_cdiv(vocab, rounds * units), 32);
    pl.width = (int)std::min<int64_t>(std::max<int64_t>(width, pl.bn / 2 + 32), pl.bn);
    return pl;
}

// K ranges for `tiles` swapped tiles of bn columns, `kb` K-blocks each: as many as
// one round of clusters takes (a second round costs more than the ranges give:
// 64 x 4096 x 12288 in 2 ranges 54 us, whole 41), while each has two slots' worth.
// Measured at 64 x 4096 x 8192: whole 33 us, 2 ranges 29; 48 x 4096 x 4096: 35, 29,
// 28 and 27 in 1 to 4.
static ProductPlan plan_splits(int bn, int64_t tiles, int64_t kb, int sms) {
    const int forced = options_snapshot().product_splits;
    ProductPlan best;
    best.bn = bn;
    for (int splits = 2; splits <= 4; ++splits)
        if (kb >= 4 * splits && (forced ? forced == splits : tiles * splits <= sms)) best.splits = splits;
    return best;
}

// A product with the tokens on the columns.
ProductPlan product_plan_tokens(int64_t tokens, int64_t cols, int64_t K, int sms) {
    const int bn = tokens <= 16 ? 16 : tokens <= 32 ? 32 : tokens <= 64 ? 64 : 128;
    return plan_splits(bn, op_cdiv(cols, kLanes) * op_cdiv(tokens, bn), op_cdiv(K, kBlockK), sms);
}

// The rank-wide activations: 64 tokens a tile, so that a prompt's tiles fill the SMs
// although each has few slots (8192 x 4096: 20 us; tiles of 128 in 2 K ranges 24).
ProductPlan product_plan_low(int64_t tokens, int64_t lanes, int64_t K, int sms) {
    const int bn = tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64;
    return plan_splits(bn, op_cdiv(lanes, kLanes) * op_cdiv(tokens, bn), op_cdiv(K, kBlockK), sms);
}

// The adapters' gradients: one tile is an adapter's rank wide.
ProductPlan product_plan_gradient(int64_t pitch, int64_t adapters, int64_t cols, int64_t tokens, int sms) {
    return plan_splits((int)pitch, op_cdiv(cols, kLanes) * adapters, op_cdiv(tokens, kBlockK), sms);
}

int product_launch(const ProductCall &c, int sms, cudaStream_t stream) {
    const int64_t kMax = 0x7fffffffLL - 512;
    const ProductPlan &pl = c.plan;
    const bool swapped = c.epilogue == kEpiSwapped || c.epilogue == kEpiGradient;
    ProductParams p = {};
    p.mode = c.mode;
    p.I = (int)c.I;
    p.J = (int)c.J;
    p.num_kb = (int)op_cdiv(c.K, kBlockK);
    p.group_i = pl.cg == 2 ? 8 : 16;
    p.splits = pl.splits;
    p.k_parts = std::max(1, pl.parts);
    p.part_rows = p.k_parts > 1 ? (int)c.part_rows : 0;
    const ProductAdapters &ad = c.ad;
    p.width = pl.width ? pl.width : pl.bn;
    int64_t ti = op_cdiv(c.I, kLanes * pl.cg), tj = op_cdiv(c.J, p.width);
    if (c.mode == kModeGradient) tj = ad.count;      // (an adapter's rank is one tile wide)
    p.tiles_first = 0x7fffffff;
    int64_t more = 0;                                // tiles of the second product
    if (c.two) {
        p.tiles_first = (int)std::min<int64_t>(ti * tj, kMax);
        p.num_kb2 = (int)op_cdiv(c.second_k, kBlockK);
        p.I2 = (int)(c.mode == kModeLow ? c.I : c.second_k);
        p.tiles_i2 = (int)op_cdiv(p.I2, kLanes);
        p.C2 = c.C2;
        p.ldc2 = c.ldc2;
        p.c_stride2 = c.c_stride2;
        p.wide2 = op_wide(c.C2, c.ldc2, 2) && (c.c_stride2 * 2) % 16 == 0;
        more = p.tiles_i2 * tj;
    }
    if ((ti * tj * p.k_parts + more) * pl.splits > kMax || (int64_t)p.k_parts * p.part_rows > kMax) return api_error(GEMM_ERR_INVALID_ARG, "too many tiles");
    p.tiles_i = (int)ti;
    p.tiles_j = (int)tj;
    p.num_tiles = (int)(ti * tj * p.k_parts + more);
    if (p.num_tiles == 0) return GEMM_OK;
    p.p_mn = c.p.mn;
    p.q_mn = c.q.mn;
    p.idesc = idesc_of(c.type, p.width, pl.cg, p.p_mn, p.q_mn);
    p.idesc_add = idesc_of(c.type, pl.bn, pl.cg, swapped ? 1 : 0, swapped ? 0 : 1);
    p.C = c.C;
    p.ldc = c.ldc;
    p.c_stride = c.c_stride;
    p.epi = c.epi;
    p.alpha = c.alpha;
    p.old = c.old;
    p.ld_old = c.ld_old;
    while ((1 << p.pitch_log2) < ad.pitch) ++p.pitch_log2;
    p.granule = ad.granule;
    p.granule_blocks = ad.granule < kBlockK ? 1 : ad.granule / kBlockK;
    p.max_slots = ad.max_slots;
    p.adapters = (int)ad.count;
    p.slots = ad.slots;
    p.counts = ad.counts;
    p.slot_of = ad.slot_of;
    p.lists = ad.lists;
    p.list_counts = ad.list_counts;
    p.granules = ad.granules;
    p.scales = ad.scales;
    p.rest = ad.rest;
    p.labels = c.loss.labels;
    p.label_bytes = c.loss.label_bytes;
    p.first = c.loss.first;
    p.softcap = c.loss.softcap;
    p.inv_softcap = c.loss.softcap != 0.f ? 1.f / c.loss.softcap : 0.f;
    p.want_sum = c.loss.want_sum;
    p.parts = c.loss.parts;
    p.sums = c.loss.sums;
    p.hits = c.loss.hits;
    p.rows = c.loss.rows;
    p.rests_out = c.loss.rests;
    p.rests = c.rests;
    p.f16 = c.type == GEMM_OUT_F16;
    p.eps_v = c.loss.eps_v;
    p.one_eps = c.loss.one_eps;
    p.early = c.early ? 1 : 0;
    const Options opt = options_snapshot();
    p.timeout_ns = (unsigned long long)opt.wait_timeout_ms * 1000000ull;
    p.debug_stall = opt.debug_stall_mma;

    Maps m;
    std::memset(&m, 0, sizeof m);
    int rc = GEMM_OK;
    const int64_t low_cols = (int64_t)ad.max_slots * ad.pitch, both = ad.rest ? 2 : 1;
    if (c.mode == kModeGradient) {
        rc = encode_operand(&m.p, c.p, c.type, c.K, kLanes);
        if (rc == GEMM_OK) rc = encode(&m.low, ad.low, c.type, c.K, low_cols, ad.ld_low, 64, both, ad.rest);
        if (rc == GEMM_OK && more) {
            rc = encode_operand(&m.q, c.second, c.type, c.K, kLanes);
            if (rc == GEMM_OK) rc = encode(&m.ad, c.ad2.low, c.type, c.K, low_cols, ad.ld_low, 64, both, ad.rest);
        }
    } else if (p.num_kb > 0) {
        if (c.mode != kModeLow) rc = encode_operand(&m.p, c.p, c.type, c.K, pl.p_rows);
        if (rc == GEMM_OK) rc = encode_operand(&m.q, c.q, c.type, c.K, p.width / pl.cg);
    }
    if (rc == GEMM_OK && c.mode == kModeLow && p.num_kb > 0)
        rc = encode(&m.ad, ad.p, c.type, ad.rank, ad.cols, ad.ld, ad.pitch, ad.count, ad.stride);
    if (rc == GEMM_OK && c.mode == kModeLow && c.two && p.num_kb2 > 0) {
        rc = encode_operand(&m.p, c.second, c.type, c.second_k, pl.bn);
        if (rc == GEMM_OK) rc = encode(&m.c, c.ad2.p, c.type, ad.rank, c.ad2.cols, c.ad2.ld, ad.pitch, ad.count, c.ad2.stride);
    }
    if (rc == GEMM_OK && c.mode == kModeAdd) {
        rc = encode(&m.ad, ad.p, c.type, ad.rank, ad.cols, ad.ld, std::min(ad.pitch, kBlockK), ad.count, ad.stride);
        if (rc == GEMM_OK)
            rc = encode(&m.low, ad.low, c.type, swapped ? c.J : c.I, low_cols, ad.ld_low, swapped ? pl.bn : kLanes, both, ad.rest);
    }
    if (rc) return rc;
    if (c.epilogue != kEpiStats) {
        const int ob = op_type_bytes(p.epi.out);
        p.wide = op_wide(c.C, c.ldc, ob) && (c.c_stride * ob) % 16 == 0;
        const int64_t cols = c.padded ? op_round_up(c.J, 64) : c.J;
        p.tma_store = !swapped && p.wide && (cols * ob) % 16 == 0;
        const int64_t rows = p.k_parts > 1 ? (int64_t)p.k_parts * p.part_rows : c.I;
        if (p.tma_store && (rc = encode(&m.c, c.C, p.epi.out, rows, cols, c.ldc, 32))) return rc;
    }
    const int64_t units = std::min<int64_t>(p.num_tiles, pl.splits > 1 ? p.num_tiles : sms / pl.cg);
    return launch_plan(pl, c.epilogue, m, p, (int)(units * pl.cg * pl.splits), stream);
}

cudaError_t project_read_and_clear_status(uint32_t words[4]) {
    cudaError_t e = cudaMemcpyFromSymbol(words, g_project_status, sizeof(uint32_t) * 4);
    if (e != cudaSuccess || words[0] == 0) return e;
    static const uint32_t zero[4] = {0, 0, 0, 0};
    return cudaMemcpyToSymbol(g_project_status, zero, sizeof zero);
}

}  // namespace tcgemm
