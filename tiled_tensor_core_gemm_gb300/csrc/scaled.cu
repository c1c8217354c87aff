// Products of FP8 matrices with a scale for each block of 128 along K:
//
//   D[i][j] = sum_kb sp(i, kb) * sq(j, kb) * sum_{k in kb} P[i][k] * Q[j][k]
//
// for one pair of matrices (gemm_run_scaled) or one per expert
// (gemm_run_experts).  P is the operand whose rows become Tensor Memory lanes,
// Q the one whose rows become its columns.  With many rows of C, P is A and Q
// is B^T; with few (a decode step) the roles are swapped, so that the 128 lanes
// carry the weights' rows and a tile is only as wide as the tokens there are:
// the MMA, the shared memory and the registers then go with the tokens, and the
// kernel streams the weights.
//
// The scales change every 128 values of K, so an MMA may sum over one K-block
// only: four MMAs of K = 32 write a fresh accumulator, and epilogue warps add
// it, scaled, to sums kept in registers.  NBUF accumulators rotate, so the MMAs
// of the next blocks run meanwhile.
//
// What bounds it (GB300, 8192^3 in 256 x 256 tiles on CTA pairs, 450 to 482 us
// over runs = 2.3 to 2.4 PFLOP/s, 59 to 64% of the FP8 rate): the epilogue
// warps.  Per K-block of 128 x 256 the MMAs take 520 cycles of an SM back to back and the kernel 850 to 900: of an
// epilogue warp's own 850, about 100 to find the MMAs complete, 270 to read the
// accumulator (two loads of 32 columns in flight), 260 for the multiply-adds (two
// warps a scheduler, 128 cycles each), the rest hand-over and lookups, each of
// which waits on shared memory that the MMAs and TMA keep busy.  Without the
// multiply-adds the same loop runs at 350 us, without reading the accumulator too
// at 337, next to 320 for the unscaled FP8 product.  The registers hold no third
// load and no more warps; a longer loop does not fit the instruction caches (two
// K-blocks unrolled: 690 us).  With a scale per column (the weight gradient) the
// multiplies by it and their loads from shared memory add half as much again.
// Few tokens stream the weights: 8 x 8192 x 8192 takes 16 us by graph replay
// against 9.9 of HBM, in two K ranges of 64 tiles.
//
// Roles: warp 0 issues the TMA loads of P and Q into a ring; warp 1 the MMAs;
// with a scale per column, warp 2 brings the lanes' scales and warp 3 the
// columns' into shared memory; the other warps hold the sums, one lane a thread,
// and write C.  Both operands are read in either major: K-major as rows of 128
// bytes, or MN-major in chunks of 128 rows of K by 128 bytes (as tc_gemm.cu reads
// B).  Every wait is bounded (a time limit, and a flag that any role raises when
// it gives up); a role that gives up waits, again bounded, for what it started.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "epilogue.cuh"
#include "ops.h"
#include "ptx.cuh"
#include "ptx_ops.cuh"

namespace tcgemm {

__device__ uint32_t g_scaled_status[4];

namespace {

constexpr int kLanes = 128;
constexpr int kBlockK = 128;
constexpr int kSmemMax = 232448;
constexpr int kCtrlBytes = 1024;       // barriers and flags
constexpr int kMaxExperts = 1024;
constexpr int kGroup = 4;              // K-blocks whose scales come together
constexpr int kSlots = 2;
constexpr int kBoxBytes = 4096;        // 32 rows x 128 bytes of C

enum Role : uint32_t { kRoleProducer = 1, kRoleMma = 2, kRoleEpilogue = 3, kRoleDrain = 4, kRoleScales = 5 };

struct ScaleView {
    const float *p;
    int64_t stride_k, stride_i, stride_e;
    int shift;                 // 7: one for 128 rows, 0: one each
};

struct ScaledParams {
    int I, J;                  // rows of P, rows of Q (experts: of the weights' side; the tokens' side is `rows`)
    int num_kb;
    int tiles_i, tiles_j;      // experts: of the weights' side
    int group_i;               // raster: lane tiles taken together
    int splits;                // CTAs of a cluster that share a tile's K
    int kb_per_split;
    int p_mn, q_mn;            // operands stored MN-major
    uint32_t idesc;
    ScaleView sp, sq;
    void *C;
    int64_t ldc;
    int swapped;               // P is B^T: C's columns are D's rows
    int wide;                  // C's rows start on 16 bytes
    int tma_store;             // and end on them: whole boxes leave by TMA
    int debug_stall;           // test hook: the MMA warp first waits for what cannot come
    EpiParams epi;
    const int32_t *offsets;    // experts: rows of each
    int experts, rows;         // 0: one product
    int tokens_on_i;           // experts: the token rows are D's rows
    unsigned long long timeout_ns;
};

template <int BN, bool QVEC, int EW, int CG>
struct Cfg {
    static constexpr int ROWS = kLanes * CG;          // D's rows of a tile (a CTA's share is 128)
    static constexpr int COLS = BN / (EW / 4);        // columns of a thread
    static constexpr int CHUNK = COLS < 32 ? COLS : 32;
    static constexpr int THREADS = 128 + EW * 32;
    // Registers a thread after the first warpgroup has given some up (0: as launched).
    static constexpr int GIVE = THREADS == 512 ? 56 : COLS > 64 ? (QVEC ? 72 : 56) : 0;
    static constexpr int TAKE = THREADS == 512 ? 152 : COLS > 64 ? (QVEC ? 216 : 224) : 0;
    static constexpr int LAUNCH = THREADS == 512 ? 128 : 168;         // what __launch_bounds__ leaves them
    static constexpr int P_BYTES = kLanes * 128;
    static constexpr int Q_BYTES = BN / CG * 128;     // each CTA of a pair loads half of Q's rows
    static constexpr int STAGE = P_BYTES + Q_BYTES;
    static constexpr int NBUF = BN > 128 ? 2 : 4;
    static constexpr int TMEM_COLS = BN >= 128 ? 512 : NBUF * BN;     // a power of two, at least 32
    static constexpr bool SWAPPED = BN < 128;          // the tiles of few tokens
    static constexpr int OUT_BYTES = SWAPPED ? 2048 : 2 * kBoxBytes;  // a warp's staging for C
    // With a scale per column, scales come four K-blocks at a time in two slots of
    // shared memory: for each K-block the lanes' 128 and the columns' BN.
    static constexpr int SCALES = QVEC ? kLanes + BN : 0;     // floats of a K-block
    static constexpr int SLOT_BYTES = kGroup * SCALES * 4;
    static constexpr int FIXED = 1024 + kCtrlBytes + kSlots * SLOT_BYTES + EW * OUT_BYTES + 2 * (kMaxExperts + 1) * 4 + 32;
    static constexpr int FIT = (kSmemMax - FIXED) / STAGE;
    static constexpr int STAGES = FIT >= 8 ? 8 : 4;                   // a power of two
    static constexpr int SMEM = FIXED + STAGES * STAGE;
    static_assert(GIVE == 0 || 128 * GIVE + EW * 32 * TAKE <= THREADS * LAUNCH, "the shares exceed the launch's registers");
    static_assert(STAGES <= FIT && SMEM <= kSmemMax, "ring");
    static_assert((2 * STAGES + NBUF + 2 * kSlots) * 8 + 16 <= kCtrlBytes, "barrier area");
    static_assert(!SWAPPED || kLanes * BN * 4 <= STAGES * STAGE, "a tile's partial sums fit in the ring");
};

__device__ __noinline__ void record_failure(uint32_t role, int tile, volatile int *abort_flag) {
    *abort_flag = 1;
    if (atomicCAS(&g_scaled_status[0], 0u, (uint32_t)GEMM_ERR_TIMEOUT) == 0u) {
        g_scaled_status[1] = role;
        g_scaled_status[2] = (uint32_t)tile;
        g_scaled_status[3] = blockIdx.x;
        __threadfence();
    }
}

// What bounds every wait of a CTA.
struct Bounds {
    volatile int *abort_flag;
    unsigned long long timeout_ns;
};

// A whole warp waits for a phase of a barrier (each try already waits a while).
// False once the time is up or another role has given up.  Kept short, for the
// loops around it have to stay in the instruction caches, and inline, for a call
// would have the epilogue warps put their sums away.
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

// A position in rings of 2^k slots, as the number of steps taken: one register
// gives the slot and the parity of the lap in every ring that steps with it.
struct Steps {
    uint32_t n = 0;
    template <int SLOTS> __device__ __forceinline__ int slot() const {
        static_assert((SLOTS & (SLOTS - 1)) == 0, "a power of two");
        return (int)(n & (uint32_t)(SLOTS - 1));
    }
    template <int SLOTS> __device__ __forceinline__ uint32_t parity() const { return (n / (uint32_t)SLOTS) & 1u; }
};

// One output tile: D's rows [i0, i1) and columns [j0, j1) of expert e (0 outside
// an expert launch), in the coordinates of the operands' tensor maps.
struct Tile {
    int i0, i1, j0, j1, e;
};

// Tile t of the launch.  Down `group_i` lane tiles, then across the columns:
// tiles that run together share both operands' panels in L2.
template <int BN, int ROWS>
__device__ __forceinline__ Tile tile_at(const ScaledParams &p, const int32_t *first_tile, const int32_t *first_row,
                                        int t) {
    Tile T;
    int e = 0, tiles_i = p.tiles_i, tiles_j = p.tiles_j, r = t;
    if (p.experts) {
        int lo = 0, hi = p.experts - 1;       // the last expert whose first tile is at or before t
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (first_tile[mid] <= t) lo = mid;
            else hi = mid - 1;
        }
        e = lo;
        r = t - first_tile[e];
        const int rows = first_row[e + 1] - first_row[e];
        if (p.tokens_on_i) tiles_i = (rows + ROWS - 1) / ROWS;
        else tiles_j = (rows + BN - 1) / BN;
    }
    const int per = p.group_i * tiles_j, g = r / per, first = g * p.group_i;
    const int gi = min(p.group_i, tiles_i - first);
    const int in = r - g * per;
    const int ti = first + in % gi, tj = in / gi;
    T.e = e;
    T.i0 = ti * ROWS;
    T.j0 = tj * BN;
    T.i1 = p.I;
    T.j1 = p.J;
    if (p.experts) {
        if (p.tokens_on_i) {
            T.i0 += first_row[e];
            T.i1 = first_row[e + 1];
        } else {
            T.j0 += first_row[e];
            T.j1 = first_row[e + 1];
        }
    }
    return T;
}

// Where the scale of row i (clamped below `end`) in K-block kb of expert e is.
__device__ __forceinline__ const float *scale_of(const ScaleView &v, int i, int end, int kb, int e) {
    i = i < end ? i : end - 1;
    return v.p + kb * v.stride_k + (int64_t)(i >> v.shift) * v.stride_i + e * v.stride_e;
}

// acc += r * s (paired: two columns an instruction).
template <int N>
__device__ __forceinline__ void add_scaled(float *acc, const uint32_t (&r)[N], float s) {
    const float2 s2 = make_float2(s, s);
#pragma unroll
    for (int c = 0; c < N; c += 2) {
        const float2 v = make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1]));
        const float2 a = __ffma2_rn(v, s2, make_float2(acc[c], acc[c + 1]));
        acc[c] = a.x;
        acc[c + 1] = a.y;
    }
}

// acc += r * (s * column scale), the scales from shared memory.
template <int N>
__device__ __forceinline__ void add_scaled_columns(float *acc, const uint32_t (&r)[N], float s, uint32_t columns) {
    const float2 s2 = make_float2(s, s);
#pragma unroll
    for (int c = 0; c < N; c += 4) {
        const float4 q = ptx::ld_shared_v4f(columns + 4u * (uint32_t)c);
        const float2 t0 = __fmul2_rn(make_float2(q.x, q.y), s2), t1 = __fmul2_rn(make_float2(q.z, q.w), s2);
        const float2 a0 = __ffma2_rn(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), t0,
                                     make_float2(acc[c], acc[c + 1]));
        const float2 a1 = __ffma2_rn(make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), t1,
                                     make_float2(acc[c + 2], acc[c + 3]));
        acc[c] = a0.x;
        acc[c + 1] = a0.y;
        acc[c + 2] = a1.x;
        acc[c + 3] = a1.y;
    }
}

// One warp's share of a tile's scales: COUNT of them a K-block, of the rows base,
// base + 1, ..., kGroup K-blocks at a time.  The next group's loads are in flight
// while one is handed over where the registers hold both; a load takes about as
// long as a K-block's MMAs, and there are two slots.
template <int COUNT>
__device__ __forceinline__ bool bring_scales(const ScaleView &v, int base, int end, int e, int kb0, int kb1, int t,
                                             Steps &sl, uint8_t *slots, int slot_bytes, int kb_floats, uint32_t scf0,
                                             uint32_t sce0, const Bounds &bounds) {
    constexpr int PER = (COUNT + 31) / 32;
    const int lane = threadIdx.x & 31;
    constexpr bool kAhead = PER <= 4;
    float cur[kGroup][PER], nxt[kGroup][PER];
    auto load = [&](int kb) {
#pragma unroll
        for (int a = 0; a < kGroup; ++a)
#pragma unroll
            for (int c = 0; c < PER; ++c)
                nxt[a][c] = kb + a < kb1 && 32 * c + lane < COUNT ? __ldg(scale_of(v, base + 32 * c + lane, end, kb + a, e))
                                                                  : 0.f;
    };
    if (kAhead) load(kb0);
    for (int kb = kb0; kb < kb1; kb += kGroup) {
        if (!kAhead) load(kb);
#pragma unroll
        for (int a = 0; a < kGroup; ++a)
#pragma unroll
            for (int c = 0; c < PER; ++c) cur[a][c] = nxt[a][c];
        if (kAhead) load(kb + kGroup);
        if (!wait_warp(sce0 + 8u * (uint32_t)sl.slot<kSlots>(), sl.parity<kSlots>() ^ 1u, bounds, kRoleScales, t)) return false;
        float *slot = reinterpret_cast<float *>(slots + sl.slot<kSlots>() * slot_bytes);
#pragma unroll
        for (int a = 0; a < kGroup; ++a)
#pragma unroll
            for (int c = 0; c < PER; ++c)
                if (32 * c + lane < COUNT) slot[a * kb_floats + 32 * c + lane] = cur[a][c];
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(scf0 + 8u * (uint32_t)sl.slot<kSlots>());
        ++sl.n;
    }
    return true;
}

// x * Phi(x), two values at a time.  Phi(-a) = 2^-P(a) for a = |x| >= 0, P a
// polynomial of degree 8 fitted to -log2 Phi(-a) on [0, 5.5] (least squares in
// the Chebyshev basis, reweighted towards the largest error in Phi; 4e-8 in FP32
// arithmetic, where erf's own rounding leaves 6e-8) and above 25 beyond, where
// Phi(-a) no longer counts.  One exponential and eight paired multiply-adds,
// where erff takes about thirty instructions.
__device__ __forceinline__ float2 gelu2(float2 x) {
    const float2 a = make_float2(fabsf(x.x), fabsf(x.y));
    auto both = [](float c) { return make_float2(c, c); };
    float2 r = both(-2.7720716e-06f);                       // -P
    r = __ffma2_rn(r, a, both(3.8620983e-05f));
    r = __ffma2_rn(r, a, both(-1.8254861e-04f));
    r = __ffma2_rn(r, a, both(-1.4586786e-04f));
    r = __ffma2_rn(r, a, both(7.0754690e-03f));
    r = __ffma2_rn(r, a, both(-5.2505028e-02f));
    r = __ffma2_rn(r, a, both(-4.5920491e-01f));
    r = __ffma2_rn(r, a, both(-1.1511058e+00f));
    r = __ffma2_rn(r, a, both(-1.0f));
    const float hx = ptx::exp2_approx(r.x), hy = ptx::exp2_approx(r.y);
    return make_float2(x.x * (x.x > 0.f ? 1.f - hx : hx), x.y * (x.y > 0.f ? 1.f - hy : hy));
}

// The epilogue's value from a whole sum (old: the element of C before, if beta).
__device__ __forceinline__ float finish(const EpiParams &e, float acc, float old, float bias) {
    float y = e.alpha * acc;
    if (e.beta != 0.f) y = fmaf(e.beta, old, y);
    y += bias;
    if (e.act == GEMM_ACT_RELU) y = ptx::relu_nan(y);
    else if (e.act == GEMM_ACT_GELU) y = gelu2(make_float2(y, y)).x;
    return y;
}

// Writes four neighbouring columns of a row of C, [cr][cc .. cc + 4), where they
// exist.
__device__ __forceinline__ void write_four(const ScaledParams &p, int64_t cr, int64_t cc, int64_t c_end, float4 v,
                                           const float (&bias)[4]) {
    float y[4] = {v.x, v.y, v.z, v.w};
    const int64_t at = cr * p.ldc + cc;
    const bool whole = p.wide && cc + 4 <= c_end;
    if (p.epi.active) {
        float old[4] = {0.f, 0.f, 0.f, 0.f};
        if (p.epi.beta != 0.f) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (cc + k < c_end) old[k] = epi_load_old(p.C, at + k, p.epi.out);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = finish(p.epi, y[k], old[k], bias[k]);
    }
    if (whole && p.epi.active && p.epi.out != GEMM_OUT_F32) {
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.C) + at) =
            make_uint2(epi_pack2(p.epi.out, y[0], y[1]), epi_pack2(p.epi.out, y[2], y[3]));
    } else if (whole) {
        *reinterpret_cast<float4 *>(static_cast<float *>(p.C) + at) = make_float4(y[0], y[1], y[2], y[3]);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (cc + k < c_end) epi_store(p.C, at + k, p.epi.active ? p.epi.out : GEMM_OUT_F32, y[k]);
    }
}

// Swapped: a warp's 32 rows x COLS columns of D are COLS rows of 32 columns of
// C.  They go through 2 KB of shared memory, 16 rows of C at a time, so that
// eight lanes hold 32 neighbouring elements of a row and the epilogue's code is
// there once (unrolled over the sums it did not fit the instruction caches).
// The sums move down as they are written.
template <int COLS>
__device__ __forceinline__ void write_swapped(const ScaledParams &p, const Tile &T, int row0, int col0,
                                              float (&acc)[COLS], uint32_t buf, int lane) {
    const int u = lane & 7;
    const int64_t cc = (int64_t)T.i0 + row0 + 4 * u;
    float bias[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) bias[k] = cc + k < T.i1 ? epi_bias(p.epi, cc + k, cc + k + 1) : 0.f;
#pragma unroll 1
    for (int c0 = 0; c0 < COLS; c0 += 16) {
        const int64_t r0 = (int64_t)T.j0 + col0 + c0;
        if (r0 >= T.j1) break;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 16; ++c) ptx::st_shared_f(buf + 4u * (uint32_t)(c * 32 + lane), acc[c]);
        __syncwarp();
#pragma unroll 1
        for (int r = lane >> 3; r < 16 && r0 + r < T.j1; r += 4) {
            const float4 v = ptx::ld_shared_v4f(buf + 128u * (uint32_t)r + 16u * (uint32_t)u);
            if (cc < T.i1) write_four(p, r0 + r, cc, T.i1, v, bias);
        }
#pragma unroll
        for (int c = 0; c + 16 < COLS; ++c) acc[c] = acc[c + 16];
    }
}

// A warp's 32 rows x COLS columns of D as rows of C, one row a thread: 32
// columns at a time through the epilogue in registers (its code is there once;
// the sums move down), rounded, and into a box of 32 rows x 128 bytes of shared
// memory with TMA's 128-byte swizzle, two boxes in turn.  A full box leaves by a TMA store where
// C's layout allows it and the rows are all this tile's (an expert's last tile
// ends inside one), else row by row with neighbouring lanes on neighbouring
// columns.
template <int COLS>
__device__ __forceinline__ void write_rows(const ScaledParams &p, const CUtensorMap *tmC, const Tile &T, int row0,
                                           int col0, float (&acc)[COLS], uint32_t bufs, int &box, int lane) {
    const bool active = p.epi.active != 0;
    const bool half = active && p.epi.out != GEMM_OUT_F32;
    const int64_t i0 = (int64_t)T.i0 + row0, i = i0 + lane;
    const bool by_tma = p.tma_store && (!p.experts || i0 + 32 <= T.i1);
#pragma unroll 1
    for (int c0 = 0; c0 < COLS; c0 += 32) {
        const int64_t j = (int64_t)T.j0 + col0 + c0;
        if (i0 >= T.i1 || j >= T.j1) break;
        if (active) {
            if (p.epi.alpha != 1.f) {
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[c] *= p.epi.alpha;
            }
            if (p.epi.beta != 0.f && i < T.i1) {
                const int64_t at = i * p.ldc + j;
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    if (j + c < T.j1) acc[c] = fmaf(p.epi.beta, epi_load_old(p.C, at + c, p.epi.out), acc[c]);
            }
            if (p.epi.bias) {
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[c] += j + c < T.j1 ? __ldg(p.epi.bias + j + c) : 0.f;
            }
            if (p.epi.act == GEMM_ACT_RELU) {
#pragma unroll
                for (int c = 0; c < 32; ++c) acc[c] = ptx::relu_nan(acc[c]);
            } else if (p.epi.act == GEMM_ACT_GELU) {
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float2 g = gelu2(make_float2(acc[c], acc[c + 1]));
                    acc[c] = g.x;
                    acc[c + 1] = g.y;
                }
            }
        }
        // a new box, in the buffer of the one before last, which its store must have read
        const bool first = !half || (c0 & 32) == 0;
        if (first) {
            ++box;
            if (lane == 0) ptx::bulk_wait_group_read<1>();
            __syncwarp();
        }
        const uint32_t buf = bufs + (uint32_t)((box & 1) * kBoxBytes);
        const uint32_t row = buf + 128u * (uint32_t)lane;
        if (half) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t unit = (uint32_t)((u + (first ? 0 : 4)) ^ (lane & 7));
                ptx::st_shared_v4(row + 16u * unit,
                                  make_uint4(epi_pack2(p.epi.out, acc[8 * u], acc[8 * u + 1]),
                                             epi_pack2(p.epi.out, acc[8 * u + 2], acc[8 * u + 3]),
                                             epi_pack2(p.epi.out, acc[8 * u + 4], acc[8 * u + 5]),
                                             epi_pack2(p.epi.out, acc[8 * u + 6], acc[8 * u + 7])));
            }
        } else {
#pragma unroll
            for (int u = 0; u < 8; ++u)
                ptx::st_shared_v4f(row + 16u * (uint32_t)(u ^ (lane & 7)),
                                   make_float4(acc[4 * u], acc[4 * u + 1], acc[4 * u + 2], acc[4 * u + 3]));
        }
        const bool last = !half || (c0 & 32) != 0 || j + 32 >= T.j1;
        if (last) {
            const int64_t jb = first ? j : j - 32;          // the box's first column
            if (by_tma) {
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    ptx::tma_store_2d(tmC, buf, (int)jb, (int)i0);
                    ptx::bulk_commit_group();
                }
            } else {
                __syncwarp();
                const int rows = T.i1 - i0 < 32 ? (int)(T.i1 - i0) : 32;
                const int cols = (int)(T.j1 - jb < (half ? 64 : 32) ? T.j1 - jb : (half ? 64 : 32));
#pragma unroll 2
                for (int r = 0; r < rows; ++r) {
                    const uint32_t from = buf + 128u * (uint32_t)r;
                    const int64_t at = (i0 + r) * p.ldc + jb + lane;
                    const uint32_t sw = (uint32_t)(r & 7) << 4;
                    if (half) {
                        uint16_t *d = static_cast<uint16_t *>(p.C) + at;
                        if (lane < cols) d[0] = ptx::ld_shared_u16(from + ((2u * (uint32_t)lane) ^ sw));
                        if (lane + 32 < cols) d[32] = ptx::ld_shared_u16(from + ((2u * (uint32_t)lane + 64u) ^ sw));
                    } else if (lane < cols) {
                        static_cast<float *>(p.C)[at] = ptx::ld_shared_f(from + ((4u * (uint32_t)lane) ^ sw));
                    }
                }
                // (an empty group, so that groups count boxes whichever way they left)
                if (lane == 0) ptx::bulk_commit_group();
                __syncwarp();
            }
        }
#pragma unroll
        for (int c = 0; c + 32 < COLS; ++c) acc[c] = acc[c + 32];
    }
}

template <int BN, bool QVEC, int EW, int CG>
__global__ void __launch_bounds__((Cfg<BN, QVEC, EW, CG>::THREADS), 1)
scaled_kernel(const __grid_constant__ CUtensorMap tmP, const __grid_constant__ CUtensorMap tmQ,
              const __grid_constant__ CUtensorMap tmC, const ScaledParams p) {
    using Cf = Cfg<BN, QVEC, EW, CG>;
    constexpr bool kPair = CG == 2;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = ptx::smem_addr(smem_raw);
    uint8_t *ring = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
    uint8_t *out_bufs = ring + Cf::STAGES * Cf::STAGE;          // 1024-byte aligned, as the ring's slots are
    uint64_t *bars = reinterpret_cast<uint64_t *>(out_bufs + EW * Cf::OUT_BYTES);
    uint8_t *scales = reinterpret_cast<uint8_t *>(bars) + kCtrlBytes;
    int32_t *first_tile = reinterpret_cast<int32_t *>(scales + kSlots * Cf::SLOT_BYTES);
    int32_t *first_row = first_tile + kMaxExperts + 1;
    constexpr int kBars = 2 * Cf::STAGES + Cf::NBUF + 2 * kSlots;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + kBars);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    const Bounds bounds = {abort_flag, p.timeout_ns};

    const uint32_t bar0 = ptx::smem_addr(bars);
    auto full = [&](int s) { return bar0 + 8u * (uint32_t)s; };
    auto done = [&](int s) { return bar0 + 8u * (uint32_t)(Cf::STAGES + s); };    // the MMAs of a stage have completed
    auto acce = [&](int b) { return bar0 + 8u * (uint32_t)(2 * Cf::STAGES + b); };
    auto scf = [&](int s) { return bar0 + 8u * (uint32_t)(2 * Cf::STAGES + Cf::NBUF + s); };
    auto sce = [&](int s) { return bar0 + 8u * (uint32_t)(2 * Cf::STAGES + Cf::NBUF + kSlots + s); };
    const uint32_t ring0 = ptx::smem_addr(ring), scales0 = ptx::smem_addr(scales), out0 = ptx::smem_addr(out_bufs), scf0 = scf(0), sce0 = sce(0);

    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = Cf::SWAPPED && p.splits > 1 ? ptx::cluster_ctarank() : 0u;   // its K range
    const uint32_t rank = kPair ? ptx::cluster_ctarank() : 0u;                     // its half of the pair's tile

    if (threadIdx.x == 0) {
        for (int s = 0; s < Cf::STAGES; ++s) {
            ptx::mbar_init(full(s), 1);
            ptx::mbar_init(done(s), 1);
        }
        for (int b = 0; b < Cf::NBUF; ++b) {
            ptx::mbar_init(acce(b), EW * CG);
        }
        for (int s = 0; s < kSlots; ++s) {
            ptx::mbar_init(scf(s), 2);       // the scale warps
            ptx::mbar_init(sce(s), EW);
        }
        *abort_flag = 0;
        ptx::fence_mbar_init();
        if (p.num_kb > 0) {
            ptx::prefetch_tensormap(&tmP);
            ptx::prefetch_tensormap(&tmQ);
        }
        if (p.tma_store) ptx::prefetch_tensormap(&tmC);
    }
    if (warp == 1) {
        ptx::tmem_alloc<CG>(ptx::smem_addr(tmem_slot), Cf::TMEM_COLS);
        ptx::tmem_relinquish<CG>();
    }
    // Global memory from here on: the previous kernel on the stream is done.
    ptx::pdl_wait();
    if (threadIdx.x == 0) ptx::pdl_launch_dependents();
    if (p.experts && warp == 2) {
        // The experts' first rows and first tiles.  Offsets are clamped to
        // ascending values within [0, rows].
        int32_t row = 0, tile = 0;
        for (int e0 = 0; e0 <= p.experts; e0 += 32) {
            const int e = e0 + (int)lane;
            int32_t o = e <= p.experts ? min(max(p.offsets[e], 0), p.rows) : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, o, d);
                if ((int)lane >= d) o = max(o, y);
            }
            o = max(o, row);
            if (e <= p.experts) first_row[e] = o;
            int32_t before = __shfl_up_sync(0xffffffffu, o, 1);
            if (lane == 0) before = e0 ? row : o;
            // tiles of the expert that ends here (e - 1)
            const int n = e > 0 && e <= p.experts ? o - before : 0;
            int32_t c = p.tokens_on_i ? (n + Cf::ROWS - 1) / Cf::ROWS * p.tiles_j : (n + BN - 1) / BN * p.tiles_i;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int32_t y = __shfl_up_sync(0xffffffffu, c, d);
                if ((int)lane >= d) c += y;
            }
            c += tile;
            if (e <= p.experts) first_tile[e] = c;
            row = __shfl_sync(0xffffffffu, o, 31);
            tile = __shfl_sync(0xffffffffu, c, 31);
        }
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
    const int num_tiles = p.experts ? first_tile[p.experts] : p.tiles_i * p.tiles_j;
    const int share = kPair ? 2 : Cf::SWAPPED ? p.splits : 1;      // CTAs of a tile
    const int unit = (int)blockIdx.x / share, units = (int)gridDim.x / share;
    const int kb0 = (int)crank * p.kb_per_split, kb1 = min(p.num_kb, kb0 + p.kb_per_split);

    // 128 columns a thread need more than the launch's 168 registers: the first
    // warpgroup gives the difference (128 x 56 + 256 x 224 = 384 x 168; with
    // a scale per column, 256 of which a warp brings, 128 x 72 + 256 x 216).
    if (warp < 4) {
        if constexpr (Cf::GIVE != 0) ptx::regs_give_back<Cf::GIVE>();
        if (warp == 0) {
            // ------------------------------------------------------ TMA producer
            // (the whole warp, one elected thread issuing, as the MMA warp)
            Steps at;
            bool ok = true;
            for (int t = unit; ok && t < num_tiles; t += units) {
                const Tile T = tile_at<BN, Cf::ROWS>(p, first_tile, first_row, t);
                const int ep = p.tokens_on_i ? 0 : T.e, eq = p.tokens_on_i ? T.e : 0;
                const int i0 = T.i0 + (int)rank * kLanes, j0 = T.j0 + (int)rank * (BN / CG);
                for (int kb = kb0; kb < kb1; ++kb) {
                    if (!wait_warp(done(at.slot<Cf::STAGES>()), at.parity<Cf::STAGES>() ^ 1u, bounds, kRoleProducer, t)) {
                        ok = false;
                        break;
                    }
                    if (ptx::elect_one()) {
                        const int stage = at.slot<Cf::STAGES>();
                        const uint32_t fb = full(stage), sp = ring0 + (uint32_t)(stage * Cf::STAGE), sq = sp + Cf::P_BYTES;
                        if (rank == 0) ptx::mbar_arrive_expect_tx(fb, (uint32_t)(Cf::STAGE * CG));
                        const int k0 = kb * kBlockK;
                        const uint32_t to = kPair ? ptx::mapa_shared(fb, 0) : fb;     // a pair's bytes count in the leader
                        ptx::tma_load_3d<CG>(sp, &tmP, to, p.p_mn ? i0 : k0, p.p_mn ? k0 : i0, ep);
                        if (p.q_mn) {
#pragma unroll
                            for (int c = 0; c < (BN / CG + 127) / 128; ++c)
                                ptx::tma_load_3d<CG>(sq + c * 16384, &tmQ, to, j0 + c * 128, k0, eq);
                        } else {
                            ptx::tma_load_3d<CG>(sq, &tmQ, to, k0, j0, eq);
                        }
                    }
                    __syncwarp();
                    ++at.n;
                }
            }
            // Until the MMAs have released every slot no read of this shared
            // memory and no arrival on its barriers is outstanding.
            const uint32_t issued = at.n;
            for (int i = 0; ok && i < Cf::STAGES; ++i, ++at.n)
                ok = wait_warp(done(at.slot<Cf::STAGES>()), at.parity<Cf::STAGES>() ^ 1u, bounds, kRoleDrain, -1);
            // Given up: the copies already issued still land in this shared memory
            // (those of a pair are counted in the leader).
            for (uint32_t n = issued > Cf::STAGES ? issued - Cf::STAGES : 0; !ok && rank == 0 && n < issued; ++n) {
                const Steps one = {n};
                wait_landed(full(one.slot<Cf::STAGES>()), one.parity<Cf::STAGES>(), p.timeout_ns);
            }
            __syncwarp();
        } else if (warp == 1) {
            // -------------------------------------------------------- MMA issuer
            // The whole warp runs the loop and one elected thread issues: the
            // descriptors then stay in uniform registers (with a loop of one
            // thread the issue of a K-block took 650 cycles, more than its MMAs).
            // One commit a K-block serves both who waits for it: the producer,
            // for the stage, and the epilogue warps, for the accumulator.
            if (rank == 0) {
                Steps at;
                bool ok = true;
                uint32_t last_bar = 0, last_parity = 0;      // of the MMAs issued last
                // descriptors in 16-byte units: leading offset, and one MMA's step along K
                const uint32_t p_lead = (p.p_mn ? 1024u : 1u) << 16, q_lead = (p.q_mn ? 1024u : 1u) << 16;
                const uint32_t p_step = p.p_mn ? 256u : 2u, q_step = p.q_mn ? 256u : 2u;
                // (no accumulator is handed back before the first has been written; half
                // the limit, so that this wait and not one behind it runs out first)
                if (p.debug_stall) ok = wait_warp(acce(0), 0u, Bounds{abort_flag, p.timeout_ns / 2}, kRoleMma, unit);
                for (int t = unit; ok && t < num_tiles; t += units) {
                    for (int kb = kb0; kb < kb1; ++kb) {
                        const int stage = at.slot<Cf::STAGES>(), buf = at.slot<Cf::NBUF>();
                        if (!wait_warp(full(stage), at.parity<Cf::STAGES>(), bounds, kRoleMma, t) ||
                            !wait_warp(acce(buf), at.parity<Cf::NBUF>() ^ 1u, bounds, kRoleMma, t)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        if (ptx::elect_one()) {
                            // K-major: K advances 32 bytes inside a 128-byte row, 8-row
                            // groups 1024 bytes apart.  MN-major: 32 rows of K further,
                            // 128-byte chunks 16 KB apart, 8-row groups 1024.
                            const uint32_t sp = ring0 + (uint32_t)(stage * Cf::STAGE);
                            const uint32_t pd = (sp >> 4) | p_lead, qd = ((sp + Cf::P_BYTES) >> 4) | q_lead;
                            const uint32_t d = tmem + (uint32_t)(buf * BN);
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                ptx::mma_f8_sw128<CG>(d, pd + p_step * kk, qd + q_step * kk, p.idesc, kk != 0 ? 1u : 0u);
                            if (kPair) ptx::mma_commit_pair(done(stage), 0x3);
                            else ptx::mma_commit(done(stage));
                        }
                        __syncwarp();
                        last_bar = done(stage);
                        last_parity = at.parity<Cf::STAGES>();
                        ++at.n;
                    }
                }
                if (!ok && last_bar) wait_landed(last_bar, last_parity, p.timeout_ns);
            }
            __syncwarp();
        } else {
            // --------------------------------------- scales (with one per column)
            Steps sl;
            bool ok = QVEC;
            for (int t = unit; ok && t < num_tiles; t += units) {
                const Tile T = tile_at<BN, Cf::ROWS>(p, first_tile, first_row, t);
                if (warp == 2)
                    ok = bring_scales<kLanes>(p.sp, T.i0 + (int)rank * kLanes, T.i1, p.tokens_on_i ? 0 : T.e, kb0, kb1, t, sl,
                                              scales, Cf::SLOT_BYTES, Cf::SCALES, scf0, sce0, bounds);
                else
                    ok = bring_scales<BN>(p.sq, T.j0, T.j1, p.tokens_on_i ? T.e : 0, kb0, kb1, t, sl, scales + kLanes * 4,
                                          Cf::SLOT_BYTES, Cf::SCALES, scf0, sce0, bounds);
            }
        }
    } else {
        if constexpr (Cf::TAKE != 0) ptx::regs_take<Cf::TAKE>();
        // ------------------------------------------------- sums and epilogue
        const uint32_t quarter = warp & 3, half = (warp - 4) >> 2;     // lanes it may read; its columns
        const int row = (int)(quarter * 32 + lane), col0 = (int)half * Cf::COLS;   // of this CTA's 128
        const uint32_t tbase = tmem + (quarter << 21) + (uint32_t)col0;   // lane field: quarter * 32 << 16
        Steps at, sl;                                                  // K-blocks, and groups of them
        int box = 0;                                                   // of C, written so far
        // One scale for 128 columns: each thread reads its row's and the columns'
        // straight from memory, two K-blocks ahead.  In 192 columns a tile's first are
        // asked for before the epilogue of the one before (in 256 the registers they
        // hold there would be spilled: 463 -> 572 us at 8192^3, one run).
        constexpr bool kEarly = BN == 192;
        const float *row_at = nullptr, *col_at = nullptr;              // of the K-block two further
        float row_even = 0.f, col_even = 0.f, row_odd = 0.f, col_odd = 0.f;
        auto first_scales = [&](int t) {
            if (QVEC || t >= num_tiles || kb0 >= kb1) return;
            const Tile T = tile_at<BN, Cf::ROWS>(p, first_tile, first_row, t);
            row_at = scale_of(p.sp, T.i0 + (int)(rank * kLanes) + row, T.i1, kb0, p.tokens_on_i ? 0 : T.e);
            col_at = scale_of(p.sq, T.j0 + col0, T.j1, kb0, p.tokens_on_i ? T.e : 0);
            row_even = __ldg(row_at);
            col_even = __ldg(col_at);
            if (kb0 + 1 < kb1) {
                row_odd = __ldg(row_at += p.sp.stride_k);
                col_odd = __ldg(col_at += p.sq.stride_k);
            }
        };
        if (kEarly) first_scales(unit);
        const uint32_t acce_to = kPair ? ptx::mapa_shared(acce(0), 0) : acce(0);   // where accumulators are handed back
        bool ok = true;
        for (int t = unit; ok && t < num_tiles; t += units) {
            float acc[Cf::COLS];
#pragma unroll
            for (int c = 0; c < Cf::COLS; ++c) acc[c] = 0.f;
            // Scales.  One for 128 columns: see above.  One per column: through shared memory, where two warps bring them, the row's next one
            // looked up between handing the accumulator back and adding the last
            // columns (the group's end, needed until then, after them).
            bool ready = false;                                  // the next K-block's MMAs have completed
            float s_next = 0.f;
            const uint32_t row_scale = scales0 + 4u * (uint32_t)row;
            auto group_begins = [&]() {
                ok = wait_warp(scf(sl.slot<kSlots>()), sl.parity<kSlots>(), bounds, kRoleEpilogue, t) && ok;
            };
            auto group_ends = [&]() {
                __syncwarp();
                ptx::mbar_arrive_if(sce(sl.slot<kSlots>()), lane == 0);
                ++sl.n;
            };
            auto in_group = [&](int kb) { return (kb - kb0) % kGroup; };
            auto scale_offset = [&](int kb) {
                return (uint32_t)(sl.slot<kSlots>() * Cf::SLOT_BYTES + in_group(kb) * Cf::SCALES * 4);
            };
            auto next_scale = [&](int kb) {
                if (in_group(kb) == 0) {
                    group_ends();
                    group_begins();
                }
                s_next = ptx::ld_shared_f(row_scale + scale_offset(kb));
            };
            if (!kEarly) first_scales(t);
            if (QVEC && kb0 < kb1) {
                group_begins();
                s_next = ptx::ld_shared_f(row_scale + scale_offset(kb0));
            }
#pragma unroll 1
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!__all_sync(0xffffffffu, ready))
                    ok = wait_warp(done(at.slot<Cf::STAGES>()), at.parity<Cf::STAGES>(), bounds, kRoleEpilogue, t) && ok;
                if (!ok) break;
                ready = false;
                ptx::tc_fence_after();
                const int buf = at.slot<Cf::NBUF>();
                const uint32_t src = tbase + (uint32_t)(buf * BN), release = acce_to + 8u * (uint32_t)buf;
                // (a scale per column) the K-block's columns' scales
                const uint32_t columns = scales0 + scale_offset(kb) + 4u * (uint32_t)(kLanes + col0);
                float s = s_next;
                ++at.n;
                if (!QVEC) {
                    // even and odd K-blocks in registers of their own: a move from one to
                    // the other would wait for a load issued one K-block ago
                    auto take = [&](float &r_scale, float &c_scale) {
                        s = r_scale * c_scale;
                        if (kb + 2 < kb1) {
                            r_scale = __ldg(row_at += p.sp.stride_k);
                            c_scale = __ldg(col_at += p.sq.stride_k);
                        }
                    };
                    if ((kb - kb0) & 1) take(row_odd, col_odd);
                    else take(row_even, col_even);
                }
                // Two loads of 32 columns in flight; each is replaced by the one
                // two further as soon as it has been added.
                constexpr int kChunks = Cf::COLS / Cf::CHUNK;
                uint32_t r[2][Cf::CHUNK];
                auto add = [&](int c) {
                    if (QVEC)
                        add_scaled_columns<Cf::CHUNK>(acc + c * Cf::CHUNK, r[c & 1], s,
                                                      columns + 4u * (uint32_t)(c * Cf::CHUNK));
                    else
                        add_scaled<Cf::CHUNK>(acc + c * Cf::CHUNK, r[c & 1], s);
                };
                ptx::tmem_load(src, r[0]);
                if (kChunks > 1) ptx::tmem_load(src + (uint32_t)Cf::CHUNK, r[1]);
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) {
                    ptx::tmem_wait(r[0]);
                    if (kChunks > 1) ptx::tmem_landed(r[1]);
                    if (c + 2 >= kChunks) {
                        // the accumulator is read: its next K-block may be summed
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (kPair) ptx::mbar_arrive_peer_if(release, lane == 0);
                        else ptx::mbar_arrive_if(release, lane == 0);
                        if (kb + 1 < kb1) {
                            ready = ptx::mbar_test(done(at.slot<Cf::STAGES>()), at.parity<Cf::STAGES>());
                            if (QVEC && in_group(kb + 1) != 0) next_scale(kb + 1);
                        }
                    }
                    add(c);
                    if (c + 2 < kChunks) ptx::tmem_load(src + (uint32_t)((c + 2) * Cf::CHUNK), r[0]);
                    if (c + 1 < kChunks) add(c + 1);
                    if (c + 3 < kChunks) ptx::tmem_load(src + (uint32_t)((c + 3) * Cf::CHUNK), r[1]);
                }
                if (QVEC && kb + 1 < kb1 && in_group(kb + 1) == 0) next_scale(kb + 1);
            }
            if (QVEC && ok && kb0 < kb1) group_ends();
            if (!ok) break;
            if (Cf::SWAPPED && p.splits > 1) {
                // this CTA's K range of the tile, for the cluster to read: [column][lane]
                float *part = reinterpret_cast<float *>(ring);
#pragma unroll
                for (int c = 0; c < Cf::COLS; ++c) part[(col0 + c) * kLanes + row] = acc[c];
                break;                                   // one tile a cluster
            }
            if (kEarly) first_scales(t + units);
            const Tile T = tile_at<BN, Cf::ROWS>(p, first_tile, first_row, t);
            const uint32_t out_buf = out0 + (warp - 4) * (uint32_t)Cf::OUT_BYTES;
            if constexpr (Cf::SWAPPED)
                write_swapped<Cf::COLS>(p, T, (int)(quarter * 32), col0, acc, out_buf, (int)lane);
            else
                write_rows<Cf::COLS>(p, &tmC, T, (int)(quarter * 32 + rank * kLanes), col0, acc, out_buf, box, (int)lane);
        }
    }

    // Before the CTA's shared memory goes, its TMA stores must have read it.
    if (warp >= 4 && lane == 0) ptx::bulk_wait_group_read<0>();
    // K ranges: every CTA of the cluster sums its share of the columns over all
    // of them, in their order, and writes it: rows of C, four neighbouring
    // elements a thread and step, two steps' loads in flight.
    if (Cf::SWAPPED && p.splits > 1) {
        __syncwarp();
        ptx::cluster_sync();
        if (warp >= 4 && unit < num_tiles && *abort_flag == 0) {
            const Tile T = tile_at<BN, Cf::ROWS>(p, first_tile, first_row, unit);
            const int share = BN / p.splits, c0 = (int)crank * share, quads = share * (kLanes / 4);
            constexpr int kStep = EW * 32;
            const int64_t cc = (int64_t)T.i0 + 4 * lane;               // (a warp's lanes take a whole row of the tile)
            float bias[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) bias[k] = cc + k < T.i1 ? epi_bias(p.epi, cc + k, cc + k + 1) : 0.f;
            for (int q = (int)threadIdx.x - 128; q < quads; q += 2 * kStep) {
                const int c = c0 + q / 32, d = c0 + min(q + kStep, quads - 1) / 32;
                const uint32_t at0 = ring0 + 4u * (uint32_t)(c * kLanes + 4 * (int)lane);
                const uint32_t at1 = ring0 + 4u * (uint32_t)(d * kLanes + 4 * (int)lane);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f), w = v;
                for (int s = 0; s < p.splits; ++s) {
                    const float4 x = ptx::ld_cluster_v4f(ptx::mapa_shared(at0, (uint32_t)s));
                    const float4 y = ptx::ld_cluster_v4f(ptx::mapa_shared(at1, (uint32_t)s));
                    v = make_float4(v.x + x.x, v.y + x.y, v.z + x.z, v.w + x.w);
                    w = make_float4(w.x + y.x, w.y + y.y, w.z + y.z, w.w + y.w);
                }
                if (T.j0 + c < T.j1 && cc < T.i1) write_four(p, (int64_t)T.j0 + c, cc, T.i1, v, bias);
                if (q + kStep < quads && T.j0 + d < T.j1 && cc < T.i1) write_four(p, (int64_t)T.j0 + d, cc, T.i1, w, bias);
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

// `count` matrices of rows x cols bytes, in boxes of box_rows x 128 bytes.
int encode_bytes(CUtensorMap *map, const void *base, int64_t rows, int64_t cols, int64_t ld, int64_t count,
                 int64_t stride, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return api_error(GEMM_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)count};
    const cuuint64_t strides[2] = {(cuuint64_t)ld, (cuuint64_t)(count > 1 ? stride : ld)};
    const cuuint32_t box[3] = {128, (cuuint32_t)box_rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return GEMM_OK;
    char msg[96];
    std::snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
    return api_error(GEMM_ERR_CUDA, msg);
}

// C in boxes of 32 rows x 128 bytes.
int encode_rows(CUtensorMap *map, void *C, int out, int64_t rows, int64_t cols, int64_t ld) {
    auto enc = tensor_map_encoder();
    if (!enc) return api_error(GEMM_ERR_CUDA, "cuTensorMapEncodeTiled is not available");
    const int ob = op_type_bytes(out);
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(ld * ob)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / ob), 32};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, out == GEMM_OUT_F32    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : out == GEMM_OUT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                       : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           2, C, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r == CUDA_SUCCESS) return GEMM_OK;
    char msg[96];
    std::snprintf(msg, sizeof msg, "cuTensorMapEncodeTiled failed for C (CUresult %d)", (int)r);
    return api_error(GEMM_ERR_CUDA, msg);
}

struct ScaledPlan {
    int swap, bn, cg, qvec, splits, grid;
};

template <int BN, bool QVEC, int EW, int CG>
int launch(const ScaledPlan &pl, const CUtensorMap &tp, const CUtensorMap &tq, const CUtensorMap &tc,
           const ScaledParams &p, cudaStream_t stream) {
    using Cf = Cfg<BN, QVEC, EW, CG>;
    auto kern = scaled_kernel<BN, QVEC, EW, CG>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM);
    if (e != cudaSuccess) return op_launched("cudaFuncSetAttribute", e);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)pl.grid, 1, 1);
    cfg.blockDim = dim3(Cf::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Cf::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    unsigned n = 0;
    if (CG == 2 || pl.splits > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = CG == 2 ? 2u : (unsigned)pl.splits;
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
    return op_launched("block-scaled product launch", cudaLaunchKernelEx(&cfg, kern, tp, tq, tc, p));
}

int launch_plan(const ScaledPlan &pl, const CUtensorMap &tp, const CUtensorMap &tq, const CUtensorMap &tc,
                const ScaledParams &p, cudaStream_t stream) {
    switch (pl.bn) {
        case 16: return launch<16, true, 4, 1>(pl, tp, tq, tc, p, stream);
        case 32: return launch<32, true, 4, 1>(pl, tp, tq, tc, p, stream);
        case 64: return launch<64, true, 8, 1>(pl, tp, tq, tc, p, stream);
        case 128:
            return pl.qvec ? launch<128, true, 8, 1>(pl, tp, tq, tc, p, stream)
                           : launch<128, false, 8, 1>(pl, tp, tq, tc, p, stream);
        case 192: return launch<192, false, 12, 2>(pl, tp, tq, tc, p, stream);
        default:
            return pl.qvec ? launch<256, true, 8, 2>(pl, tp, tq, tc, p, stream)
                           : launch<256, false, 8, 2>(pl, tp, tq, tc, p, stream);
    }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return cdiv(a, b) * b; }

// One operand as the caller gave it: `rows` x `cols` bytes in memory.
struct Operand {
    const char *name;
    const void *p;
    int64_t rows, cols, ld;
    bool pack;               // TMA cannot address it
    int64_t ld_use;
};

void plan_operand(Operand *o) {
    // (the pitch of a single row is nobody's)
    if (o->rows <= 1) o->ld = round_up(o->cols, 16);
    o->pack = (uintptr_t)o->p % 16 != 0 || o->ld % 16 != 0;
    o->ld_use = o->pack ? round_up(o->cols, 16) : o->ld;
}

int check_scale(const char *name, const gemm_block_scale_t *s, bool tile_ok, int64_t extent, int64_t num_kb,
                int64_t experts, int64_t stride_e, OpSpan *span) {
    char msg[128];
    const int64_t kMax = 1LL << 36;
    if (!s || !(s->block == 1 || (tile_ok && s->block == 128)) || s->stride_k < 0 || s->stride_i < 0 ||
        s->stride_k > kMax || s->stride_i > kMax || stride_e < 0 || stride_e > (1LL << 46)) {
        std::snprintf(msg, sizeof msg, "%s: NULL, or block or strides out of range", name);
        return api_error(GEMM_ERR_INVALID_ARG, msg);
    }
    const int64_t n = s->block == 128 ? cdiv(extent, 128) : extent;
    *span = OpSpan{name, s->scale, op_bytes({{num_kb, s->stride_k}, {n, s->stride_i}, {experts, stride_e}}, 4), 4, false};
    return GEMM_OK;
}

ScaleView view_of(const gemm_block_scale_t *s, int64_t stride_e) {
    return ScaleView{s->scale, s->stride_k, s->stride_i, stride_e, s->block == 128 ? 7 : 0};
}

uint32_t idesc_of(int dtype, int bn, int cg, int p_mn, int q_mn) {
    // D f32 (bit 4), A/B format (bits 7-9, 10-12: e4m3 0, e5m2 1), A / B MN-major
    // (bits 15, 16), N >> 3 (bits 17-22), M >> 4 (bits 24-28)
    const uint32_t fmt = dtype == GEMM_E5M2 ? 1u : 0u;
    return (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)p_mn << 15) | ((uint32_t)q_mn << 16) |
           ((uint32_t)(bn >> 3) << 17) | ((uint32_t)((kLanes * cg) >> 4) << 24);
}

// Tile shape, roles and K ranges of one product: the cheapest by a model of the
// kernel's pace, in units of a 16-column tile's K-block (about 0.3 us):
//   swapped tiles of 16, 32, 64 columns   1, 1.05, 1.15 a K-block, 2 or 3 a tile
//   128 x 128                             1.25 a K-block, 5 a tile
//   256 x 256, 256 x 192 on a CTA pair    1.5, 1.3 a K-block, 13.5, 7.7 a tile
// and 8 or 9 more for K cut in 2 or 4 ranges (the cluster's exchange: measured
// 2.4 us; 8 ranges cost 9 us and are never taken).  Both sides measured in one run, in us:
// 256 columns 463 at 8192^3, 107 at 8192 x 8192 x 1024, 28 at 2048^3; 192 columns
// (three warpgroups' sums, half the epilogue) 517, 103 and 31.
ScaledPlan plan_product(int64_t M, int64_t N, int64_t num_kb, bool a_col, bool b_col, bool b_tile, int sms) {
    ScaledPlan best = {};
    double least = 0.;
    auto consider = [&](int swap, int bn, int cg, int splits, double per_kb, double per_tile) {
        const int64_t tiles = swap ? cdiv(N, kLanes) * cdiv(M, bn) : cdiv(M, kLanes * cg) * cdiv(N, bn);
        if (splits > 1 && (tiles * splits > sms || num_kb < 2 * splits)) return;
        const int64_t at_once = sms / cg, rounds = cdiv(tiles * splits, at_once);
        const double cost = rounds * (cdiv(num_kb, splits) * per_kb + per_tile) +
                            (splits == 1 ? 0. : splits == 2 ? 8. : 9.);
        if (best.bn && cost >= least) return;
        least = cost;
        best.swap = swap;
        best.bn = bn;
        best.cg = cg;
        best.qvec = swap || !b_tile;
        best.splits = splits;
        best.grid = (int)(splits > 1 ? tiles * splits : std::min<int64_t>(tiles, at_once) * cg);
    };
    // (swapped, A is read by the MMA's column side, which takes an M-major
    // operand only in chunks of 128)
    if (!a_col)
        for (int splits = 1; splits <= 4; splits *= 2) {
            if (M <= 16) consider(1, 16, 1, splits, 1., 2.);
            else if (M <= 32) consider(1, 32, 1, splits, 1.05, 2.);
            else consider(1, 64, 1, splits, 1.15, 3.);
        }
    if (M > 64 || a_col) {
        consider(0, 128, 1, 1, 1.25, 5.);
        consider(0, 256, 2, 1, 1.5, 13.5);
        if (b_tile && b_col) consider(0, 192, 2, 1, 1.3, 7.7);     // (whole 128-column chunks of B otherwise)
    }
    return best;
}

// Tile shape and roles of an expert product, from the rows an expert has on average.
ScaledPlan plan_experts(int64_t rows, int64_t N, int64_t num_kb, int64_t experts, bool b_col, bool b_tile, int sms) {
    ScaledPlan pl = {};
    const int64_t used = std::max<int64_t>(1, std::min(rows, experts)), avg = cdiv(rows, used);
    pl.cg = 1;
    pl.splits = 1;
    // One tile should hold most experts' rows, which scatter around the average:
    // swapped tiles up to 48 rows, 128 x 128 tiles up to 112, 256 x 256 beyond.
    // Measured (2048 x 4096, 64 experts): 64 rows on average 143 us in swapped
    // tiles of 64 columns, where every second expert needs two, 113 us in 128 x 128.
    if (avg <= 48) {
        pl.swap = 1;
        pl.bn = avg <= 12 ? 16 : avg <= 24 ? 32 : 64;
        pl.qvec = 1;
    } else if (avg <= 112) {
        pl.bn = 128;
    } else {
        // 256 or 192 columns as plan_product has it, the tiles' fixed cost higher here
        // (32768 rows over 32 experts 4096 x 2048: 391 us and 380; 16384 over 64,
        // 2048 x 4096: 231 and 246)
        const double wide = (double)cdiv(N, 256) * (1.5 * num_kb + 18.), narrow = (double)cdiv(N, 192) * (1.3 * num_kb + 8.7);
        pl.bn = b_col && b_tile && narrow < wide ? 192 : 256;
        pl.cg = 2;
    }
    const int64_t wt = pl.swap ? cdiv(N, kLanes) : cdiv(N, pl.bn), rt = pl.swap ? pl.bn : kLanes * pl.cg;
    pl.grid = (int)std::min<int64_t>(sms / pl.cg, wt * (cdiv(rows, rt) + used)) * pl.cg;
    return pl;
}

int check_common(int dtype, const gemm_epilogue_t *epi_in, EpiParams *epi) {
    if (dtype != GEMM_E4M3 && dtype != GEMM_E5M2) return api_error(GEMM_ERR_INVALID_ARG, "dtype must be E4M3 or E5M2");
    return api_epilogue(epi_in, epi);
}

// Copies the operands TMA cannot address into one workspace (returned to free).
int pack_operands(Operand *a, Operand *b, int dev, void **ws, cudaStream_t stream) {
    *ws = nullptr;
    const uint64_t na = a->pack ? (uint64_t)a->rows * a->ld_use : 0, nb = b->pack ? (uint64_t)b->rows * b->ld_use : 0;
    const uint64_t off = (na + 255) / 256 * 256;
    if (!na && !nb) return GEMM_OK;
    cudaError_t e = op_malloc(ws, off + nb, dev, stream);
    if (e != cudaSuccess) {
        cudaGetLastError();
        *ws = nullptr;
        char msg[128];
        std::snprintf(msg, sizeof msg, "workspace of %llu bytes: %s", (unsigned long long)(off + nb),
                      cudaGetErrorString(e));
        return api_error(GEMM_ERR_NO_MEMORY, msg);
    }
    for (int i = 0; i < 2; ++i) {
        Operand *o = i ? b : a;
        if (!o->pack) continue;
        uint8_t *dst = static_cast<uint8_t *>(*ws) + (i ? off : 0);
        uint64_t lo = 0, hi = 0;
        int rc = api_check_device_span_range(o->name, o->p, op_extent(o->rows, o->cols, o->ld, 1), dev, &lo, &hi);
        if (rc == GEMM_OK)
            rc = op_launched("operand pack", pack_rows_launch(o->p, o->ld, dst, o->ld_use, o->rows, o->cols, 1, lo, hi, stream));
        if (rc) {
            cudaFreeAsync(*ws, stream);
            *ws = nullptr;
            return rc;
        }
        o->p = dst;
    }
    return GEMM_OK;
}

// The two operands' tensor maps as the plan takes them, then the kernel.
int encode_and_launch(const ScaledPlan &pl, ScaledParams &p, const Operand &a, int a_major, const Operand &b,
                      int b_major, int64_t experts, int64_t b_expert, int dtype, cudaStream_t stream) {
    const Operand &P = pl.swap ? b : a, &Q = pl.swap ? a : b;
    p.p_mn = pl.swap ? !b_major : a_major;
    p.q_mn = pl.swap ? a_major : !b_major;
    p.idesc = idesc_of(dtype, pl.bn, pl.cg, p.p_mn, p.q_mn);
    p.swapped = pl.swap;
    p.splits = pl.splits;
    p.kb_per_split = (int)cdiv(p.num_kb, pl.splits);
    p.group_i = 16;
    const Options opt = options_snapshot();
    p.timeout_ns = (unsigned long long)opt.wait_timeout_ms * 1000000ull;
    p.debug_stall = opt.debug_stall_mma;
    CUtensorMap tp, tq, tc;
    std::memset(&tp, 0, sizeof tp);
    std::memset(&tq, 0, sizeof tq);
    std::memset(&tc, 0, sizeof tc);
    if (p.num_kb > 0) {
        const int64_t pe = pl.swap ? experts : 1, qe = pl.swap ? 1 : experts;
        int rc = encode_bytes(&tp, P.p, P.rows, P.cols, P.ld_use, pe, b_expert, kLanes);
        if (rc == GEMM_OK)
            rc = encode_bytes(&tq, Q.p, Q.rows, Q.cols, Q.ld_use, qe, b_expert, p.q_mn ? 128 : pl.bn / pl.cg);
        if (rc) return rc;
    }
    const int out = p.epi.active ? p.epi.out : GEMM_OUT_F32, ob = op_type_bytes(out);
    const int64_t rows = pl.swap ? p.J : p.I, cols = pl.swap ? p.I : p.J;
    p.wide = op_wide(p.C, p.ldc, ob);
    p.tma_store = !pl.swap && pl.splits == 1 && p.wide && (cols * ob) % 16 == 0;
    if (p.tma_store) {
        const int rc = encode_rows(&tc, p.C, out, rows, cols, p.ldc);
        if (rc) return rc;
    }
    return launch_plan(pl, tp, tq, tc, p, stream);
}

}  // namespace

cudaError_t scaled_read_and_clear_status(uint32_t words[4]) {
    cudaError_t e = cudaMemcpyFromSymbol(words, g_scaled_status, sizeof(uint32_t) * 4);
    if (e != cudaSuccess || words[0] == 0) return e;
    static const uint32_t zero[4] = {0, 0, 0, 0};
    return cudaMemcpyToSymbol(g_scaled_status, zero, sizeof zero);
}

}  // namespace tcgemm

using namespace tcgemm;

extern "C" {

int gemm_run_scaled(int64_t M, int64_t N, int64_t K, int dtype, const void *A, int64_t lda, int a_major,
                    const gemm_block_scale_t *a_scale, const void *B, int64_t ldb, int b_major,
                    const gemm_block_scale_t *b_scale, void *C, int64_t ldc, const gemm_epilogue_t *epi_in,
                    struct CUstream_st *stream_) {
    api_clear_error();
    EpiParams epi;
    int rc = check_common(dtype, epi_in, &epi);
    if (rc) return rc;
    const int64_t kMax = 0x7fffffffLL - 512, kLdMax = 1LL << 36;
    if (M < 0 || N < 0 || K < 0 || M > kMax || N > kMax || K > kMax)
        return api_error(GEMM_ERR_INVALID_ARG, "size negative or out of range");
    if ((a_major != 0 && a_major != 1) || (b_major != 0 && b_major != 1))
        return api_error(GEMM_ERR_INVALID_ARG, "a_major and b_major are 0 or 1");
    Operand a = {"A", A, a_major ? K : M, a_major ? M : K, lda, false, 0};
    Operand b = {"B", B, b_major ? N : K, b_major ? K : N, ldb, false, 0};
    if (lda < std::max<int64_t>(a.cols, 1) || ldb < std::max<int64_t>(b.cols, 1) || ldc < std::max<int64_t>(N, 1) ||
        lda > kLdMax || ldb > kLdMax || ldc > kLdMax)
        return api_error(GEMM_ERR_INVALID_ARG, "leading dimension out of range");
    const int64_t num_kb = cdiv(K, kBlockK);
    const int ob = epi.active ? op_type_bytes(epi.out) : 4;
    OpSpan spans[6] = {{"A", A, op_extent(a.rows, a.cols, lda, 1), 1, false},
                       {"B", B, op_extent(b.rows, b.cols, ldb, 1), 1, false},
                       {"C", C, op_extent(M, N, ldc, ob), ob, true},
                       {"bias", epi.active ? epi.bias : nullptr, epi.active && epi.bias ? (uint64_t)N * 4 : 0, 4, false}};
    if ((rc = check_scale("a_scale", a_scale, true, M, num_kb, 1, 0, &spans[4]))) return rc;
    if ((rc = check_scale("b_scale", b_scale, true, N, num_kb, 1, 0, &spans[5]))) return rc;
    if (M == 0 || N == 0) return GEMM_OK;
    int sms = 0;
    if ((rc = op_check(spans, 6, &sms))) return rc;
    plan_operand(&a);
    plan_operand(&b);
    const ScaledPlan pl = plan_product(M, N, num_kb, a_major != 0, b_major != 0, b_scale->block == 128, sms);
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    ScaledParams p = {};
    p.I = (int)(pl.swap ? N : M);
    p.J = (int)(pl.swap ? M : N);
    p.num_kb = (int)num_kb;
    const int64_t ti = cdiv(p.I, kLanes * pl.cg), tj = cdiv(p.J, pl.bn);
    if (ti * tj * pl.splits > kMax) return api_error(GEMM_ERR_INVALID_ARG, "too many tiles");
    p.tiles_i = (int)ti;
    p.tiles_j = (int)tj;
    p.sp = view_of(pl.swap ? b_scale : a_scale, 0);
    p.sq = view_of(pl.swap ? a_scale : b_scale, 0);
    p.C = C;
    p.ldc = ldc;
    p.epi = epi;
    p.tokens_on_i = !pl.swap;
    int dev = 0;
    cudaGetDevice(&dev);
    void *ws = nullptr;
    if (num_kb > 0 && (rc = pack_operands(&a, &b, dev, &ws, stream))) return rc;
    rc = encode_and_launch(pl, p, a, a_major, b, b_major, 1, 0, dtype, stream);
    if (ws) {
        const cudaError_t e = cudaFreeAsync(ws, stream);
        if (rc == GEMM_OK) rc = op_launched("cudaFreeAsync", e);
    }
    return rc;
}

int gemm_run_experts(int64_t rows, int64_t N, int64_t K, int64_t experts, int dtype, const void *A, int64_t lda,
                     const gemm_block_scale_t *a_scale, const int32_t *offsets, const void *B, int64_t ldb,
                     int64_t b_expert, int b_major, const gemm_block_scale_t *b_scale, int64_t b_scale_expert, void *C,
                     int64_t ldc, const gemm_epilogue_t *epi_in, struct CUstream_st *stream_) {
    api_clear_error();
    EpiParams epi;
    int rc = check_common(dtype, epi_in, &epi);
    if (rc) return rc;
    if (epi.active && (epi.beta != 0.f || epi.bias))
        return api_error(GEMM_ERR_INVALID_ARG, "the expert product takes beta = 0 and no bias");
    const int64_t kMax = 0x7fffffffLL - 512, kLdMax = 1LL << 36;
    if (rows < 0 || N < 0 || K < 0 || rows > kMax || N > kMax || K > kMax)
        return api_error(GEMM_ERR_INVALID_ARG, "size negative or out of range");
    if (experts < 1 || experts > kMaxExperts) return api_error(GEMM_ERR_INVALID_ARG, "experts must be in [1, 1024]");
    if (b_major != 0 && b_major != 1) return api_error(GEMM_ERR_INVALID_ARG, "b_major is 0 or 1");
    Operand a = {"A", A, rows, K, lda, false, 0};
    Operand b = {"B", B, b_major ? N : K, b_major ? K : N, ldb, false, 0};
    if (lda < std::max<int64_t>(K, 1) || ldb < std::max<int64_t>(b.cols, 1) || ldc < std::max<int64_t>(N, 1) ||
        lda > kLdMax || ldb > kLdMax || ldc > kLdMax)
        return api_error(GEMM_ERR_INVALID_ARG, "leading dimension out of range");
    if (b_expert < 0 || b_expert > (1LL << 39)) return api_error(GEMM_ERR_INVALID_ARG, "b_expert out of range");
    const int64_t num_kb = cdiv(K, kBlockK);
    const int ob = epi.active ? op_type_bytes(epi.out) : 4;
    OpSpan spans[6] = {{"A", A, op_extent(rows, K, lda, 1), 1, false},
                       {"B", B, op_bytes({{experts, b_expert}, {b.rows, ldb}, {b.cols, 1}}, 1), 1, false},
                       {"C", C, op_extent(rows, N, ldc, ob), ob, true},
                       {"offsets", offsets, (uint64_t)(experts + 1) * 4, 4, false}};
    if ((rc = check_scale("a_scale", a_scale, false, rows, num_kb, 1, 0, &spans[4]))) return rc;
    if ((rc = check_scale("b_scale", b_scale, true, N, num_kb, experts, b_scale_expert, &spans[5]))) return rc;
    if (rows == 0 || N == 0) return GEMM_OK;
    plan_operand(&a);
    if (b.rows <= 1) b.ld = round_up(b.cols, 16);       // (the pitch of a single row is nobody's)
    if (num_kb > 0 && ((uintptr_t)B % 16 != 0 || b.ld % 16 != 0 || b_expert % 16 != 0))
        return api_error(GEMM_ERR_UNSUPPORTED, "B's base, pitch and b_expert must be multiples of 16 bytes");
    int sms = 0;
    if ((rc = op_check(spans, 6, &sms))) return rc;
    b.ld_use = b.ld;
    ScaledPlan pl = plan_experts(rows, N, num_kb, experts, b_major != 0, b_scale->block == 128, sms);
    if (!pl.swap) pl.qvec = b_scale->block != 128;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    ScaledParams p = {};
    p.I = (int)(pl.swap ? N : rows);
    p.J = (int)(pl.swap ? rows : N);
    p.num_kb = (int)num_kb;
    p.tiles_i = pl.swap ? (int)cdiv(N, kLanes) : 0;
    p.tiles_j = pl.swap ? 0 : (int)cdiv(N, pl.bn);
    if ((cdiv(rows, 16) + experts) * cdiv(N, kLanes) > kMax)
        return api_error(GEMM_ERR_INVALID_ARG, "too many tiles");
    p.sp = view_of(pl.swap ? b_scale : a_scale, pl.swap ? b_scale_expert : 0);
    p.sq = view_of(pl.swap ? a_scale : b_scale, pl.swap ? 0 : b_scale_expert);
    p.C = C;
    p.ldc = ldc;
    p.epi = epi;
    p.offsets = offsets;
    p.experts = (int)experts;
    p.rows = (int)rows;
    p.tokens_on_i = !pl.swap;
    int dev = 0;
    cudaGetDevice(&dev);
    void *ws = nullptr;
    if (num_kb > 0) {
        Operand none = {"", nullptr, 0, 0, 0, false, 0};
        if ((rc = pack_operands(&a, &none, dev, &ws, stream))) return rc;
    }
    rc = encode_and_launch(pl, p, a, 0, b, b_major, experts, b_expert, dtype, stream);
    if (ws) {
        const cudaError_t e = cudaFreeAsync(ws, stream);
        if (rc == GEMM_OK) rc = op_launched("cudaFreeAsync", e);
    }
    return rc;
}

}  // extern "C"
