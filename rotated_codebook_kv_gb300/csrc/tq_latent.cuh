// tq_latent.cuh -- what the attention kernels over latent pages share: arguments, the dealing out of the work, small helpers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace latent {

constexpr int kRope = TQ_LATENT_ROPE_DIM;
constexpr int kUnitCost = 1;     // what a unit costs beside its tiles, in tiles
constexpr int kMinShare = 3;     // least cost of a worker's share
constexpr int kMaxWorkers = 256;
constexpr int kSoftWarps = 8, kSoft = 32 * kSoftWarps;
constexpr float kLog2e = 1.4426950408889634f;
// The reference m stands 2^kMargin above the running maximum when it is set, and O is rescaled only when the maximum passes
// it: P <= 1 always, and 2^-16 where it was set, so that sums of 2^16 values near the largest number do not overflow before the
// division; bf16 has the exponents for what is smaller.
constexpr float kMargin = 16.f;

struct Args {
    const uint16_t *pool;
    const int32_t *block_table, *seq_lens;
    int B, Tq, Hq, R, RT;  // R = Tq Hq rows of a sequence, in RT blocks (of 128, or of 64 in the narrow kernel)
    int P, pshift, max_blocks;
    int64_t num_blocks;
    int workers;           // pairs of CTAs, or CTAs
    float sm_scale;
    int4 *rec;             // [workers] unit whose first piece is this worker's: b, row block, pieces (0: none)
    float2 *ml;            // [2 workers][rows of a unit] reference, denominator
    float *acc;            // [2 workers][rows of a unit][DL]
    uint16_t *out;
    unsigned *status;
    long long wait_limit;
};

__device__ __forceinline__ uint32_t saddr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v)
{
    float2 f;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
    return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// The softmax warps' barrier; whether any of their threads says so.
__device__ __forceinline__ bool any_of_softmax(bool x)
{
    uint32_t r;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbarrier.cta.red.or.pred p, 1, %2, q;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(r) : "r"(static_cast<uint32_t>(x)), "n"(kSoft) : "memory");
    return r != 0;
}

// A unit's piece: tokens of tiles t0 .. t1 - 1 of `tiles`, rows of block rt of sequence b.
struct Piece {
    int b, rt, n, L, t0, t1, tiles;
    long long end;  // the unit's last cost + 1
};

// The unit u's sequence, row block (of ROWS), tokens that its last row sees, and tiles (of TOKENS).
template <int ROWS, int TOKENS>
__device__ __forceinline__ void unit_of(const Args &A, int u, Piece &p)
{
    p.b = u / A.RT;
    p.rt = u - p.b * A.RT;
    const int L = min(max(__ldg(A.seq_lens + p.b), 0), A.max_blocks << A.pshift);
    const int last = A.Tq == 1 ? 0 : (min((p.rt + 1) * ROWS, A.R) - 1) / A.Hq;
    p.L = L;
    p.n = max(0, L - A.Tq + last + 1);
    p.tiles = (p.n + TOKENS - 1) / TOKENS;
}

// A worker's share: costs x0 .. x1 - 1 of the units' costs laid end to end, from unit u, whose first cost is a.
template <int ROWS, int TOKENS>
struct Share {
    long long x0, x1, a;
    int u, units;
    // The next piece (t0 < t1), or a unit without a token (tiles 0).
    __device__ __forceinline__ bool next(const Args &A, Piece &p)
    {
        while (u < units && a < x1) {
            unit_of<ROWS, TOKENS>(A, u, p);
            const long long first = a + kUnitCost;
            a = first + p.tiles;
            p.end = a;
            ++u;
            if (p.tiles == 0) {
                if (first - kUnitCost >= x0) {
                    p.t0 = p.t1 = 0;
                    return true;
                }
                continue;
            }
            p.t0 = static_cast<int>(min(max(x0 - first, 0LL), static_cast<long long>(p.tiles)));
            p.t1 = static_cast<int>(min(max(x1 - first, 0LL), static_cast<long long>(p.tiles)));
            if (p.t0 < p.t1) return true;
        }
        return false;
    }
};

// The share of worker w: a scan of the units' costs, a stretch of units per thread of the block.  `sums` holds one number a
// warp, then the first unit's first cost, and the unit; shared memory that nothing else uses.  Synchronises the block.
template <int ROWS, int TOKENS, int THREADS>
__device__ __forceinline__ Share<ROWS, TOKENS> deal(const Args &A, int w, bool report, long long *sums, long long &total, long long &shares)
{
    constexpr int kWarps = THREADS / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Share<ROWS, TOKENS> share;
    share.units = A.B * A.RT;
    const int per = (share.units + THREADS - 1) / THREADS;
    const int u0 = min(tid * per, share.units), u1 = min(u0 + per, share.units);
    long long mine = 0;
    for (int u = u0; u < u1; ++u) {
        Piece p;
        unit_of<ROWS, TOKENS>(A, u, p);
        mine += p.tiles + kUnitCost;
        if (report && p.rt == 0 && __ldg(A.seq_lens + p.b) > (A.max_blocks << A.pshift)) atomicOr(A.status, TQ_DEVERR_SEQ_RANGE);
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long long before = upto - mine;
    total = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        const long long v = sums[k];
        if (k < warp) before += v;
        total += v;
    }
    shares = min(static_cast<long long>(A.workers), max(total / kMinShare, 1LL));
    share.x0 = w < shares ? w * total / shares : total;
    share.x1 = w < shares ? (w + 1) * total / shares : total;
    if (before <= share.x0 && share.x0 < before + mine) {  // one thread
        long long a = before;
        int u = u0;
        for (;; ++u) {
            Piece p;
            unit_of<ROWS, TOKENS>(A, u, p);
            if (a + p.tiles + kUnitCost > share.x0) break;
            a += p.tiles + kUnitCost;
        }
        sums[kWarps] = a;
        sums[kWarps + 1] = u;
    }
    __syncthreads();
    share.a = sums[kWarps];
    share.u = share.x0 < share.x1 ? static_cast<int>(sums[kWarps + 1]) : share.units;
    return share;
}

// Two stages do not quite cover HBM's latency: the tile behind them is asked into L2, 16 tokens (which lie on one page) by every
// other lane.  131k tokens of 32 heads 65.0 -> 62.4 us, 8 x 32k of 128 heads 87.5 -> 83.6; further ahead it takes bandwidth
// from the loads (two tiles 65.4, three 69).
template <int D>
__device__ __forceinline__ void prefetch_rows(const Args &A, int pos, int blk, bool mine)
{
    if (mine && !(threadIdx.x & 1) && blk >= 0 && blk < A.num_blocks)
        l2_prefetch_bulk(A.pool + ((static_cast<int64_t>(blk) << A.pshift) + (pos & (A.P - 1))) * D, 16 * D * 2);
}

// Rows of a sequence that the narrow kernel takes (one CTA, 64 rows); longer ones go to pairs of CTAs.
constexpr int kNarrowRows = 64;
// The narrow kernel's launch, in its own translation unit; tk: boxes of a group's blocks (narrow_group), tq: 64 rows.
int narrow_group(int dl);
cudaError_t launch_narrow(const CUtensorMap &tk, const CUtensorMap &tq, int dl, const Args &a, cudaStream_t st);

}  // namespace latent
}  // namespace tq
