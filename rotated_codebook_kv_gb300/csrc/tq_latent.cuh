// tq_latent.cuh -- what the attention kernels over latent pages share: arguments, the dealing out of the work, small helpers.
#pragma once

#include <utility>

#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace latent {

constexpr int kRope = TQ_LATENT_ROPE_DIM;
// What a unit costs beside its tiles (Q, the first loads, its output), in tiles: 1 to 3 and 5 to 8 were up to 4% slower over mixed
// batches, drafted tokens and chunks.
constexpr int kUnitCost = 4;
constexpr int kMinShare = 3;     // least cost of a worker's share: 6 to 16 leave SMs idle in small calls (11.5 -> 13.8 us at 16)
constexpr int kMaxWorkers = 256;
// Rows of a sequence that the narrow kernel takes (one CTA, 64 rows); longer ones go to pairs of CTAs.
constexpr int kNarrowRows = 64;
constexpr int kSoftWarps = 8, kSoft = 32 * kSoftWarps;
constexpr float kLog2e = 1.4426950408889634f;
// P = 2^(c (s - r) - kMargin), c = |sm_scale| log2(e), r the largest score when it was set (the reference).  It moves, and O is
// rescaled, when a score passes it by more than kSlack powers of two: P is 2^-32 at r and 2^-16 at most, so that no sum of 2^16
// values, however large each is, overflows before the division.  At the other end O keeps steps of 2^-149, of 2^-117 after the
// division (latents of 2^-104 are still right to bf16's last bit, of 2^-110 to 1 - 5%).  (A slack of 8: more rescaling, a long
// prompt's chunk 2.86 -> 2.96 ms.)
// c s - (c r + kMargin), one operation, is off by the rounding of c r: 2^-14 at kFar.  Where a reference lies beyond, the
// difference s - r comes first, so that scores of any size keep P in its range (for every tile: 1.5% of a long chunk; the branch
// itself 0.4%).
constexpr float kMargin = 32.f, kSlack = 16.f, kFar = 1024.f;

struct Args {
    const uint16_t *pool;
    const int32_t *block_table, *seq_lens;
    int B, Tq, Hq, R, RT;  // R = Tq Hq rows of a sequence, in RT blocks (of 128, or of 64 in the narrow kernel)
    int P, pshift, max_blocks;
    bool few;              // a warp's lanes are enough to count the units
    int64_t num_blocks;
    int workers;           // pairs of CTAs, or CTAs
    int least_workers;     // a share's costs could pass 1.5 x 2^30 with fewer
    float sm_scale;
    int *done;             // [workers] blocks that have written their pieces of the unit whose first piece is this worker's
    float2 *ml;            // [2 workers][rows of a unit] reference, denominator (kNothing: the piece has no sums)
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
// 32 bytes, a whole sector a lane.
__device__ __forceinline__ void stg256(float *p, const float (&v)[8])
{
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]),
                 "f"(v[6]), "f"(v[7])
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// The softmax warps' barrier; whether any of their threads says so.  The warp is gathered for it, and behind it: accesses to
// tensor memory want whole warps.
__device__ __forceinline__ bool any_of_softmax(bool x)
{
    uint32_t r;
    __syncwarp();
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 q, %1, 0;\nbarrier.cta.red.or.pred.aligned p, 1, %2, q;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(r) : "r"(static_cast<uint32_t>(x)), "n"(kSoft) : "memory");
    return r != 0;
}

// A unit's piece: tokens of tiles t0 .. t1 - 1 of `tiles`, rows of block rt of sequence b.
struct Piece {
    int b, rt, n, L, t0, t1, tiles;
};

// The unit u's sequence, row block (of ROWS), tokens that its last row sees, and tiles (of TOKENS).
template <int ROWS, int TOKENS>
__device__ __forceinline__ void unit_of(const Args &A, int u, Piece &p)
{
    const bool one = ROWS == kNarrowRows || A.RT == 1;  // a unit a sequence, whose last row is of the last token
    p.b = one ? u : u / A.RT;
    p.rt = one ? 0 : u - p.b * A.RT;
    const int L = min(max(__ldg(A.seq_lens + p.b), 0), A.max_blocks << A.pshift);
    p.L = p.n = L;
    if (!one) {
        const int last = (min((p.rt + 1) * ROWS, A.R) - 1) / A.Hq;
        p.n = max(0, L - A.Tq + last + 1);
    }
    p.tiles = (p.n + TOKENS - 1) / TOKENS;
}

// A worker's share: `len` of the units' costs laid end to end, from unit u, whose first cost stands at a <= 0 against the share's
// first.
template <int ROWS, int TOKENS>
struct Share {
    int a, len, u, units;
    // The next piece (t0 < t1), or a unit without a token (tiles 0).
    __device__ __forceinline__ bool next(const Args &A, Piece &p)
    {
        while (u < units && a < len) {
            unit_of<ROWS, TOKENS>(A, u, p);
            const int first = a + kUnitCost;
            a = first + p.tiles;
            ++u;
            if (p.tiles == 0) {
                if (first < kUnitCost) continue;  // an earlier share's
                p.t0 = p.t1 = 0;
                return true;
            }
            p.t0 = min(max(-first, 0), p.tiles);
            p.t1 = min(max(len - first, 0), p.tiles);
            if (p.t0 < p.t1) return true;
        }
        return false;
    }
};

// Where share w of n begins in `total` costs: quotients of 32 bits where they do.
__device__ __forceinline__ long long share_start(int w, long long total, int n)
{
    if (total < (1 << 23)) return static_cast<unsigned>(w) * static_cast<unsigned>(total) / static_cast<unsigned>(n);
    return w * total / n;
}

// Deals out the work: a scan of the units' costs, a stretch of units per thread of the block.  `sums` holds one number a warp,
// then the first unit's place, and the unit; shared memory that nothing else uses.
template <int ROWS, int TOKENS, int THREADS>
struct Dealer {
    static constexpr int kWarps = THREADS / 32;
    long long before, mine, total, x0, x1;
    int u0, w, shares;
    bool active;

    // The unit that cost x lies in, and its first cost, by the thread that counted it.
    __device__ __forceinline__ int find(const Args &A, long long x, Piece &p, long long &a) const
    {
        a = before;
        for (int u = u0;; ++u) {
            unit_of<ROWS, TOKENS>(A, u, p);
            if (a + p.tiles + kUnitCost > x) return u;
            a += p.tiles + kUnitCost;
        }
    }

    // The share of worker w_.  Synchronises the block.
    __device__ __forceinline__ Share<ROWS, TOKENS> deal(const Args &A, int w_, bool report, long long *sums, int4 *jobs)
    {
        const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
        Share<ROWS, TOKENS> share;
        w = w_;
        share.units = A.B * A.RT;
        if (tid < 2) jobs[tid] = make_int4(0, 0, 0, 0);
        if (A.few) {
            // a unit per lane: every warp counts them for itself and meets no other (0.5 us less than the way below, which 65 units
            // on 32 lanes lose again)
            u0 = min(lane, share.units);
            int m = 0;
            if (lane < share.units) {
                Piece p;
                unit_of<ROWS, TOKENS>(A, lane, p);
                m = p.tiles + kUnitCost;
                if (report && warp == 0 && p.rt == 0 && __ldg(A.seq_lens + p.b) > (A.max_blocks << A.pshift)) atomicOr(A.status, TQ_DEVERR_SEQ_RANGE);
            }
            int upto = m;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= o) upto += v;
            }
            const int all = __shfl_sync(0xffffffffu, upto, 31), b = upto - m;
            before = b;
            mine = m;
            total = all;
            shares = min(A.workers, max(all / kMinShare, 1));
            active = w < shares;
            auto start = [&](int s) -> int { return static_cast<int>(static_cast<unsigned>(s) * static_cast<unsigned>(all) / static_cast<unsigned>(shares)); };
            const int y0 = active ? start(w) : 0, y1 = active ? start(w + 1) : 0;  // all < 2^23 + 2^8, s <= 2^8
            x0 = y0;
            x1 = y1;
            const int src = __ffs(__ballot_sync(0xffffffffu, b <= y0 && y0 < b + m)) - 1;  // the lane of the unit that y0 lies in
            share.len = y1 - y0;
            share.a = __shfl_sync(0xffffffffu, b, src) - y0;
            share.u = active ? src : share.units;
            __syncthreads();
            return share;
        }
        const int per = (share.units + THREADS - 1) / THREADS;
        u0 = min(tid * per, share.units);
        const int u1 = min(u0 + per, share.units);
        mine = 0;
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
        before = upto - mine;
        total = 0;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const long long v = sums[k];
            if (k < warp) before += v;
            total += v;
        }
        shares = static_cast<int>(min(static_cast<long long>(A.workers), max(total / kMinShare, 1LL)));
        active = w < shares;
        x0 = active ? share_start(w, total, shares) : 0;
        x1 = active ? share_start(w + 1, total, shares) : 0;
        share.len = static_cast<int>(x1 - x0);
        if (active && before <= x0 && x0 < before + mine) {
            Piece p;
            long long a;
            const int u = find(A, x0, p, a);
            sums[kWarps] = a - x0;
            sums[kWarps + 1] = u;
            // the block ids that the first loads wait for
            const int t0 = max(0, static_cast<int>(x0 - a) - kUnitCost);
            asm volatile("prefetch.global.L1 [%0];" ::"l"(A.block_table + static_cast<int64_t>(p.b) * A.max_blocks + min(t0 * TOKENS >> A.pshift, A.max_blocks - 1)));
        }
        __syncthreads();
        share.a = static_cast<int>(sums[kWarps]);
        share.u = active ? static_cast<int>(sums[kWarps + 1]) : share.units;
        return share;
    }

    // The units that this worker shares with others, at most two, by the threads that counted them, while the first loads are on
    // their way: the first worker with a tile of the unit, how many there are, the sequence and the row block.
    __device__ __forceinline__ void find_jobs(const Args &A, int4 *jobs) const
    {
        if (!active || (A.few && threadIdx.x >= 32)) return;
        // the least s with (s + 1) total / shares >= v, for v <= total
        auto reaches = [&](long long v) -> int {
            if (total < (1 << 23))
                return (static_cast<unsigned>(v) * static_cast<unsigned>(shares) + static_cast<unsigned>(total) - 1u) / static_cast<unsigned>(total) - 1;
            return static_cast<int>((v * shares + total - 1) / total) - 1;
        };
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            const long long x = side == 0 ? x0 : x1 - 1;
            if (!(before <= x && x < before + mine)) continue;
            Piece p;
            long long a;
            find(A, x, p, a);
            if (side == 1 && a <= x0) continue;  // the first border's unit
            // its tiles have the costs a + kUnitCost .. a + kUnitCost + tiles - 1
            const int f = reaches(a + kUnitCost + 1), l = reaches(a + kUnitCost + p.tiles);
            if (p.tiles > 0 && f < l && f <= w && w <= l) jobs[side] = make_int4(f, l - f + 1, p.b, p.rt);
        }
    }
};

// Joins the pieces of a unit that several workers shared, by all of their blocks (block q of Q), once every piece is there: a warp
// per row where the pieces are few, a block per 256 coordinates of a row (a stretch of the pieces a warp) where they are many.
// A kernel of its own for it, launched as the attention's blocks ended, took 5-10 us longer, and a barrier over the grid 3-8.
// A piece whose scores are all -inf has the denominator 0 and counts all the same: its sums hold 0 times what is infinite.
constexpr int kFewPieces = 16;
constexpr float kNothing = -1.f;
struct Merge {
    float4 part[16][2][32];
    float2 dens[16];  // reference, denominator
};
template <int DL, int ROWS, int THREADS>
__device__ __forceinline__ void merge_unit(const Args &A, const int4 job, int q, int Q, Merge &S)
{
    constexpr int kWarps = THREADS / 32;
    constexpr int N = DL / 128;  // stretches of 128 coordinates of a row, a float4 per lane
    constexpr int K = 8 / N;     // pieces of a row on their way together (16 / N: 0.5 to 1 us slower, 24 / N spills, 4 / N slower)
    static_assert(kWarps <= 16, "a row of partial sums per warp");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = job.y, row0 = job.w * ROWS, rows = min(ROWS, A.R - row0);
    // piece 0 is the first worker's last one, piece k the first one of the k-th after it
    auto slot = [&](int k, int r) -> size_t { return (k == 0 ? 2 * job.x + 1 : 2 * (job.x + k)) * static_cast<size_t>(ROWS) + r; };
    auto add = [&](float4 &o, float a, float4 v) {
        o.x = fmaf(a, v.x, o.x);
        o.y = fmaf(a, v.y, o.y);
        o.z = fmaf(a, v.z, o.z);
        o.w = fmaf(a, v.w, o.w);
    };
    auto put = [&](int r, int j4, float4 o, float den) {
        const float inv = den == 0.f ? 0.f : 1.f / den;
        reinterpret_cast<uint2 *>(A.out + (static_cast<size_t>(job.z) * A.R + row0 + r) * DL)[j4] =
            make_uint2(bf16x2_of(o.x * inv, o.y * inv), bf16x2_of(o.z * inv, o.w * inv));
    };
    // 2^(c (m - M)), M the larger of two references
    const float c = fabsf(A.sm_scale) * kLog2e;
    auto scale_of = [c](float m, float M) -> float { return m == -INFINITY ? 0.f : fast_exp2((m - M) * c); };
    const float4 *acc = reinterpret_cast<const float4 *>(A.acc);
    if (n <= kFewPieces) {
        for (int r = warp * Q + q; r < rows; r += kWarps * Q) {
            float m = -INFINITY, den = 0.f;
            float4 o[N] = {};
            for (int k0 = 0; k0 < n; k0 += K) {
                float2 ml[K];
                float4 v[K][N];
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    ml[k] = make_float2(-INFINITY, kNothing);
                    if (k0 + k < n) {
                        ml[k] = __ldcg(A.ml + slot(k0 + k, r));
#pragma unroll
                        for (int i = 0; i < N; ++i) v[k][i] = __ldcg(acc + slot(k0 + k, r) * (DL / 4) + lane + 32 * i);
                    }
                }
                const float m_old = m;
#pragma unroll
                for (int k = 0; k < K; ++k) m = fmaxf(m, ml[k].x);
                const float al = scale_of(m_old, m);
                den *= al;
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = make_float4(al * o[i].x, al * o[i].y, al * o[i].z, al * o[i].w);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    if (ml[k].y == kNothing) continue;
                    const float a = scale_of(ml[k].x, m);
                    den = fmaf(a, ml[k].y, den);
#pragma unroll
                    for (int i = 0; i < N; ++i) add(o[i], a, v[k][i]);
                }
            }
#pragma unroll
            for (int i = 0; i < N; ++i) put(r, lane + 32 * i, o[i], den);
        }
        return;
    }
    for (int e = q; e < rows * (N / 2); e += Q) {
        const int r = e / (N / 2), i0 = e % (N / 2) * 2;
        float m = -INFINITY, den = 0.f;
        float4 o[2] = {};
        constexpr int kDeep = 4;
        for (int k0 = warp; k0 < n; k0 += kDeep * kWarps) {
            float2 ml[kDeep];
            float4 v[kDeep][2];
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                const int k = k0 + j * kWarps;
                ml[j] = make_float2(-INFINITY, kNothing);
                if (k < n) {
                    ml[j] = __ldcg(A.ml + slot(k, r));
#pragma unroll
                    for (int i = 0; i < 2; ++i) v[j][i] = __ldcg(acc + slot(k, r) * (DL / 4) + lane + 32 * (i0 + i));
                }
            }
            const float m_old = m;
#pragma unroll
            for (int j = 0; j < kDeep; ++j) m = fmaxf(m, ml[j].x);
            const float al = scale_of(m_old, m);
            den *= al;
#pragma unroll
            for (int i = 0; i < 2; ++i) o[i] = make_float4(al * o[i].x, al * o[i].y, al * o[i].z, al * o[i].w);
#pragma unroll
            for (int j = 0; j < kDeep; ++j) {
                if (ml[j].y == kNothing) continue;
                const float a = scale_of(ml[j].x, m);
                den = fmaf(a, ml[j].y, den);
#pragma unroll
                for (int i = 0; i < 2; ++i) add(o[i], a, v[j][i]);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) S.part[warp][i][lane] = o[i];
        if (lane == 0) S.dens[warp] = make_float2(m, den);
        __syncthreads();
        if (warp < 2) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, S.dens[w].x);
            float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
            den = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float a = scale_of(S.dens[w].x, M);
                den = fmaf(a, S.dens[w].y, den);
                add(t, a, S.part[w][warp][lane]);
            }
            put(r, lane + 32 * (i0 + warp), t, den);
        }
    }
}

// Zeros in the rows that merge_unit would have written.
template <int DL, int ROWS, int THREADS>
__device__ __forceinline__ void clear_unit(const Args &A, const int4 job, int q, int Q)
{
    constexpr int kWarps = THREADS / 32, N = DL / 256;  // stretches of 256 coordinates of a row, a uint4 per lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row0 = job.w * ROWS, rows = min(ROWS, A.R - row0);
    uint4 *out = reinterpret_cast<uint4 *>(A.out + (static_cast<size_t>(job.z) * A.R + row0) * DL) + lane;
    const bool few = job.y <= kFewPieces;
    for (int e = few ? (warp * Q + q) * N : q; e < rows * N; e += few ? kWarps * Q * N : Q)
        if (few || warp == 0)
            for (int i = 0; i < (few ? N : 1); ++i) out[(e + i) * 32] = make_uint4(0u, 0u, 0u, 0u);
}

// The end of a block (part of `parts` of worker w) whose pieces are all written: says so to the workers that it shares units
// with, waits for theirs, and joins its part of them.  The wait is for blocks of the same launch, which all run at once
// (launch_together), and whose own waits are bounded.  Shares are equal, so what another block may still need grows with what
// this one took since `born`: the handle's wait limit, and as much again for each time that the default limit has passed
// meanwhile.  A block that gives up reports it and writes zeros.  The caller has synchronised the block behind its last
// writes, so that the release covers them all.
template <int DL, int ROWS, int THREADS>
__device__ __forceinline__ void join(const Args &A, const int4 *jobs, int w, int part, int parts, long long born, Merge &S)
{
    if (threadIdx.x == 0)
        for (int i = 0; i < 2; ++i)
            if (jobs[i].y > 1) asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(A.done + jobs[i].x) : "memory");
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        const int4 job = jobs[i];
        if (job.y < 2) continue;
        bool late = false;
        if (threadIdx.x == 0) {
            const long long t0 = clock64();
            const float limit = static_cast<float>(A.wait_limit) * (1.f + static_cast<float>(t0 - born) * (1.f / kDefaultWaitLimit));
            for (;;) {
                int have;
                asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(have) : "l"(A.done + job.x) : "memory");
                if (have >= job.y * parts) break;
                if (static_cast<float>(clock64() - t0) >= limit) {
                    late = true;
                    atomicOr(A.status, TQ_DEVERR_TIMEOUT);
                    break;
                }
            }
        }
        const int q = (w - job.x) * parts + part, Q = job.y * parts;
        if (__syncthreads_or(late)) clear_unit<DL, ROWS, THREADS>(A, job, q, Q);
        else merge_unit<DL, ROWS, THREADS>(A, job, q, Q, S);
    }
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

// Launches `workers` workers of `size` blocks (a cluster), or as many as fit on the SMs that the stream may use where those are
// fewer (a limited context): they all run at once, for they wait for one another before the pieces are joined.  The query takes
// 0.15 us.
template <typename... P, typename... V>
cudaError_t launch_together(void (*kernel)(P...), int size, int threads, size_t smem, cudaStream_t st, Args a, V... maps)
{
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(size);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(size * a.workers);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int fit = 0;
    e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (fit < a.least_workers) return cudaErrorCooperativeLaunchTooLarge;
    if (fit < a.workers) a.workers = fit;
    cfg.gridDim = dim3(size * a.workers);
    attr = {};
    attr.id = cudaLaunchAttributeCooperative;
    attr.val.cooperative = 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps..., a);
}

// The narrow kernel's launch, in its own translation unit; tk: boxes of a group's blocks (narrow_group), tq: 64 rows.
int narrow_group(int dl);
cudaError_t launch_narrow(const CUtensorMap &tk, const CUtensorMap &tq, int dl, const Args &a, cudaStream_t st);

}  // namespace latent
}  // namespace tq
