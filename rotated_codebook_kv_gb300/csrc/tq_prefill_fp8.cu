// tq_prefill_fp8.cu -- causal attention of the last tokens of every sequence over 8-bit
// pages, on the 5th-generation tensor cores.
//
//   S[c][t] = <q_c 2^e, kc_t>          kind::f8f6f4: the key codes as stored, q 2^e as two e4m3 terms (exact,
//                                      see tq_decode_fp8.cu), M = 128 columns c, N = KT tokens t
//   O[c][j] += sum_t P[c][t] vc_t[j]   kind::f16: P in fp16 from tensor memory, the value codes widened to fp16
//                                      (exact) in shared memory, N = D coordinates j
// with y = sm_scale log2(e) 2^-e ks[page] S + log2 vs[page], P = 2^(y - m), m a running maximum that is
// only moved when the maximum has grown far beyond it (below), and the
// denominator the sum of kSumUnit P / vs in fp32.
//
// A CTA takes NQ tiles of 128 columns, (query token, head) pairs of one sequence and kv head, and the
// KT-token tiles that they see (of units behind the last whole wave: a piece of those).  Two tiles at head
// dim 128: while one's scores are turned into P, the tensor core works for the other.  At head dim 256 tensor
// memory holds one tile's O (256 columns), two score buffers and the query terms (128).  P overwrites the scores
// that it came from.
//
// Warps (one CTA per SM):
//   4 NQ      one thread per column: online softmax, output (and, with the next ones, the query operands at first)
//   4         value codes of a tile to fp16 (rows of 64 coordinates, 128-byte swizzle, one row per token)
//   1 + NQ    MMA issue: the scores (and tensor-memory allocation); P.V of a column tile each
//   1         page copies (TMA boxes of a page x 128 bytes, 128-byte swizzle), scales
// Every wait is bounded by the handle's wait limit; a timeout sets TQ_DEVERR_TIMEOUT, stops the CTA (its rows
// then carry no weight), lets copies and MMAs in flight finish, and frees tensor memory.
//
// Bound: the softmax warps.  Measured on a GB300: the last 4096 of 16,384 tokens, 32 query and 8 kv heads of 128, 828 us =
// 1.16 PFLOP/s of useful products (cuBLAS bf16: 1.91), 756 steps of a tile pair an SM, 1.1 us each, half of which the tensor
// pipe is active; 64 tokens of 32 sequences of 1024 to 8192 195 us; the last 1000 of 2 sequences of 5000 to 8192, 16 and 8
// heads of 256, 214 us.
#include <climits>

#include "tq_fp8.cuh"
#include "tq_umma.cuh"

namespace tq {
namespace fp8 {
namespace {

template <int D>
struct Tc {
    static constexpr int NQ = D == 128 ? 2 : 1;         // column tiles
    static constexpr int KT = 64;                       // tokens per tile
    static constexpr int NB = 2;                        // score buffers per column tile
    static constexpr bool kQTm = NQ == 1;               // query operands in tensor memory (two column tiles leave no room)
    static constexpr int XB = D / 128;                  // 128-byte column blocks of a row of codes
    static constexpr int kSoftWarps = 4 * NQ;
    static constexpr int kConvWarps = 4;
    static constexpr int kMmaWarp = kSoftWarps + kConvWarps;  // scores; then a warp per column tile for P.V
    static constexpr int kLoadWarp = kMmaWarp + 1 + NQ;
    static constexpr int kThreads = 32 * (kMmaWarp + 4);  // whole warpgroups (one idle warp at head dim 256)
    // registers: 512 threads start with 128 each; the column warps take 192 and leave 64 to the others
    // (2 x 128 x 192 + 2 x 128 x 64 = 512 x 128).  384 threads have 168 each and keep them.
    static constexpr bool kSplitRegs = NQ == 2;
    static constexpr int KS = 4, RS = 3, VS = 3;  // stages: keys, value codes, fp16 values
    static constexpr int GR = KT / 16;                  // 16-token groups of a tile (a page holds one or two)
    static constexpr int kRing = 8;                     // tiles whose scales are kept
    static constexpr uint32_t kQBytes = 128u * D;       // one term of one column tile
    static constexpr uint32_t kKBytes = static_cast<uint32_t>(KT) * D;
    static constexpr uint32_t kQOff = 0;
    static constexpr uint32_t kKOff = kQOff + (kQTm ? 0 : 2 * NQ * kQBytes);
    static constexpr uint32_t kROff = kKOff + KS * kKBytes;
    static constexpr uint32_t kVOff = kROff + RS * kKBytes;
    static constexpr uint32_t kInfoOff = kVOff + VS * 2 * kKBytes;  // [ring][GR] (ks, log2 vs, kSumUnit / vs, -)
    static constexpr uint32_t kOkOff = kInfoOff + kRing * GR * 16;  // [ring] bit g: group g's page is valid
    static constexpr uint32_t kBarOff = kOkOff + kRing * 4;
    // barriers
    static constexpr int bQ = 0;                 // query terms in shared memory, and every column's factor
    static constexpr int bQTm = 1;               // query terms in tensor memory
    static constexpr int bKFull = 2;             // [KS] keys landed (one arrival, and bytes)
    static constexpr int bKFree = bKFull + KS;   // [KS] the score MMAs of every tile are done
    static constexpr int bRFull = bKFree + KS;   // [RS] value codes landed
    static constexpr int bRFree = bRFull + RS;   // [RS] widened
    static constexpr int bVFull = bRFree + RS;   // [VS] fp16 values ready
    static constexpr int bVFree = bVFull + VS;   // [VS] the P.V MMAs of every tile are done
    static constexpr int bSFull = bVFree + VS;   // [NQ][NB] scores in tensor memory
    static constexpr int bPFull = bSFull + NQ * NB;  // [NQ][NB] P in tensor memory, O rescaled
    static constexpr int bPvDone = bPFull + NQ * NB;  // [NQ][NB] O += P V of a score buffer's P done
    static constexpr int bEnd = bPvDone + NQ * NB;    // teardown: every MMA issued is done
    static constexpr int kBars = bEnd + 1;
    static constexpr uint32_t kMiscOff = kBarOff + 8 * kBars;  // tensor-memory base, abort flag
    static constexpr uint32_t kNanOff = (kMiscOff + 8 + 15) / 16 * 16;  // [D] first token behind a causal limit with a NaN value
    static constexpr uint32_t kFacOff = kNanOff + 4 * D;  // [128 NQ] sm_scale log2(e) 2^-e of a column
    static constexpr uint32_t kStageOff = kQTm ? kVOff : kQOff;  // query terms on their way to tensor memory; output rows
    static constexpr size_t kSmem = 1024 + kFacOff + 4 * 128 * NQ;
    // tensor-memory columns
    static constexpr uint32_t kTmS = 0;                              // [NQ][NB] KT columns
    static constexpr uint32_t kTmQ = NQ * NB * KT;                   // D / 4 columns of either term
    static constexpr uint32_t kTmO = kTmQ + (kQTm ? D / 2 : 0);      // [NQ] D columns
    static constexpr uint32_t kTmCols = 512;
    static_assert(KT == 64, "the softmax holds a column's 64 scores");
    static_assert(KS + NB < kRing, "a tile's scales are written over those of a tile that every column is done with");
    static_assert(kTmO + NQ * D <= kTmCols, "tensor memory");
    static_assert(kSmem <= 232448, "shared memory");
};

// The reference m of a column's probabilities is set 2^4 below the scores' maximum and O rescaled only when the maximum
// has since passed m by kLazy (log2 units): the largest P = 2^(y - m) so far lies in 2^4 .. 2^15 (fp16 ends at 65504), so
// that everything down to 2^-18 of it keeps 11 bits and a P is never off by more than 2^-29 of it (2^17 tokens behind a
// strong one: 2^-12 of that in all; with m above the maximum their sum lost a tenth).  A rescale waits for the tensor core
// and moves all of O, so a few strong tokens in every tile made it the longest step of many tiles.  Long prefill below, the
// same with 2^-1 | 2^2 | 2^4 | 2^6 | 2^8: 814 | 822 | 825 | 828 | 832 us; 64 tokens of 32 sequences 187 | 190 | 195 | 196 | 198.
constexpr float kAim = -4.f, kLazy = 15.f;
// Value scales may lie 2^220 apart (an empty page's is 2^-100), and then the P = 2^(y - m) of a page of small values, which its
// part of the denominator is made from, below what fp32 holds: a tile with a group of 16 tokens whose P are all below
// 2^kFar is looked through for those, and the factors of a rescale and of the merge are taken as squares of their roots.
constexpr float kFar = -60.f;

__device__ __forceinline__ uint32_t saddr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void warp_arrive(uint64_t *mb)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(mb)) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t pair)
{
    uint32_t h;
    const uint16_t c = static_cast<uint16_t>(pair);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(c));
    return h;
}

__device__ __forceinline__ uint32_t half2_of(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 lanes side by side: one issue slot for two multiply-adds or sums.
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

// A column's 64 scores of a tile, and the tile's scales: a = fac ks, b = log2 vs, inv = kSumUnit / vs per 16 tokens.
struct Scores {
    uint32_t v[64];
    float a[4], b[4], inv[4];
};

// The largest y of the tile, and the least of its groups' largest.  WHOLE: every token is seen, else those below rem of the
// groups in okm.
template <bool WHOLE>
__device__ __forceinline__ float tile_max(const Scores &s, uint32_t okm, int rem, float &low)
{
    float top = -INFINITY;
    low = INFINITY;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
        for (int k = 16 * g; k < 16 * g + 16; k += 4) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = WHOLE || k + j < rem ? __uint_as_float(s.v[k + j]) : -INFINITY;
            m0 = max3(m0, x[0], x[1]);
            m1 = max3(m1, x[2], x[3]);
        }
        m0 = fmaxf(m0, m1);
        if (WHOLE || ((okm >> g & 1u) && m0 != -INFINITY)) {
            const float y = fmaf(m0, s.a[g], s.b[g]);
            top = fmaxf(top, y);
            low = fminf(low, y);
        }
    }
    return top;
}

// P = 2^(y - ref) in fp16, two tokens per word; returns the sum of kSumUnit P / vs.
template <bool WHOLE>
__device__ __forceinline__ float tile_exp(const Scores &s, uint32_t (&p)[32], float ref, uint32_t okm, int rem)
{
    float l = 0.f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const float sh = s.b[g] - ref;
        const uint64_t a2 = pack2(s.a[g], s.a[g]), sh2 = pack2(sh, sh);
        const bool gok = WHOLE || (okm >> g & 1u);
        uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
        for (int k = 16 * g; k < 16 * g + 16; k += 4) {
            float2 x0 = unpack2(fma2(pack2(__uint_as_float(s.v[k]), __uint_as_float(s.v[k + 1])), a2, sh2));
            float2 x1 = unpack2(fma2(pack2(__uint_as_float(s.v[k + 2]), __uint_as_float(s.v[k + 3])), a2, sh2));
            x0.x = fast_exp2(x0.x);
            x0.y = fast_exp2(x0.y);
            x1.x = fast_exp2(x1.x);
            x1.y = fast_exp2(x1.y);
            if (!WHOLE) {
                if (!gok || k >= rem) x0.x = 0.f;
                if (!gok || k + 1 >= rem) x0.y = 0.f;
                if (!gok || k + 2 >= rem) x1.x = 0.f;
                if (!gok || k + 3 >= rem) x1.y = 0.f;
            }
            sum0 = add2(sum0, pack2(x0.x, x0.y));
            sum1 = add2(sum1, pack2(x1.x, x1.y));
            p[k / 2] = half2_of(x0.x, x0.y);
            p[k / 2 + 1] = half2_of(x1.x, x1.y);
        }
        const float2 t = unpack2(add2(sum0, sum1));
        if (gok) l = fmaf(t.x + t.y, s.inv[g], l);
    }
    return l;
}

// What tile_exp leaves out of a column's denominator: the P below 2^-126 (2^180 times them are summed).  The scores come from
// tensor memory once more, a group at a time: a second way through tile_exp made every tile 3 % slower, this after tile_exp as
// well.
__device__ __forceinline__ float flushed_part(uint32_t ts, const float4 *info, float fac, uint32_t okm, int rem, float ref)
{
    float l = 0.f;
#pragma unroll 1
    for (int g = 0; g < 4; ++g) {
        float v[16];
        umma::ld16(ts + 16 * g, v);
        const float4 f = info[g];
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            const float y = fmaf(v[k], fac * f.x, f.y - ref);
            if (y < -126.f && 16 * g + k < rem) sum += fast_exp2(y + 180.f);
        }
        if (okm >> g & 1u) l = fmaf(sum * 0x1p-58f * f.z, 0x1p-122f, l);  // in an order that keeps to fp32's range
    }
    return l;
}

template <int D>
__global__ void __launch_bounds__(Tc<D>::kThreads, 1)
    prefill_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Args A)
{
    using T = Tc<D>;
    constexpr int NQ = T::NQ, KT = T::KT, NB = T::NB, XB = T::XB, GR = T::GR;
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // The units that fill whole waves of CTAs stay whole; the ones behind them are cut into A.splits pieces.
    // The query blocks of one sequence and kv head are neighbours (they share its pages in L2), the longest first.
    const int at = static_cast<int>(blockIdx.x) - A.whole;
    const int unit = at < 0 ? static_cast<int>(blockIdx.x) : A.whole + at / A.splits, split = at < 0 ? 0 : at % A.splits;
    const bool uncut = at < 0 || A.splits == 1;
    const int qt = A.nqt - 1 - unit % A.nqt, kvh = unit / A.nqt % A.Hkv, b = unit / A.nqt / A.Hkv;
    const int G = A.G, P = A.P;
    int L = A.seq_lens[b];
    if (L < 0) L = 0;
    if (L > A.max_blocks * P) {
        if (split == 0 && kvh == 0 && qt == 0 && tid == 0) atomicOr(A.status, TQ_DEVERR_SEQ_RANGE);
        L = A.max_blocks * P;
    }
    const int q0 = qt * A.qpc;
    const int ncol = min(A.qpc, A.Tq - q0) * G;
    const int ginv = (65536 + G - 1) / G;  // c / G = c ginv >> 16 for c < 256
    auto col_row = [&](int c) -> size_t {
        const int t = c * ginv >> 16;
        return (static_cast<size_t>(b) * A.Tq + q0 + t) * A.Hq + static_cast<size_t>(kvh) * G + (c - t * G);
    };
    auto col_lim = [&](int c) -> int { return max(0, L - A.Tq + q0 + (c * ginv >> 16) + 1); };
    const size_t rows_total = static_cast<size_t>(A.B) * A.Tq * A.Hq;
    const int tok0 = split * A.pages_per_split * P;
    const int tok1 = min(col_lim(ncol - 1), uncut ? A.max_blocks * P : tok0 + A.pages_per_split * P);
    auto dead_row = [&](int c) {  // a row that this CTA has nothing for
        const size_t rr = col_row(c);
        if (uncut) {
            uint4 *dst = reinterpret_cast<uint4 *>(A.out + rr * D);
            for (int i = 0; i < D / 8; ++i) dst[i] = make_uint4(0u, 0u, 0u, 0u);
        } else {
            float *ml = A.ml + (static_cast<size_t>(split) * rows_total + rr) * 2;
            ml[0] = -INFINITY;
            ml[1] = 0.f;
        }
    };
    if (tok0 >= tok1) {
        for (int c = tid; c < ncol; c += T::kThreads) dead_row(c);
        return;
    }
    int nt[NQ];  // token tiles that a column tile sees
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const int last = min(ncol, 128 * (q + 1)) - 1;
        nt[q] = last < 128 * q ? 0 : max(0, (min(col_lim(last), tok1) - tok0 + KT - 1) / KT);
    }
    const int nt_all = (tok1 - tok0 + KT - 1) / KT;

    uint64_t *mbar = reinterpret_cast<uint64_t *>(smem + T::kBarOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + T::kMiscOff);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + T::kMiscOff + 4);
    const uint32_t sbase = saddr(smem);
    int *nan_at = reinterpret_cast<int *>(smem + T::kNanOff);
    const int ppt = KT / P;  // pages per tile

    if (warp == T::kMmaWarp) umma::tmem_alloc(tmem_slot, T::kTmCols);
    if (tid < D) nan_at[tid] = INT_MAX;
    if (tid == 0) {
        umma::mbar_init(&mbar[T::bQ], T::kMmaWarp);
        umma::mbar_init(&mbar[T::bQTm], T::kSoftWarps);
        for (int i = 0; i < T::KS; ++i) {
            umma::mbar_init(&mbar[T::bKFull + i], 1);
            umma::mbar_init(&mbar[T::bKFree + i], 1);
        }
        for (int i = 0; i < T::RS; ++i) {
            umma::mbar_init(&mbar[T::bRFull + i], 1);
            umma::mbar_init(&mbar[T::bRFree + i], T::kConvWarps);
        }
        for (int i = 0; i < T::VS; ++i) {
            umma::mbar_init(&mbar[T::bVFull + i], T::kConvWarps);
            umma::mbar_init(&mbar[T::bVFree + i], NQ);
        }
        for (int i = 0; i < NQ * NB; ++i) {
            umma::mbar_init(&mbar[T::bSFull + i], 1);
            umma::mbar_init(&mbar[T::bPFull + i], 4);
            umma::mbar_init(&mbar[T::bPvDone + i], 1);
        }
        umma::mbar_init(&mbar[T::bEnd], 1 + NQ);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tbase = *tmem_slot;

    // bounded wait: gives up on the CTA's abort flag or after the wait limit (then raising the flag and the
    // status bit); a zero limit tests once
    auto wait_bar = [&](int i, uint32_t par) -> bool {
        uint64_t *mb = &mbar[i];
        bool ok = umma::mbar_test_wait(mb, par);
        if (__all_sync(0xffffffffu, ok)) return true;  // the usual way, without a look at the clock
        if (A.wait_limit > 0) {
            const long long t0 = clock64();
            while (!(ok = umma::mbar_try_wait_for(mb, par, 10000))) {
                if (*abort_flag || clock64() - t0 > A.wait_limit) break;
            }
        }
        if (!ok && !*abort_flag) {
            *abort_flag = 1;
            atomicOr(A.status, TQ_DEVERR_TIMEOUT);
        }
        return __all_sync(0xffffffffu, ok);  // the lanes poll separately: decide as a warp
    };

    // the same by one thread alone
    auto wait_one = [&](int i, uint32_t par) -> bool {
        uint64_t *mb = &mbar[i];
        if (A.wait_limit > 0 ? umma::mbar_try_wait(mb, par) : umma::mbar_test_wait(mb, par)) return true;
        const long long t0 = clock64();
        while (A.wait_limit > 0 && !*abort_flag && clock64() - t0 <= A.wait_limit)
            if (umma::mbar_try_wait(mb, par)) return true;
        if (!*abort_flag) {
            *abort_flag = 1;
            atomicOr(A.status, TQ_DEVERR_TIMEOUT);
        }
        return false;
    };

    float *s_fac = reinterpret_cast<float *>(smem + T::kFacOff);
    if (warp < T::kMmaWarp) {
        // ================= query operands =================
        // Coordinates 8 j .. 8 j + 7 of a row by lane j of its D / 8 lanes.  All rows of a warp are copied first, each to where
        // its two terms go (which take the same bytes), so that one latency is paid; then a short loop splits them.  A
        // thread per row, all unrolled, took 10-14 thousand cycles of a unit's 240: ~2000 instructions that run once, and
        // loads that touch 32 rows each.
        constexpr int kLanes = D / 8, kRows = 32 / kLanes;
        const int j = lane % kLanes, sub = lane / kLanes;
        auto row_at = [&](int c) -> uint32_t { return T::kQTm ? T::kStageOff + c * 512 : T::kQOff + 2 * (c >> 7) * T::kQBytes + (c & 127) * 128; };
        constexpr uint32_t kLo = T::kQTm ? 256 : T::kQBytes;  // from the first term to the second
        const uint32_t raw = (j & 7) * 16 + (T::kQTm ? (j >> 3) * 128 : (j >> 3) * kLo);
#pragma unroll 2
        for (int n = warp; n < 128 * NQ / kRows; n += T::kMmaWarp) {
            const int c = n * kRows + sub;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                         ::"r"(sbase + row_at(c) + raw), "l"(A.q + col_row(c < ncol ? c : 0) * D + 8 * j), "r"(c < ncol ? 16 : 0) : "memory");
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 2
        for (int n = warp; n < 128 * NQ / kRows; n += T::kMmaWarp) {
            const int c = n * kRows + sub;
            const uint4 w = lds128(sbase + row_at(c) + raw);  // what this lane copied
            const uint32_t v[4] = {w.x, w.y, w.z, w.w};
            uint32_t m = __vmaxu2(__vmaxu2(v[0] & 0x7fff7fffu, v[1] & 0x7fff7fffu), __vmaxu2(v[2] & 0x7fff7fffu, v[3] & 0x7fff7fffu));
            m = max(m & 0xffffu, m >> 16);  // the largest magnitude's bits
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
            const int ex = min(max(static_cast<int>(m >> 7) - 127, -100), 127);  // 2^(7 - ex) brings the largest into [2^7, 2^8)
            float up = __uint_as_float(static_cast<uint32_t>(7 - ex + 127) << 23);
            if (j == 0)  // >= 0: a negative scale goes into q's sign; an infinity or NaN makes the row NaN
                s_fac[c] = m >= 0x7f80u ? __uint_as_float(0x7fc00000u)
                                        : fabsf(A.sm_scale) * kLog2e * __uint_as_float(static_cast<uint32_t>(ex - 7 + 127) << 23);
            if (A.sm_scale < 0.f) up = -up;
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float x0 = __uint_as_float(v[2 * k] << 16) * up, x1 = __uint_as_float(v[2 * k] & 0xffff0000u) * up;
                float x2 = __uint_as_float(v[2 * k + 1] << 16) * up, x3 = __uint_as_float(v[2 * k + 1] & 0xffff0000u) * up;
                hi[k] = e4m3x2_rest(x0, x1);
                hi[k] |= e4m3x2_rest(x2, x3) << 16;
                lo[k] = e4m3x2(x0, x1) | (e4m3x2(x2, x3) << 16);
            }
            // chunks of 16 coordinates, the 128-byte swizzle of the operand
            const uint32_t at = row_at(c) + (((j >> 1) ^ (c & 7)) << 4) + 8 * (j & 1);
            __syncwarp();  // every lane of the row has read
            *reinterpret_cast<uint2 *>(smem + at) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(smem + at + kLo) = make_uint2(lo[0], lo[1]);
        }
        if constexpr (!T::kQTm) umma::fence_proxy_async();
        warp_arrive(&mbar[T::bQ]);
    }
    if constexpr (T::kSplitRegs) {
        if (warp < T::kSoftWarps) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    }
    if (warp < T::kSoftWarps) {
        // ================= columns: query operands, softmax, output =================
        const int q = warp >> 2, r = tid & 127, c = 128 * q + r;
        const bool cv = c < ncol;
        const uint32_t lane_base = tbase + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        bool ok = wait_bar(T::bQ, 0);
        const float fac = s_fac[c];
        if constexpr (T::kQTm) {
            if (ok) {
                const uint32_t row = sbase + T::kStageOff + r * 512;
#pragma unroll 1
                for (int x = 0; x < 4; ++x) {  // 128 coordinates of a term
                    uint32_t w[32];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint4 v = lds128(row + (((8 * x + i) ^ (r & 7)) << 4));
                        w[4 * i] = v.x;
                        w[4 * i + 1] = v.y;
                        w[4 * i + 2] = v.z;
                        w[4 * i + 3] = v.w;
                    }
                    umma::st32(lane_base + T::kTmQ + 32 * x, w);
                }
                umma::wait_st();
                umma::fence_before_sync();
                warp_arrive(&mbar[T::bQTm]);
            }
        }
        const int lim = cv ? min(col_lim(c), tok1) : tok1;  // an idle column (zero query) goes the way of the full ones
        const int my_nt = q ? nt[NQ - 1] : nt[0];
        float m_run = -INFINITY, l_run = 0.f;
        for (int i = 0; ok && i < my_nt; ++i) {
            if (!(ok = wait_bar(T::bSFull + q * NB + i % NB, (i / NB) & 1))) break;
            umma::fence_after_sync();
            const uint32_t ts = lane_base + T::kTmS + (q * NB + i % NB) * KT;
            Scores s;
            const float4 *info = reinterpret_cast<const float4 *>(smem + T::kInfoOff) + (i % T::kRing) * GR;
#pragma unroll
            for (int g = 0; g < GR; ++g) {
                const float4 f = info[g];
                s.a[g] = fac * f.x;
                s.b[g] = f.y;
                s.inv[g] = f.z;
            }
            const uint32_t okm = reinterpret_cast<const uint32_t *>(smem + T::kOkOff)[i % T::kRing];
            const int rem = lim - (tok0 + i * KT);  // tokens of the tile that this column sees
            const bool whole = __all_sync(0xffffffffu, rem >= KT) && okm == (1u << GR) - 1u;
            umma::ld64(ts, s.v);
            float low;
            const float top = whole ? tile_max<true>(s, okm, rem, low) : tile_max<false>(s, okm, rem, low);
            // ---- lazy rescale ----
            const bool need = m_run != -INFINITY && top > m_run + kLazy;
            if (m_run == -INFINITY) m_run = top + kAim;  // O's row is zero or unwritten so far
            if (__any_sync(0xffffffffu, need)) {
                if (i > 0 && !(ok = wait_bar(T::bPvDone + q * NB + (i - 1) % NB, ((i - 1) / NB) & 1))) break;  // O is at rest
                umma::fence_after_sync();
                const float root = need ? fast_exp2(0.5f * (m_run - (top + kAim))) : 1.f, al = root * root;
                const uint32_t to = lane_base + T::kTmO + q * D;
#pragma unroll 1
                for (int ch = 0; ch < D; ch += 64) {
                    uint32_t o[64];
                    umma::ld64(to + ch, o);
#pragma unroll
                    for (int k = 0; k < 64; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
                    umma::st64(to + ch, o);
                }
                umma::wait_st();
                l_run = l_run * root * root;  // see kFar
                if (need) m_run = top + kAim;
            }
            if (__any_sync(0xffffffffu, low < m_run + kFar)) l_run += flushed_part(ts, info, fac, okm, rem, m_run);
            // ---- P = 2^(y - m) over the scores ----
            const float ref = m_run == -INFINITY ? 0.f : m_run;
            uint32_t p[32];
            l_run += whole ? tile_exp<true>(s, p, ref, okm, rem) : tile_exp<false>(s, p, ref, okm, rem);
            umma::st32(ts, p);
            umma::wait_st();
            umma::fence_before_sync();
            warp_arrive(&mbar[T::bPFull + q * NB + i % NB]);
        }
        if (ok && my_nt > 0) ok = wait_bar(T::bPvDone + q * NB + (my_nt - 1) % NB, ((my_nt - 1) / NB) & 1);
        if (ok && my_nt > 0) {
            umma::fence_after_sync();
            const size_t rr = col_row(cv ? c : 0);
            const float inv = l_run == 0.f ? 0.f : kSumUnit / l_run;
            bool nan = false;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) nan |= nan_at[32 * k + lane] != INT_MAX;
            nan = __any_sync(0xffffffffu, nan);
            // through shared memory, so that the lanes of a warp write whole rows (a row per thread: 6 thousand cycles)
            const uint32_t stage = sbase + T::kStageOff + (128 * q + 32 * (warp & 3)) * (2 * D);  // 32 rows of 2 D bytes
            auto fetch = [&](int col, uint32_t (&o)[32]) {  // 32 coordinates of O, NaN where the column sees one
                umma::ld32_issue(lane_base + T::kTmO + q * D + col, o);
                umma::wait_ld32(o);
                if (!nan) return;
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    const int4 at = *reinterpret_cast<const int4 *>(nan_at + col + k);
                    if (at.x < lim) o[k] = 0x7fffffffu;
                    if (at.y < lim) o[k + 1] = 0x7fffffffu;
                    if (at.z < lim) o[k + 2] = 0x7fffffffu;
                    if (at.w < lim) o[k + 3] = 0x7fffffffu;
                }
            };
            auto put = [&](int chunk, uint4 v) { sts128(stage + lane * (2 * D) + ((chunk ^ (lane & 7)) << 4), v); };
            auto write_rows = [&](char *base, size_t pitch) {  // row rr of 2 D bytes at base + rr pitch
                __syncwarp();
                constexpr int kLanes = D / 8, kRows = 32 / kLanes;
                const int piece = lane % kLanes;
#pragma unroll 4
                for (int n0 = 0; n0 < 32; n0 += kRows) {
                    const int n = n0 + lane / kLanes;
                    const size_t at = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(rr), n);
                    if (128 * q + 32 * (warp & 3) + n < ncol)
                        *reinterpret_cast<uint4 *>(base + at * pitch + 16 * piece) = lds128(stage + n * (2 * D) + ((piece ^ (n & 7)) << 4));
                }
                __syncwarp();
            };
            if (uncut) {
#pragma unroll 1
                for (int col = 0; col < D; col += 32) {
                    uint32_t o[32];
                    fetch(col, o);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t w[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m)  // with nothing seen O is zero
                            w[m] = bf16x2_of(__uint_as_float(o[8 * k + 2 * m]) * inv, __uint_as_float(o[8 * k + 2 * m + 1]) * inv);
                        put(col / 8 + k, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                }
                write_rows(reinterpret_cast<char *>(A.out), 2 * D);
            } else {
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += D / 2) {  // half a row of sums fits
#pragma unroll 1
                    for (int col = 0; col < D / 2; col += 32) {
                        uint32_t o[32];
                        fetch(c0 + col, o);
#pragma unroll
                        for (int k = 0; k < 8; ++k) put(col / 4 + k, make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]));
                    }
                    write_rows(reinterpret_cast<char *>(A.acc + static_cast<size_t>(split) * rows_total * D + c0), 4 * D);
                }
            }
            if (cv && !uncut) {
                float *ml = A.ml + (static_cast<size_t>(split) * rows_total + rr) * 2;
                ml[0] = m_run;
                ml[1] = l_run;
            }
        } else if (cv && my_nt == 0) {
            dead_row(c);
        }
        umma::fence_before_sync();
    } else if (warp < T::kMmaWarp) {
        // ================= value codes to fp16 =================
        // item (token t, chunk of 16 codes): eight lanes take four chunks of tokens t and t ^ 5, whose reads
        // and writes fall in eight different 16-byte bank groups
        const int ct = tid - 32 * T::kSoftWarps;
        const int hi = (ct >> 3) % (2 * XB), tp = ct / (16 * XB), x = hi >> 1, ch = 4 * (hi & 1) + (ct & 3);
        const int t = 8 * (tp >> 2) + ((ct & 4) ? (tp & 3) ^ 5 : tp & 3);  // further items: 16 / XB tokens on
        const uint32_t off_raw = x * (KT * 128) + t * 128 + ((ch ^ (t & 7)) << 4);
        const uint32_t off_dst = (2 * x + (ch >> 2)) * (KT * 128) + t * 128;
        const uint32_t off0 = off_dst + (((2 * (ch & 3)) ^ (t & 7)) << 4), off1 = off_dst + (((2 * (ch & 3) + 1) ^ (t & 7)) << 4);
        const bool go = !T::kQTm || wait_bar(T::bQTm, 0);  // the query terms went through these stages
        for (int i = 0; go && i < nt_all; ++i) {
            if (!wait_bar(T::bRFull + i % T::RS, (i / T::RS) & 1)) break;
            if (i >= T::VS && !wait_bar(T::bVFree + i % T::VS, (i / T::VS - 1) & 1)) break;
            const uint32_t raw = sbase + T::kROff + (i % T::RS) * T::kKBytes + off_raw;
            const uint32_t dst = sbase + T::kVOff + (i % T::VS) * 2 * T::kKBytes, dst0 = dst + off0, dst1 = dst + off1;
            const uint32_t okm = reinterpret_cast<const uint32_t *>(smem + T::kOkOff)[i % T::kRing];
            const int rem = tok1 - (tok0 + i * KT);
            const bool whole = rem >= KT && okm == (1u << GR) - 1u;
            const int seen = col_lim(0) - (tok0 + i * KT);  // tokens of the tile that every column sees
            // four reads ahead of their writes
#pragma unroll
            for (int n0 = 0; n0 < KT * D / 16 / (32 * T::kConvWarps); n0 += 4) {
                uint4 w[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int dt = (n0 + n) * (16 / XB);
                    w[n] = lds128(raw + dt * 128);
                    if (!whole && (t + dt >= rem || !(okm >> ((t + dt) >> 4) & 1u))) w[n] = make_uint4(0u, 0u, 0u, 0u);  // no token: holds anything
                }
                if (seen < KT) {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int dt = (n0 + n) * (16 / XB);
                        if (t + dt >= seen) hide_nan(w[n], nan_at + 128 * x + 16 * ch, tok0 + i * KT + t + dt);
                    }
                }
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const int dt = (n0 + n) * (16 / XB);
                    const uint32_t v[4] = {w[n].x, w[n].y, w[n].z, w[n].w};
                    uint32_t h[8];
#pragma unroll
                    for (int k2 = 0; k2 < 4; ++k2) {
                        h[2 * k2] = e4m3_to_half2(v[k2]);
                        h[2 * k2 + 1] = e4m3_to_half2(v[k2] >> 16);
                    }
                    sts128(dst0 + dt * 128, make_uint4(h[0], h[1], h[2], h[3]));
                    sts128(dst1 + dt * 128, make_uint4(h[4], h[5], h[6], h[7]));
                }
            }
            umma::fence_proxy_async();
            warp_arrive(&mbar[T::bRFree + i % T::RS]);
            warp_arrive(&mbar[T::bVFull + i % T::VS]);
        }
    } else if (warp < T::kLoadWarp) {
        // ================= MMA issue: a warp for the scores, one per column tile for P.V =================
        // Each has its own waits, so that work is queued at the tensor core while another one's operands are awaited.
        // One elected thread runs the loop: votes and converged issues around every wait had made a warp's round of
        // waits longer (~2000 cycles) than the MMAs of a tile (~1300).  Descriptors are built once; a step only adds to
        // their low words (the address in units of 16 bytes).
        if (umma::elect_one()) {
            if (warp == T::kMmaWarp) {
                constexpr uint32_t id_s = (1u << 4) | (static_cast<uint32_t>(KT >> 3) << 17) | (8u << 24);  // e4m3, fp32, M = 128
                const uint64_t dq = umma::make_desc_sw128(sbase + T::kQOff, 16, 1024);
                const uint64_t dk = umma::make_desc_sw128(sbase + T::kKOff, 16, 1024);
                const uint32_t q_lo = static_cast<uint32_t>(dq), k_lo = static_cast<uint32_t>(dk), hi = static_cast<uint32_t>(dk >> 32);
                bool ok = wait_one(T::kQTm ? T::bQTm : T::bQ, 0);
                for (int i = 0; ok && i < nt_all; ++i) {
                    const int st = i % T::KS, buf = i % NB;
                    ok = wait_one(T::bKFull + st, (i / T::KS) & 1);
#pragma unroll
                    for (int q = 0; q < NQ; ++q) {
                        if (!ok || i >= nt[q]) continue;
                        if (i >= NB && !(ok = wait_one(T::bPvDone + q * NB + buf, (i / NB - 1) & 1))) continue;
                        umma::fence_after_sync();
                        const uint32_t ka = k_lo + st * (T::kKBytes / 16), qa = q_lo + 2 * q * (T::kQBytes / 16);
                        const uint32_t ds = tbase + T::kTmS + (q * NB + buf) * KT;
#pragma unroll
                        for (int k = 0; k < D / 32; ++k) {
                            const uint32_t kd = ka + (k >> 2) * (KT * 8) + 2 * (k & 3), qd = qa + (k >> 2) * (128 * 8) + 2 * (k & 3);
                            if constexpr (T::kQTm) {
                                umma::mma_e4m3_tmem_a(ds, tbase + T::kTmQ + 8 * k, kd, hi, id_s, k > 0 ? 1 : 0);
                                umma::mma_e4m3_tmem_a(ds, tbase + T::kTmQ + D / 4 + 8 * k, kd, hi, id_s, 1);
                            } else {
                                umma::mma_e4m3_lohi(ds, qd, hi, kd, hi, id_s, k > 0 ? 1 : 0);
                                umma::mma_e4m3_lohi(ds, qd + T::kQBytes / 16, hi, kd, hi, id_s, 1);
                            }
                        }
                        umma::commit(&mbar[T::bSFull + q * NB + buf]);
                    }
                    umma::commit(&mbar[T::bKFree + st]);
                }
            } else {
                const int q = warp - T::kMmaWarp - 1;
                const int my_nt = q ? nt[NQ - 1] : nt[0];
                constexpr uint32_t id_o = umma::idesc_f16(128, 128) | (1u << 16);  // B along N
                const uint64_t dv = umma::make_desc_sw128(sbase + T::kVOff, KT * 128, 1024);
                const uint32_t v_lo = static_cast<uint32_t>(dv), hi = static_cast<uint32_t>(dv >> 32);
                const uint32_t tm_s = tbase + T::kTmS + q * NB * KT, tm_o = tbase + T::kTmO + q * D;
                for (int i = 0; i < nt_all; ++i) {
                    const int st = i % T::VS, buf = i % NB;
                    if (!wait_one(T::bVFull + st, (i / T::VS) & 1)) break;
                    if (i >= my_nt) {  // only the other column tile sees it: hand the stage on
                        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(&mbar[T::bVFree + st])) : "memory");
                        continue;
                    }
                    if (!wait_one(T::bPFull + q * NB + buf, (i / NB) & 1)) break;
                    umma::fence_after_sync();
                    const uint32_t va = v_lo + st * (2 * T::kKBytes / 16), tp = tm_s + buf * KT;
#pragma unroll
                    for (int k = 0; k < KT / 16; ++k)
#pragma unroll
                        for (int x = 0; x < XB; ++x)  // 128 coordinates at a time
                            umma::mma_f16_tmem_a(tm_o + 128 * x, tp + 8 * k, va + x * (2 * KT * 8) + 128 * k, hi, id_o,
                                                 (i > 0 || k > 0) ? 1 : 0);
                    umma::commit(&mbar[T::bPvDone + q * NB + buf]);
                    umma::commit(&mbar[T::bVFree + st]);
                }
            }
            // every MMA issued must be done before tensor memory is freed
            umma::commit(&mbar[T::bEnd]);
            const long long t0 = clock64();
            while (!umma::mbar_try_wait(&mbar[T::bEnd], 0) && clock64() - t0 < kDrainLimit) {
            }
        }
        __syncwarp();
    } else if (warp == T::kLoadWarp) {
        // ================= page copies and scales =================
        // The copies of all tiles go through this warp one after another, so little stands between two: block ids are
        // read three tiles ahead and scales two, and a tile's scales are written while the tile before it is copied.
        int k_issued = 0, r_issued = 0;
        const int32_t *table = A.block_table + static_cast<int64_t>(b) * A.max_blocks;
        const bool mine = lane < ppt;  // lane p: a tile's page p
        auto fetch_id = [&](int i) -> int {
            const int pos = tok0 + (i * ppt + lane) * P;
            return mine && pos < tok1 ? __ldg(table + (pos >> A.pshift)) : -1;
        };
        auto valid = [&](int blk) -> bool { return blk >= 0 && blk < A.num_blocks; };
        auto scale_of = [&](const float *p, int blk) -> float {
            return valid(blk) ? __ldg(p + static_cast<int64_t>(blk) * A.Hkv + kvh) : 0.f;
        };
        auto write_info = [&](int i, int blk, float ks, float vs) -> uint32_t {  // returns the tile's valid pages
            const bool good = valid(blk);
            if (mine && !good && tok0 + (i * ppt + lane) * P < tok1) atomicOr(A.status, TQ_DEVERR_BLOCK_RANGE);
            const uint32_t pages = __ballot_sync(0xffffffffu, good);
            const int slot = i % T::kRing;
            if (mine) {
                const float lv = log2_scale(vs);
                const float4 f = make_float4(ks, lv, fast_exp2(-lv) * kSumUnit, 0.f);
                float4 *info = reinterpret_cast<float4 *>(smem + T::kInfoOff) + slot * GR;
                if (P == 16) {
                    info[lane] = f;
                } else {
                    info[2 * lane] = f;
                    info[2 * lane + 1] = f;
                }
            }
            if (lane == 0)  // a bit per 16-token group
                reinterpret_cast<uint32_t *>(smem + T::kOkOff)[slot] = P == 16 ? pages : (pages & 1u) * 3u + (pages >> 1 & 1u) * 12u;
            return pages;
        };
        int blk = fetch_id(0), blk1 = fetch_id(1), blk2 = fetch_id(2);
        float ks1 = scale_of(A.k_scales, blk1), vs1 = scale_of(A.v_scales, blk1);
        uint32_t pages = write_info(0, blk, scale_of(A.k_scales, blk), scale_of(A.v_scales, blk));
        const uint32_t k_dst = sbase + T::kKOff + lane * P * 128, r_dst = sbase + T::kROff + lane * P * 128;
        for (int i = 0; i < nt_all; ++i) {
            const int blk3 = fetch_id(i + 3);
            const float ks2 = scale_of(A.k_scales, blk2), vs2 = scale_of(A.v_scales, blk2);
            const bool good = valid(blk);
            const int y = static_cast<int>((static_cast<int64_t>(blk) * A.Hkv + kvh) * P);
            const uint32_t bytes = __popc(pages) * static_cast<uint32_t>(P * D);
            auto copy = [&](const CUtensorMap &tm, uint32_t dst, int bar) {
                const uint32_t mb = saddr(&mbar[bar]);
                if (lane == 0)
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mb), "r"(bytes) : "memory");
                __syncwarp();
                if (good) {
#pragma unroll
                    for (int x = 0; x < XB; ++x)
                        asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                                     ::"r"(dst + x * (KT * 128)), "l"(reinterpret_cast<uint64_t>(&tm)), "r"(x * 128), "r"(y), "r"(mb)
                                     : "memory");
                }
            };
            if (i >= T::KS && !wait_bar(T::bKFree + i % T::KS, (i / T::KS - 1) & 1)) break;
            copy(tmK, k_dst + (i % T::KS) * T::kKBytes, T::bKFull + i % T::KS);
            k_issued = i + 1;
            if (i >= T::RS && !wait_bar(T::bRFree + i % T::RS, (i / T::RS - 1) & 1)) break;
            // (the widening warps order their reads before these writes: a proxy fence ahead of their arrival; one here
            // waited for the loads of ids and scales in flight, ~700 cycles of every tile)
            copy(tmV, r_dst + (i % T::RS) * T::kKBytes, T::bRFull + i % T::RS);
            r_issued = i + 1;
            if (i + 1 < nt_all) pages = write_info(i + 1, blk1, ks1, vs1);  // that tile's keys arrive after this
            blk = blk1;
            blk1 = blk2;
            blk2 = blk3;
            ks1 = ks2;
            vs1 = vs2;
        }
        // copies in flight must land before the CTA exits, also when another warp gives up later: the last
        // issue of each stage (long done in a run that consumed them)
        auto drain = [&](int bar, int n, int stages) {
            for (int t = max(0, n - stages); t < n; ++t) {
                const long long t0 = clock64();
                while (!umma::mbar_try_wait(&mbar[bar + t % stages], (t / stages) & 1) && clock64() - t0 < kDrainLimit) {
                }
            }
        };
        drain(T::bKFull, k_issued, T::KS);
        drain(T::bRFull, r_issued, T::RS);
    }

    // ---- teardown ----
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    if (*abort_flag && tid < 128 * NQ && tid < ncol) dead_row(tid);  // a wait gave up: nothing of this CTA counts
    if (warp == T::kMmaWarp) umma::tmem_dealloc(tbase, T::kTmCols);
}

template <int D>
cudaError_t launch(const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, cudaStream_t st)
{
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(prefill_fp8_kernel<D>), Tc<D>::kSmem);
    if (e != cudaSuccess) return e;
    const unsigned units = static_cast<unsigned>(a.B) * a.Hkv * a.nqt, grid = a.whole + (units - a.whole) * a.splits;
    prefill_fp8_kernel<D><<<grid, Tc<D>::kThreads, Tc<D>::kSmem, st>>>(tk, tv, a);
    return cudaGetLastError();
}

}  // namespace

int prefill_tc_columns(int d) { return d == 128 ? 128 * Tc<128>::NQ : 128 * Tc<256>::NQ; }

cudaError_t launch_prefill_tc(const CUtensorMap &tk, const CUtensorMap &tv, int d, const Args &a, cudaStream_t st)
{
    return d == 128 ? launch<128>(tk, tv, a, st) : launch<256>(tk, tv, a, st);
}

}  // namespace fp8
}  // namespace tq
