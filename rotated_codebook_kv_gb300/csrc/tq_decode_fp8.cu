// tq_decode_fp8.cu -- attention over 8-bit pages: e4m3 codes with one scale per
// (page, kv head) for keys and for values.
//
// The pages of a 32-token round come by the tensor memory accelerator (boxes of one page x 128 bytes, 128-byte
// swizzle) into a warp's own stages.  Codes enter the products as they are stored (mma.m16n8k32, e4m3 in, fp32
// sums), nothing is widened first:
//   S[t][h] = <kc_t, q_h 2^e>, tokens as M, heads as N; q 2^e as two e4m3 terms, which is
//             exact: a bf16 has 8 significant bits, an e4m3 4 and a sign for the rest;
//   O[j][h] += sum_t vc_t[j] P[t][h], coordinates as M (bytes of two tokens side by side
//             from ldmatrix.trans, four by one byte permutation), tokens as K.
// The value scale enters through the exponent: with x = sm_scale log2(e) ks[page] 2^-e S
// and y = x + log2 vs[page], P = 2^(y - max y + 8) (max: of the round) carries exp(x) vs, so that pages of
// any scales share one accumulator, and the denominator adds P / vs.  P enters as
// two e4m3 terms (about 8 bits: 4 and their rest), the rest is fp32.  fp16 P would need
// the value codes widened and mma at a quarter of the rate (0.5 against 1.9 instructions per cycle and SM, measured).
// P is taken against the maximum of its own round of 32 tokens, and the round's product added to O with the factor
// between that and the running maximum: both terms end at 2^-18 of what they are taken against, and against the running
// maximum the weak tail behind one strong token would lie below that (8 % of the output gone at 13 nats and 32k tokens).
// 32 multiply-adds a round at head dim 128; the times stayed (174.5 us long, 179 at head dim 256).  Only for rounds far
// below the running maximum, by a second copy of the product's code: 177 and 186.  Value scales 2^220 apart (squares of
// roots, see below) took them to 176 and 181, a branch for the rounds that need it 177 and 183.
//
// Work is dealt out on the GPU, where the lengths are: the rounds of all (sequence, kv head) units in a row, an
// equal share for each of one wave of CTAs (three of four warps per SM at head dim 128, one of seven at 256).  A CTA's
// share is cut at unit ends into segments; the warps of a CTA take a segment's rounds in turn and merge.  A unit that one
// CTA has whole is written at once, the others' partials (max, denominator, numerators) are merged by merge_fp8_kernel.
// With one split a CTA has one whole unit.  Up to eight (query token, head) columns of a sequence and kv head go through
// this kernel, more through tq_prefill_fp8.cu.
//
// Bound: HBM.  Measured on a GB300 (copy 6783 GB/s): 4 sequences of 131,072 tokens, 8 kv heads, head dim 128: 1.08 GB
// in 176 us = 6.1 TB/s; head dim 256: 181 us, 5.9 TB/s.  A short call takes 10-11 us: checks, tensor maps, launch (9.1 by
// graph replay, two CTAs for 512 tokens of two kv heads).
// Warps of a CTA x CTAs per SM x stages, when chosen, at head dim 128: 4 x 3 x 2 175 us, 3 x 3 x 3 231, 4 x 2 x 3 193,
// 7 x 1 x 4 213, 7 x 2 x 2 255; at 256: 7 x 1 x 2 179, 4 x 1 x 3 223.
#include <climits>
#include <cmath>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tq.h"
#include "tq_fp8.cuh"

namespace tq {
namespace {

using namespace fp8;

constexpr int kTok = 32;                  // tokens of a warp's round
constexpr int kBoxBytes = kTok * 128;     // one 128-byte-wide column block of a round
constexpr int kUnitCost = 8;               // what a unit costs beside its rounds, in rounds (queries, first copies, merge)
constexpr float kPShift = 8.f;            // probabilities enter the product as 2^8 p <= 256

template <int D>
struct Fp8Smem {
    static constexpr int kWarps = D == 128 ? 4 : 7;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kCtas = D == 128 ? 3 : 1;
    static constexpr int kStages = 2;
    static constexpr int kTileBytes = kTok * D;       // keys or values of one round
    static constexpr int kStage = 2 * kTileBytes;     // keys, then values
    static constexpr size_t kData = static_cast<size_t>(kWarps) * kStages * kStage;
    static constexpr size_t kBytes = 1024 + kData + 128 + 4 * D;  // alignment slack, stages, barriers and flag, NaN tokens
    static_assert(kBytes <= 232448, "shared memory");
    static_assert(kData >= sizeof(float) * kWarps * (D * 8 + 16), "merge area");
};

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                 "{%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t &a0, uint32_t &a1, uint32_t &a2, uint32_t &a3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3) : "r"(addr) : "memory");
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t &a0, uint32_t &a1, uint32_t &a2, uint32_t &a3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3) : "r"(addr) : "memory");
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ bool mbar_test(uint32_t mb, uint32_t par)
{
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done) : "r"(mb), "r"(par) : "memory");
    return done != 0;
}

__device__ __forceinline__ bool mbar_try(uint32_t mb, uint32_t par)
{
    uint32_t done;
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done) : "r"(mb), "r"(par) : "memory");
    return done != 0;
}

// Size of a unit of L tokens when work is dealt out: its rounds and what it costs beside them.
__device__ __forceinline__ int unit_size(int L) { return L > 0 ? (L + kTok - 1) / kTok + kUnitCost : 0; }

// The sequences' sizes, summed, and the longest one's, by the whole block.
template <int THREADS>
__device__ __forceinline__ void count_rounds(const Args &A, long long *s_sum, int *s_max, long long &total, int &longest)
{
    long long sum = 0;
    int mx = 0;
    for (int b = threadIdx.x; b < A.B; b += THREADS) {
        const int L = A.seq_lens[b];
        if (L > A.max_blocks * A.P && blockIdx.x == 0) atomicOr(A.status, TQ_DEVERR_SEQ_RANGE);
        const int r = unit_size(min(max(L, 0), A.max_blocks * A.P));
        sum += r;
        mx = max(mx, r);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if ((threadIdx.x & 31) == 0) {
        s_sum[threadIdx.x >> 5] = sum;
        s_max[threadIdx.x >> 5] = mx;
    }
    __syncthreads();
    total = 0;
    longest = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        total += s_sum[w];
        longest = max(longest, s_max[w]);
    }
    __syncthreads();
}

// The columns of a CTA are the (query token, head) pairs of a sequence and kv head, eight at most, each with its causal
// limit (one query token: the G heads, which see all; MANY: several, which is a kernel of its own because what it does for
// values that only some see cost the decode 2-4 % at head dim 128).
template <int D, bool MANY>
__global__ void __launch_bounds__(Fp8Smem<D>::kThreads, Fp8Smem<D>::kCtas)
    attention_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Args A)
{
    using SM = Fp8Smem<D>;
    constexpr int kWarps = SM::kWarps, kThreads = SM::kThreads, kStages = SM::kStages;
    constexpr int KS = D / 32;   // k-steps of the score product
    constexpr int MT = D / 16;   // m-tiles of the value product
    constexpr int XB = D / 128;  // 128-byte column blocks of a row
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *mbar = reinterpret_cast<uint64_t *>(smem + SM::kData);  // [warp][stage]
    volatile int *cta_abort = reinterpret_cast<volatile int *>(mbar + kStages * kWarps);
    int *nan_at = reinterpret_cast<int *>(smem + SM::kData + 128);  // [D] first token behind the causal limits with a NaN value
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int quad = lane & 3, row = lane >> 2;
    const int P = A.P, G = A.G, ncol = A.Tq * G;
    const size_t rows_total = static_cast<size_t>(A.B) * A.Tq * A.Hq;

    if (tid < kStages * kWarps)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(&mbar[tid]))));
    if (tid == 0) *cta_abort = 0;
    if (MANY)
        for (int j = tid; j < D; j += kThreads) nan_at[j] = INT_MAX;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();

    // ---- this CTA's share: [pos, end) of all units' sizes in a row, and the unit that it begins in ----
    long long pos, end, share, unit0;  // unit0: where the unit at hand begins
    int b, kvh;
    auto length = [&](int i) -> int { return min(max(A.seq_lens[i], 0), A.max_blocks * P); };
    if (A.splits == 1) {
        b = blockIdx.x / A.Hkv;
        kvh = blockIdx.x % A.Hkv;
        if (kvh == 0 && tid == 0 && A.seq_lens[b] > A.max_blocks * P) atomicOr(A.status, TQ_DEVERR_SEQ_RANGE);
        pos = unit0 = 0;
        end = share = max(1, unit_size(length(b)));
    } else {
        long long *s_sum = reinterpret_cast<long long *>(smem);
        int *s_max = reinterpret_cast<int *>(smem + 128);
        long long total;
        int longest;
        count_rounds<kThreads>(A, s_sum, s_max, total, longest);
        total *= A.Hkv;
        // at least two rounds a warp, and no unit in more pieces than there are splits
        share = (total + gridDim.x - 1) / gridDim.x;
        share = max(share, static_cast<long long>(2 * kWarps + kUnitCost));
        share = max(share, static_cast<long long>((longest + A.splits - 2) / (A.splits - 1)));
        pos = share * blockIdx.x;
        end = min(total, pos + share);
        if (pos >= end) return;
        // the sequence that holds round pos: running sums over blockDim sequences at a time
        long long before = 0;  // rounds of the sequences before this stretch, all kv heads
        int *s_b = reinterpret_cast<int *>(smem + 192);
        long long *s_u = reinterpret_cast<long long *>(smem + 200);
        b = 0;
        for (int b0 = 0;; b0 += kThreads) {
            const long long r = b0 + tid < A.B ? static_cast<long long>(unit_size(length(b0 + tid))) * A.Hkv : 0;
            long long inc = r;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) s_sum[warp] = inc;
            __syncthreads();
            long long base = before, all = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (w < warp) base += s_sum[w];
                all += s_sum[w];
            }
            const bool here = pos >= base + inc - r && pos < base + inc;
            if (here) {
                *s_b = b0 + tid;
                *s_u = base + inc - r;
            }
            before += all;
            if (__syncthreads_or(here) || b0 + kThreads >= A.B) break;
        }
        b = *s_b;
        unit0 = *s_u;
        const int per = unit_size(length(b));
        kvh = static_cast<int>((pos - unit0) / per);
        unit0 += static_cast<long long>(kvh) * per;
        __syncthreads();  // the stages may be written
    }

    const uint32_t sbase = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    auto stage_addr = [&](int st) -> uint32_t { return sbase + static_cast<uint32_t>((warp * kStages + st) * SM::kStage); };
    auto mbar_addr = [&](int st) -> uint32_t {
        return static_cast<uint32_t>(__cvta_generic_to_shared(&mbar[warp * kStages + st]));
    };
    auto drain = [&](int st, uint32_t par) {
        const long long t0 = clock64();
        while (!mbar_try(mbar_addr(st), par) && clock64() - t0 < kDrainLimit) {
        }
    };
    // this lane's ldmatrix offsets; a k-step or coordinate chunk flips address bits 4-6
    const int mi = lane >> 3, ri = lane & 7;
    const int krow = ri + 8 * (mi & 1);  // keys: matrices (rows 0-7 | 8-15) x (chunk c | c + 1)
    const uint32_t koff = krow * 128 + (((mi >> 1) ^ ri) << 4), voff = SM::kTileBytes + lane * 128 + (ri << 4);
    const int half = lane & 1;  // a round's scales and ids: even lanes hold its first 16 tokens', odd ones its last

    int done = 0;  // rounds that this warp has computed since the start: stage done % kStages
    for (;;) {
        const int L = length(b);
        const int size = max(1, unit_size(L));
        // a unit's rounds stand behind its cost: a share may end within that and hold none of them
        const int r0 = max(0, static_cast<int>(pos - unit0) - kUnitCost);
        const int r1 = max(0, static_cast<int>(min(end, unit0 + size) - unit0) - kUnitCost);
        auto col_row = [&](int c) -> size_t {  // output row of column c
            return (static_cast<size_t>(b) * A.Tq + c / G) * A.Hq + static_cast<size_t>(kvh) * G + c % G;
        };
        auto col_lim = [&](int c) -> int { return max(0, L - A.Tq + c / G + 1); };  // positions that it sees
        const int tok1 = min(L, r1 * kTok);
        const int32_t *table = A.block_table + static_cast<int64_t>(b) * A.max_blocks;
        auto round_tok = [&](int c) -> int { return (r0 + warp + kWarps * c) * kTok; };
        auto fetch_id = [&](int c) -> int {  // block of this lane's half of a round, -1 past the end
            const int t = round_tok(c) + 16 * half;
            return t < tok1 ? __ldg(table + (t >> A.pshift)) : -1;
        };
        auto good = [&](int blk) -> bool { return blk >= 0 && blk < A.num_blocks; };
        auto record = [&](int blk) -> int { return blk * A.Hkv + kvh; };  // below 2^31 / P
        auto issue = [&](int c, int st, int blk) {  // the round's pages into a stage
            const bool page = lane < 2 && (P == 16 || lane == 0);
            const unsigned ok = __ballot_sync(0xffffffffu, page && good(blk));
            const uint32_t mb = mbar_addr(st);
            if (page && !good(blk) && round_tok(c) + 16 * half < tok1) atomicOr(A.status, TQ_DEVERR_BLOCK_RANGE);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // this warp's accesses of the stage are done
            if (lane == 0)
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mb),
                             "r"(__popc(ok) * static_cast<uint32_t>(2 * P * D))
                             : "memory");
            __syncwarp();
            if (ok >> lane & 1u) {
                const int y = record(blk) * P;
                const uint32_t dk = stage_addr(st) + lane * 16 * 128;
#pragma unroll
                for (int x = 0; x < XB; ++x) {
                    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                                 ::"r"(dk + x * kBoxBytes), "l"(reinterpret_cast<uint64_t>(&tmK)), "r"(x * 128), "r"(y), "r"(mb)
                                 : "memory");
                    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                                 ::"r"(dk + SM::kTileBytes + x * kBoxBytes), "l"(reinterpret_cast<uint64_t>(&tmV)), "r"(x * 128),
                                 "r"(y), "r"(mb)
                                 : "memory");
                }
            }
        };

        const int my_rounds = r1 - r0 > warp ? (r1 - r0 - warp + kWarps - 1) / kWarps : 0;  // rounds r0 + warp, + kWarps, ...
        // blocks of this and the next kStages rounds; kStages - 1 rounds are on their way while one is computed
        int id[kStages + 1];
#pragma unroll
        for (int n = 0; n <= kStages; ++n) id[n] = n < my_rounds ? fetch_id(n) : -1;
#pragma unroll
        for (int n = 0; n < kStages - 1; ++n)
            if (n < my_rounds) issue(n, (done + n) % kStages, id[n]);
        // a zero limit tests the first copy at once, while it cannot be done: the way to the timeout path
        const bool first_ok = A.wait_limit > 0 || my_rounds == 0 || mbar_test(mbar_addr(done % kStages), (done / kStages) & 1);

        // query fragments (B operand of the score product): column `row`, coordinates 32 s + 4 quad (+ 16)
        uint32_t qh[KS][2], ql[KS][2];
        float qfac;  // 2^-e of column `row`
        {
            const bool cv = row < ncol;
            const uint2 *qr = reinterpret_cast<const uint2 *>(A.q + col_row(cv ? row : 0) * D);
            uint2 w[KS][2];
            float mx = 0.f;
            bool nan = false;
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) w[s][i] = cv ? __ldg(qr + 8 * s + 4 * i + quad) : make_uint2(0u, 0u);
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t u[2] = {w[s][i].x, w[s][i].y};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float x0 = fabsf(__uint_as_float(u[k] << 16)), x1 = fabsf(__uint_as_float(u[k] & 0xffff0000u));
                        nan |= !(x0 <= 3.4e38f) || !(x1 <= 3.4e38f);
                        mx = fmaxf(mx, fmaxf(x0, x1));
                    }
                }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            nan = (__ballot_sync(0xffffffffu, nan) >> (lane & ~3)) & 15u;
            // 2^e brings the largest element into [2^7, 2^8)
            int ex = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
            ex = min(max(ex, -100), 127);
            const float up = __uint_as_float(static_cast<uint32_t>(7 - ex + 127) << 23);
            qfac = nan ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(ex - 7 + 127) << 23);
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float x0 = __uint_as_float(w[s][i].x << 16) * up, x1 = __uint_as_float(w[s][i].x & 0xffff0000u) * up;
                    float x2 = __uint_as_float(w[s][i].y << 16) * up, x3 = __uint_as_float(w[s][i].y & 0xffff0000u) * up;
                    const uint32_t lo = e4m3x2_rest(x0, x1), hi = e4m3x2_rest(x2, x3);
                    qh[s][i] = lo | (hi << 16);
                    ql[s][i] = e4m3x2(x0, x1) | (e4m3x2(x2, x3) << 16);
                }
        }
        float fac[2];  // columns 2 quad + e: sm_scale log2(e) 2^-e
        int lim[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int c = 2 * quad + e;
            fac[e] = __shfl_sync(0xffffffffu, qfac, 4 * c) * A.sm_scale * kLog2e;
            lim[e] = min(tok1, c < ncol ? col_lim(c) : tok1);
        }
        const int low = min(tok1, col_lim(0));  // every column sees the positions below

        float o[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        float m_run[2] = {-INFINITY, -INFINITY};  // columns 2 quad + e
        float l_run[2] = {0.f, 0.f};              // this lane's tokens' share of the denominators

        auto scale_of = [&](const float *p, int blk) -> float { return good(blk) ? __ldg(p + record(blk)) : 0.f; };
        float ks = scale_of(A.k_scales, id[0]), vs = scale_of(A.v_scales, id[0]);  // of this lane's half of the round
        for (int c = 0; c < my_rounds; ++c, ++done) {
            const int st = done % kStages;
            __syncwarp();  // every lane is done with the stage the next copy overwrites
            if (c + kStages - 1 < my_rounds) issue(c + kStages - 1, (done + kStages - 1) % kStages, id[kStages - 1]);
            const float ks1 = scale_of(A.k_scales, id[1]), vs1 = scale_of(A.v_scales, id[1]);
            const int id_new = c + kStages + 1 < my_rounds ? fetch_id(c + kStages + 1) : -1;
            // One page's values more than 2^90 below the other's count as 2^90 below, so that P / vs of either half stays in fp32's
            // range (squares for every P: 178.6 us against 176).  Among several query tokens, some of which may not see the other
            // page, squares it is.
            float lvl = log2_scale(vs);
            if (!MANY) lvl = fmaxf(lvl, __shfl_xor_sync(0xffffffffu, lvl, 1) - 90.f);
            const float downl = fast_exp2(kLShift - kPShift - lvl);
            const int t = round_tok(c);
            const unsigned okm = __ballot_sync(0xffffffffu, good(id[0]));
            {
                const uint32_t par = (done / kStages) & 1;
                bool ok = true;
                if (A.wait_limit <= 0) {
                    ok = c == 0 ? first_ok : mbar_test(mbar_addr(st), par);
                } else if (!mbar_try(mbar_addr(st), par)) {
                    const long long t0 = clock64();
                    while (!(ok = mbar_try(mbar_addr(st), par)))
                        if (clock64() - t0 > A.wait_limit) break;
                }
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    if (lane == 0) {
                        atomicOr(A.status, TQ_DEVERR_TIMEOUT);
                        *cta_abort = 1;
                    }
                    for (int n = 0; n < kStages && c + n < my_rounds; ++n) drain((done + n) % kStages, ((done + n) / kStages) & 1);
                    break;
                }
            }
            const uint32_t stage = stage_addr(st);
            const bool whole = (okm & 3u) == 3u && t + kTok <= low;  // every token is seen by every column
            int nv[2];                                               // tokens of each half
#pragma unroll
            for (int h = 0; h < 2; ++h) nv[h] = (okm >> h & 1u) ? max(0, min(16, tok1 - t - 16 * h)) : 0;
            if (!whole && (nv[0] + nv[1] < kTok || MANY)) {
                // rows behind the end or of a bad page hold anything: zero the values; among query tokens, NaN that some do not see
                unsigned char *vz = smem + (stage - sbase) + SM::kTileBytes;
                for (int e = lane; e < kTok * (D / 16); e += 32) {
                    const int rr = e / (D / 16), cc = e % (D / 16);
                    uint4 *at = reinterpret_cast<uint4 *>(vz + (cc / 8) * kBoxBytes + rr * 128 + (cc % 8) * 16);
                    if ((rr & 15) >= nv[rr >> 4]) {
                        *at = make_uint4(0u, 0u, 0u, 0u);
                    } else if (MANY && t + rr >= low) {
                        uint4 w = *at;
                        hide_nan(w, nan_at + (cc / 8) * 128 + ((cc ^ rr) & 7) * 16, t + rr);
                        *at = w;
                    }
                }
                __syncwarp();
            }
            // ---- scores ----
            float sc[2][4] = {};
            const uint32_t kat = stage + koff;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a0, a1, a2, a3;
                    ldsm_x4((kat ^ (32 * (s & 3))) + (s >> 2) * kBoxBytes + h * 16 * 128, a0, a1, a2, a3);
                    mma_e4m3(sc[h], a0, a1, a2, a3, qh[s][0], qh[s][1]);
                    mma_e4m3(sc[h], a0, a1, a2, a3, ql[s][0], ql[s][1]);
                }
            }
            // ---- mask, online softmax (base 2): this lane holds tokens row, row + 8 of each half, columns 2 quad + e ----
            float y[2][2][2], down[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float k1 = __shfl_sync(0xffffffffu, ks, h), lv = __shfl_sync(0xffffffffu, lvl, h);
                down[h] = __shfl_sync(0xffffffffu, downl, h);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float a = fac[e] * k1;
#pragma unroll
                    for (int r = 0; r < 2; ++r) y[h][r][e] = fmaf(sc[h][2 * r + e], a, lv);
                }
            }
            if (!whole) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int i = row + 8 * r;
                            if (i >= nv[h] || t + 16 * h + i >= lim[e]) y[h][r][e] = -INFINITY;
                        }
            }
            // A page of small values may lie 2^220 below another by its scale (an empty one's is 2^-100): the factors between rounds
            // are squares of these roots, which the denominator is multiplied by twice.
            float alpha[2], shift[2], fall[2], alpha_root[2], fall_root[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float top = max3(y[0][0][e], y[0][1][e], fmaxf(y[1][0][e], y[1][1][e]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                const float m = fmaxf(top, m_run[e]);
                alpha_root[e] = m == m_run[e] ? 1.f : fast_exp2(0.5f * (m_run[e] - m));
                const bool none = top == -INFINITY;  // nothing of the round is seen (or only NaN)
                fall_root[e] = none ? 1.f : fast_exp2(0.5f * (top - m));
                shift[e] = none ? kPShift : kPShift - top;
                alpha[e] = alpha_root[e] * alpha_root[e];
                fall[e] = fall_root[e] * fall_root[e];
                m_run[e] = m;
            }
            if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    o[mt][0] *= alpha[0]; o[mt][1] *= alpha[1]; o[mt][2] *= alpha[0]; o[mt][3] *= alpha[1];
                }
            }
            // ---- P as the B operand: byte pairs (high, low) of a token and column, transposed
            // to (column `row`; tokens 2 quad, 2 quad + 1 | + 8, + 9), then high and low bytes apart ----
            uint32_t bh[2], bl[2];
            float l_round[2] = {0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t tr[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float p0 = y[h][r][0] + shift[0], p1 = y[h][r][1] + shift[1];
                    if (MANY) {
                        const float r0 = fast_exp2(0.5f * p0), r1 = fast_exp2(0.5f * p1);
                        l_round[0] = fmaf(r0, r0 * down[h], l_round[0]);
                        l_round[1] = fmaf(r1, r1 * down[h], l_round[1]);
                        p0 = r0 * r0;
                        p1 = r1 * r1;
                    } else {
                        p0 = fast_exp2(p0);
                        p1 = fast_exp2(p1);
                        l_round[0] = fmaf(p0, down[h], l_round[0]);
                        l_round[1] = fmaf(p1, down[h], l_round[1]);
                    }
                    __half2 p = __floats2half2_rn(p0, p1);  // 11 bits, of which the two terms keep about 8
                    const uint32_t hi = e4m3x2_rest(p);
                    tr[r] = movmatrix_trans(__byte_perm(hi, e4m3x2(p), 0x5140));
                }
                bh[h] = __byte_perm(tr[0], tr[1], 0x6420);
                bl[h] = __byte_perm(tr[0], tr[1], 0x7531);
            }
            // ---- O[coordinate][column] += V^T P: the m-tile's rows are its even coordinates, then its odd ones ----
            const uint32_t vat = stage + voff;
            auto value_tile = [&](int mt, float (&c)[4]) {
                uint32_t v0, v1, v2, v3;
                ldsm_x4_trans((vat ^ ((mt & 7) << 4)) + (mt >> 3) * kBoxBytes, v0, v1, v2, v3);
                const uint32_t a0 = __byte_perm(v0, v1, 0x6420), a1 = __byte_perm(v0, v1, 0x7531);
                const uint32_t a2 = __byte_perm(v2, v3, 0x6420), a3 = __byte_perm(v2, v3, 0x7531);
                mma_e4m3(c, a0, a1, a2, a3, bh[0], bh[1]);
                mma_e4m3(c, a0, a1, a2, a3, bl[0], bl[1]);
            };
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float c4[4] = {0.f, 0.f, 0.f, 0.f};
                value_tile(mt, c4);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][i] = fmaf(fall[i & 1], c4[i], o[mt][i]);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                l_run[e] = fmaf(fall_root[e], fall_root[e] * l_round[e], alpha_root[e] * (alpha_root[e] * l_run[e]));
            ks = ks1;
            vs = vs1;
#pragma unroll
            for (int n = 0; n < kStages; ++n) id[n] = id[n + 1];
            id[kStages] = id_new;
        }
        __syncthreads();  // every warp is done with the stages before they hold merge data
        const bool dead = *cta_abort != 0;
        float *red = reinterpret_cast<float *>(smem);
        float *r_m = red;                   // [warps][8]
        float *r_l = r_m + kWarps * 8;      // [warps][8]
        float *r_o = r_l + kWarps * 8;      // [warps][D][8]
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 4);
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 8);
            l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 16);
        }
        if (row == 0) {
            r_m[warp * 8 + 2 * quad] = m_run[0];
            r_m[warp * 8 + 2 * quad + 1] = m_run[1];
            r_l[warp * 8 + 2 * quad] = l_run[0];
            r_l[warp * 8 + 2 * quad + 1] = l_run[1];
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float *p = r_o + (warp * D + 16 * mt + 2 * row) * 8 + 2 * quad;
            *reinterpret_cast<float2 *>(p) = make_float2(o[mt][0], o[mt][1]);
            *reinterpret_cast<float2 *>(p + 8) = make_float2(o[mt][2], o[mt][3]);
        }
        __syncthreads();
        // a unit's pieces are numbered from the CTA that holds its first round; a unit in one piece is done here
        const long long first = unit0 / share;
        const int pieces = A.splits == 1 ? 1 : static_cast<int>((unit0 + size - 1) / share - first) + 1;
        const int piece = A.splits == 1 ? 0 : static_cast<int>(blockIdx.x - first);
        if (piece == 0 && tid == 0 && A.splits > 1) A.pieces[static_cast<int64_t>(b) * A.Hkv + kvh] = pieces;
        const float downp = fast_exp2(-kPShift), ldown = fast_exp2(-kLShift);
        for (int e = tid; e < ncol * D; e += kThreads) {
            const int c = e / D, j = e - c * D;
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, r_m[w * 8 + c]);
            const float ref = M == -INFINITY ? 0.f : M;
            float acc = 0.f, l = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                if (r_l[w * 8 + c] == 0.f) continue;  // a warp that saw nothing
                const float f = r_m[w * 8 + c] == -INFINITY ? 1.f : fast_exp2(0.5f * (r_m[w * 8 + c] - ref));
                acc = fmaf(f * f, r_o[(w * D + j) * 8 + c], acc);
                l = fmaf(f, f * r_l[w * 8 + c], l);
            }
            acc *= downp;
            l *= ldown;
            if (MANY && nan_at[j] < col_lim(c)) acc = __int_as_float(0x7fffffff);
            if (dead) {
                M = -INFINITY;
                acc = l = 0.f;
            }
            const size_t orow = col_row(c);
            if (pieces == 1) {
                A.out[orow * D + j] = float_to_bf16_bits(l == 0.f ? 0.f : acc / l);
            } else {
                const size_t pr = static_cast<size_t>(piece) * rows_total + orow;
                A.acc[pr * D + j] = acc;
                if (j == 0) {
                    A.ml[2 * pr] = M;
                    A.ml[2 * pr + 1] = l;
                }
            }
        }
        // ---- the next unit of the share ----
        pos = unit0 + size;
        unit0 = pos;
        if (pos >= end) return;
        if (++kvh == A.Hkv) {
            kvh = 0;
            do ++b;
            while (length(b) == 0);  // pos < end: there is a later unit with rounds
        }
        __syncthreads();  // the merge data is read
        if (MANY) {
            for (int j = tid; j < D; j += kThreads) nan_at[j] = INT_MAX;
            __syncthreads();
        }
        // the waits of a CTA that gave up are not in step with its stages any more: its other units count as unseen
        if (dead) {
            for (;;) {
                const int n = unit_size(length(b));
                const long long f0 = unit0 / share;
                const int np = static_cast<int>((unit0 + n - 1) / share - f0) + 1;
                if (blockIdx.x == f0 && tid == 0) A.pieces[static_cast<int64_t>(b) * A.Hkv + kvh] = np;
                for (int e = tid; e < ncol * D; e += kThreads) {
                    const size_t orow = (static_cast<size_t>(b) * A.Tq + e / D / G) * A.Hq + static_cast<size_t>(kvh) * G + e / D % G;
                    if (np == 1) A.out[orow * D + e % D] = 0;
                    else if (e % D == 0) {
                        const size_t pr = static_cast<size_t>(blockIdx.x - f0) * rows_total + orow;
                        A.ml[2 * pr] = -INFINITY;
                        A.ml[2 * pr + 1] = 0.f;
                    }
                }
                unit0 += n;
                if (unit0 >= end) return;
                if (++kvh == A.Hkv) {
                    kvh = 0;
                    do ++b;
                    while (length(b) == 0);
                }
            }
        }
    }
}

// Merges the pieces of an output row: o = sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s.
// A block per row: D / 4 threads side by side over the coordinates, 512 / D groups of them over the pieces, so that a
// row's partials are all on their way at once.  A piece that saw nothing (l = 0) has no partial to read.  A NaN of any
// piece stays one.  A unit in one piece is done, an empty sequence gives zeros.
template <int D>
__global__ void __launch_bounds__(128) merge_fp8_kernel(const Args A, const int64_t rows)
{
    constexpr int TC = D / 4, GROUPS = 128 / TC;
    __shared__ float s_w[1024];
    __shared__ float s_part[GROUPS][D];
    __shared__ float s_red[4], s_den;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const int64_t b = row / A.Hq / A.Tq;
    const int splits = A.seq_lens[b] > 0 ? A.pieces[b * A.Hkv + row % A.Hq / A.G] : 0;
    if (splits == 1) return;
    const float2 *ml = reinterpret_cast<const float2 *>(A.ml);
    float M = -INFINITY;
    for (int s = tid; s < splits; s += 128) M = fmaxf(M, __ldg(ml + s * rows + row).x);
    M = warp_max(M);
    if (lane == 0) s_red[warp] = M;
    __syncthreads();
    M = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    const float ref = M == -INFINITY ? 0.f : M;
    __syncthreads();
    float den = 0.f;
    for (int s = tid; s < splits; s += 128) {
        const float2 v = __ldg(ml + s * rows + row);
        const float root = v.x == -INFINITY ? 1.f : fast_exp2(0.5f * (v.x - ref));
        s_w[s] = v.y == 0.f ? -1.f : root * root;  // -1: nothing to read
        den += v.y == 0.f ? 0.f : root * (root * v.y);
    }
    den = warp_sum(den);
    if (lane == 0) s_red[warp] = den;
    __syncthreads();
    if (tid == 0) s_den = (s_red[0] + s_red[1]) + (s_red[2] + s_red[3]);
    const int col = 4 * (tid % TC);
    float4 n = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = tid / TC; s < splits; s += GROUPS) {
        const float w = s_w[s];
        if (w == -1.f) continue;
        const float4 v = __ldg(reinterpret_cast<const float4 *>(A.acc + (s * rows + row) * D + col));
        n.x = fmaf(w, v.x, n.x);
        n.y = fmaf(w, v.y, n.y);
        n.z = fmaf(w, v.z, n.z);
        n.w = fmaf(w, v.w, n.w);
    }
    *reinterpret_cast<float4 *>(&s_part[tid / TC][col]) = n;
    __syncthreads();
    const float inv = s_den == 0.f ? 0.f : 1.f / s_den;
    for (int j = 2 * tid; j < D; j += 256) {
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            x += s_part[g][j];
            y += s_part[g][j + 1];
        }
        reinterpret_cast<uint32_t *>(A.out + row * D)[j / 2] =
            float_to_bf16_bits(x * inv) | (static_cast<uint32_t>(float_to_bf16_bits(y * inv)) << 16);
    }
}

// The same for the prefill's rows, many in few pieces, with denominators in kSumUnit: a warp per row, D / 32 coordinates a
// lane; the rows of the first A.whole units are done.
template <int D>
__global__ void __launch_bounds__(128) merge_rows_fp8_kernel(const Args A, const int64_t rows)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int64_t t = row / A.Hq, b = t / A.Tq;
    const int qt = static_cast<int>(t - b * A.Tq) / A.qpc, kvh = static_cast<int>(row - t * A.Hq) / A.G;
    if ((b * A.Hkv + kvh) * A.nqt + A.nqt - 1 - qt < A.whole) return;
    const float2 *ml = reinterpret_cast<const float2 *>(A.ml);
    float M = -INFINITY;
    for (int s = lane; s < A.splits; s += 32) M = fmaxf(M, __ldg(ml + s * rows + row).x);
    M = warp_max(M);
    const float ref = M == -INFINITY ? 0.f : M;
    float n[E] = {}, den = 0.f;
    for (int s0 = 0; s0 < A.splits; s0 += 32) {
        float root = 0.f, l = 0.f;
        if (s0 + lane < A.splits) {
            const float2 v = __ldg(ml + (s0 + lane) * rows + row);
            l = v.y;
            root = v.y == 0.f ? 0.f : (v.x == -INFINITY ? 1.f : fast_exp2(0.5f * (v.x - ref)));
        }
        const float w = root * root;
        den += warp_sum(l == 0.f ? 0.f : root * (root * l));
        const unsigned some = __ballot_sync(0xffffffffu, l != 0.f);
        const int k1 = min(32, A.splits - s0);
#pragma unroll 4
        for (int k = 0; k < k1; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            if (!(some >> k & 1u)) continue;
            const float *p = A.acc + ((s0 + k) * rows + row) * D + lane * E;
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4 *>(p + i));
                n[i] = fmaf(wk, v.x, n[i]);
                n[i + 1] = fmaf(wk, v.y, n[i + 1]);
                n[i + 2] = fmaf(wk, v.z, n[i + 2]);
                n[i + 3] = fmaf(wk, v.w, n[i + 3]);
            }
        }
    }
    const float inv = den == 0.f ? 0.f : kSumUnit / den;
    uint32_t *dst = reinterpret_cast<uint32_t *>(A.out + row * D + lane * E);
#pragma unroll
    for (int i = 0; i < E; i += 2)
        dst[i / 2] = float_to_bf16_bits(n[i] * inv) | (static_cast<uint32_t>(float_to_bf16_bits(n[i + 1] * inv)) << 16);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// The pieces of a unit: [splits][rows] (max, denominator), [splits][rows][d] numerators, and how many there are.
size_t workspace_bytes(int d, int64_t rows, int splits)
{
    if (splits <= 1) return 0;
    return align256(static_cast<size_t>(splits) * rows * 2 * sizeof(float)) +
           align256(static_cast<size_t>(splits) * rows * d * sizeof(float)) + align256(static_cast<size_t>(rows) * sizeof(int));
}

template <int D>
cudaError_t launch(const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, bool tc, int num_sms, cudaStream_t st)
{
    cudaError_t e;
    if (tc) {
        e = launch_prefill_tc(tk, tv, D, a, st);
    } else {
        const size_t smem = Fp8Smem<D>::kBytes;
        auto *kernel = a.Tq == 1 ? attention_fp8_kernel<D, false> : attention_fp8_kernel<D, true>;
        e = ensure_smem_attr(reinterpret_cast<const void *>(kernel), smem);
        if (e != cudaSuccess) return e;
        const unsigned grid = a.splits == 1 ? static_cast<unsigned>(a.B) * a.Hkv : static_cast<unsigned>(num_sms) * Fp8Smem<D>::kCtas;
        kernel<<<grid, Fp8Smem<D>::kThreads, smem, st>>>(tk, tv, a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || a.splits == 1) return e;
    const int64_t rows = static_cast<int64_t>(a.B) * a.Tq * a.Hq;
    if (tc) merge_rows_fp8_kernel<D><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, st>>>(a, rows);
    else merge_fp8_kernel<D><<<static_cast<unsigned>(rows), 128, 0, st>>>(a, rows);
    return cudaGetLastError();
}

int clamp_splits(long long splits, long long most)
{
    if (splits > most) splits = most;
    if (splits > 64) splits = 64;
    return splits < 1 ? 1 : static_cast<int>(splits);
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// Both entry points: Tq = 1 is the decode.
tq_status attend(const char *who, tq_handle h, const uint16_t *q, const uint8_t *k_pool, const uint8_t *v_pool,
                 const float *k_scales, const float *v_scales, const int32_t *block_table, const int32_t *seq_lens,
                 int batch, int q_tokens, int Hq, int Hkv, int P, int max_blocks, int64_t num_blocks, float sm_scale,
                 int splits, void *workspace, size_t ws_bytes, uint16_t *out, void *stream)
{
    if (!h) return api_error(TQ_ERR_INVALID_ARG, "%s: NULL handle", who);
    const Codec &c = handle_codec(h);
    if (P != 16 && P != 32) return api_error(TQ_ERR_UNSUPPORTED, "%s: page_size %d not in {16, 32}", who, P);
    if (batch < 0 || q_tokens < 1 || Hq < 1 || Hkv < 1 || max_blocks < 1 || num_blocks < 1 || splits < 0)
        return api_error(TQ_ERR_INVALID_ARG, "%s: bad sizes", who);
    if (Hq % Hkv || Hq / Hkv > 8)
        return api_error(TQ_ERR_UNSUPPORTED, "%s: num_q_heads / num_kv_heads must be an integer in 1..8", who);
    if (!std::isfinite(sm_scale)) return api_error(TQ_ERR_INVALID_ARG, "%s: sm_scale not finite", who);
    if (max_blocks > (1 << 30) / P || Hkv > 65535)
        return api_error(TQ_ERR_UNSUPPORTED, "%s: more than 2^30 positions or 65535 kv heads", who);
    if (num_blocks >= (int64_t(1) << 31) / (static_cast<int64_t>(Hkv) * P))
        return api_error(TQ_ERR_UNSUPPORTED, "%s: pool of %lld blocks is too large", who, static_cast<long long>(num_blocks));
    if (batch == 0) return TQ_OK;
    Args a{};
    a.G = Hq / Hkv;
    a.Tq = q_tokens;
    // up to eight (query token, head) columns fit the mma.sync kernel of the decode; more go to the tcgen05 one
    const bool tc = q_tokens * static_cast<int64_t>(a.G) > 8;
    a.qpc = tc ? prefill_tc_columns(c.d) / a.G : q_tokens;
    a.nqt = (q_tokens + a.qpc - 1) / a.qpc;
    const int64_t rows = static_cast<int64_t>(batch) * q_tokens * Hq;
    if ((!tc && batch > 65535) || rows >= (int64_t(1) << 31) ||
        static_cast<int64_t>(batch) * a.nqt * Hkv * (splits ? splits : 256) >= (int64_t(1) << 31))
        return api_error(TQ_ERR_UNSUPPORTED, "%s: too many sequences x query tokens in one call", who);
    if (!q || !k_pool || !v_pool || !k_scales || !v_scales || !block_table || !seq_lens || !out)
        return api_error(TQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(k_scales, 4) ||
        !aligned(v_scales, 4) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256) ||
        !aligned(out, 16))
        return api_error(TQ_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    if (splits == 0)
        splits = q_tokens == 1 ? tq_decode_splits_fp8(h, batch, Hkv, max_blocks, P)
                               : tq_prefill_splits_fp8(h, batch, q_tokens, Hq, Hkv, max_blocks, P);
    if (splits > 1024) return api_error(TQ_ERR_UNSUPPORTED, "%s: splits %d above 1024", who, splits);
    const size_t need = workspace_bytes(c.d, rows, splits);
    if (ws_bytes < need || (need && !workspace))
        return api_error(TQ_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", who, workspace ? ws_bytes : 0, need);
    CUtensorMap tk, tv;
    cudaError_t e = cudaSuccess;
    const int64_t prows = num_blocks * Hkv * P;
    if (!encode_pool_map(&tk, k_pool, false, c.d, prows, 128, P, &e) ||
        !encode_pool_map(&tv, v_pool, false, c.d, prows, 128, P, &e))
        return api_error(TQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled: %s", who, cudaGetErrorString(e));
    a.q = q;
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.B = batch;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.P = P;
    a.pshift = P == 16 ? 4 : 5;
    a.max_blocks = max_blocks;
    a.num_blocks = num_blocks;
    a.sm_scale = sm_scale;
    a.splits = splits;
    a.pages_per_split = (max_blocks + splits - 1) / splits;
    const int64_t units = static_cast<int64_t>(batch) * Hkv * a.nqt;
    a.whole = tc && splits > 1 ? static_cast<int>(units / c.num_sms * c.num_sms) : 0;
    a.ml = static_cast<float *>(workspace);
    a.acc = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                      align256(static_cast<size_t>(splits) * rows * 2 * sizeof(float)));
    a.pieces = reinterpret_cast<int *>(reinterpret_cast<char *>(a.acc) +
                                       align256(static_cast<size_t>(splits) * rows * c.d * sizeof(float)));
    a.out = out;
    a.status = c.status;
    a.wait_limit = c.wait_limit;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = c.d == 128 ? launch<128>(tk, tv, a, tc, c.num_sms, st) : launch<256>(tk, tv, a, tc, c.num_sms, st);
    if (e != cudaSuccess) return api_error(TQ_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return TQ_OK;
}

}  // namespace
}  // namespace tq

extern "C" int tq_decode_splits_fp8(tq_handle h, int batch, int num_kv_heads, int max_blocks_per_seq, int page_size)
{
    if (!h || batch < 1 || num_kv_heads < 1 || max_blocks_per_seq < 1 || page_size < 1) return 1;
    // Up to 1024 positions a CTA per (sequence, kv head) and no merge.  Else one wave of CTAs shares the rounds, and a
    // unit of four times the mean length may still be cut at every CTA's share.
    if (static_cast<long long>(max_blocks_per_seq) * page_size <= 1024) return 1;
    const long long units = static_cast<long long>(batch) * num_kv_heads;
    const tq::Codec &c = tq::handle_codec(h);
    const long long ctas = static_cast<long long>(c.num_sms) * (c.d == 128 ? tq::Fp8Smem<128>::kCtas : tq::Fp8Smem<256>::kCtas);
    const long long tiles = (static_cast<long long>(max_blocks_per_seq) * page_size + 127) / 128;
    const int splits = tq::clamp_splits((4 * ctas + units - 1) / units + 1, tiles);
    return splits < 2 ? 2 : splits;
}

extern "C" size_t tq_workspace_bytes_fp8(tq_handle h, int batch, int num_q_heads, int splits)
{
    if (!h || batch < 0 || num_q_heads < 0 || splits < 1) return 0;
    return tq::workspace_bytes(tq::handle_codec(h).d, static_cast<int64_t>(batch) * num_q_heads, splits);
}

extern "C" tq_status tq_decode_attention_fp8(tq_handle h, const uint16_t *q, const uint8_t *k_pool,
                                             const uint8_t *v_pool, const float *k_scales, const float *v_scales,
                                             const int32_t *block_table, const int32_t *seq_lens, int batch,
                                             int num_q_heads, int num_kv_heads, int page_size, int max_blocks_per_seq,
                                             int64_t num_blocks, float sm_scale, int splits, void *workspace,
                                             size_t ws_bytes, uint16_t *out, void *stream)
{
    return tq::attend("tq_decode_attention_fp8", h, q, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens, batch,
                      1, num_q_heads, num_kv_heads, page_size, max_blocks_per_seq, num_blocks, sm_scale, splits,
                      workspace, ws_bytes, out, stream);
}

extern "C" int tq_prefill_splits_fp8(tq_handle h, int batch, int q_tokens, int num_q_heads, int num_kv_heads,
                                     int max_blocks_per_seq, int page_size)
{
    if (!h || batch < 1 || q_tokens < 1 || num_kv_heads < 1 || num_q_heads < num_kv_heads || max_blocks_per_seq < 1 ||
        page_size < 1)
        return 1;
    const int G = num_q_heads / num_kv_heads;
    if (static_cast<long long>(q_tokens) * G <= 8)  // the decode's kernel
        return tq_decode_splits_fp8(h, batch, num_kv_heads, max_blocks_per_seq, page_size);
    const int qpc = tq::fp8::prefill_tc_columns(tq::handle_codec(h).d) / G;
    const long long units = static_cast<long long>(batch) * num_kv_heads * ((q_tokens + qpc - 1) / qpc);
    // One CTA per SM.  Whole waves of units stay whole; the rest is cut into the pieces (of 512 tokens at least) that take
    // the least time, in steps of 64 tokens (about a microsecond) of a sequence that fills its table, as all are taken to:
    // waves of pieces, each with a start and an end, the merge's launch, and 45 pieces' sums written and read a step.  When
    // chosen (batches of equal length but the last, tables no wider than the longest sequence), in one | two | three |
    // four | five pieces, us: 128 units of 128 steps at head dim 256 136 | 159 | 170 | 178 | 189, 256 units 212 | 232 | 230
    // | 227 | 219, 64 units 134 | 86 | 102 | 96 | 86; at 128, 512 units of 256 steps 869 | 840 | 834 | 819 | 816, 128 units
    // 259 | 281 | 294 | 297 | 310, 256 units of up to 128 steps 204 | 204 | 196 | 192 | 194.
    const tq::Codec &c = tq::handle_codec(h);
    const long long sms = c.num_sms, rest = units % sms, tokens = static_cast<long long>(max_blocks_per_seq) * page_size;
    const double steps = static_cast<double>((tokens + 63) / 64), start = c.d == 128 ? 5 : 9, cut_start = c.d == 128 ? 6 : 11;
    if (rest == 0) return 1;
    int best = 1;
    double least = steps + start;
    for (int n = 2; n <= 64 && 512LL * (n - 1) < tokens; ++n) {
        const double t = static_cast<double>((rest * n + sms - 1) / sms) * (steps / n + cut_start) + 3 + rest * n / 45.;
        if (t < least) {
            least = t;
            best = n;
        }
    }
    return best;
}

extern "C" tq_status tq_prefill_attention_fp8(tq_handle h, const uint16_t *q, const uint8_t *k_pool,
                                              const uint8_t *v_pool, const float *k_scales, const float *v_scales,
                                              const int32_t *block_table, const int32_t *seq_lens, int batch,
                                              int q_tokens, int num_q_heads, int num_kv_heads, int page_size,
                                              int max_blocks_per_seq, int64_t num_blocks, float sm_scale, int splits,
                                              void *workspace, size_t ws_bytes, uint16_t *out, void *stream)
{
    return tq::attend("tq_prefill_attention_fp8", h, q, k_pool, v_pool, k_scales, v_scales, block_table, seq_lens,
                      batch, q_tokens, num_q_heads, num_kv_heads, page_size, max_blocks_per_seq, num_blocks, sm_scale,
                      splits, workspace, ws_bytes, out, stream);
}
