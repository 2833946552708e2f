// tq_decode_fp8.cu -- attention over 8-bit pages: e4m3 codes with one scale per
// (page, kv head) for keys and for values.
//
// One CTA = (split, kv head, sequence), W warps (four at head dim 128, three at 256);
// warp w takes the 32-token rounds w, w + W, ... of its split.  The pages of a round come by the tensor memory
// accelerator (boxes of one page x 128 bytes, 128-byte swizzle) into the warp's own
// stages.  Codes enter the products as they are stored (mma.m16n8k32, e4m3 in, fp32
// sums), nothing is widened first:
//   S[t][h] = <kc_t, q_h 2^e>, tokens as M, heads as N; q 2^e as two e4m3 terms, which is
//             exact: a bf16 has 8 significant bits, an e4m3 4 and a sign for the rest;
//   O[j][h] += sum_t vc_t[j] P[t][h], coordinates as M (bytes of two tokens side by side
//             from ldmatrix.trans, four by one byte permutation), tokens as K.
// The value scale enters through the exponent: with x = sm_scale log2(e) ks[page] 2^-e S
// and y = x + log2 vs[page], P = 2^(y - max y + 8) carries exp(x) vs, so that pages of
// any scales share one accumulator, and the denominator adds P / vs.  P enters as
// two e4m3 terms (about 8 bits of the largest), the rest is fp32.
//
// Split partials (max, denominator, numerators) are merged by merge_kernel; with one
// split the CTA writes the output itself.  Up to eight (query token, head) columns of a
// sequence and kv head go through this kernel, more through tq_prefill_fp8.cu.
#include <cmath>
#include <cuda.h>
#include <cuda_runtime.h>

#include "tq.h"
#include "tq_fp8.cuh"

namespace tq {
namespace {

using namespace fp8;

constexpr int kTok = 32;                  // tokens of a warp's round
constexpr int kStages = 2;
constexpr int kBoxBytes = kTok * 128;     // one 128-byte-wide column block of a round
constexpr float kPShift = 8.f;            // probabilities enter the product as 2^8 p <= 256

template <int D>
struct Fp8Smem {
    static constexpr int kWarps = D == 128 ? 4 : 3;   // with two stages each: 64 KB and 96 KB a CTA, three and two CTAs per SM
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kCtas = D == 128 ? 3 : 2;
    static constexpr int kTileBytes = kTok * D;       // keys or values of one round
    static constexpr int kStage = 2 * kTileBytes;     // keys, then values
    static constexpr size_t kData = static_cast<size_t>(kWarps) * kStages * kStage;
    static constexpr size_t kBytes = 1024 + kData + 128;  // alignment slack, stages, barriers and flag
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

// The eight columns of a CTA are (query token, head of the group) pairs: with one query
// token per sequence its G heads, else qpc = 8 / G tokens, each with its causal limit.
template <int D>
__global__ void __launch_bounds__(Fp8Smem<D>::kThreads, Fp8Smem<D>::kCtas)
    attention_fp8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Args A)
{
    using SM = Fp8Smem<D>;
    constexpr int kWarps = SM::kWarps, kThreads = SM::kThreads;
    constexpr int KS = D / 32;   // k-steps of the score product
    constexpr int MT = D / 16;   // m-tiles of the value product
    constexpr int XB = D / 128;  // 128-byte column blocks of a row
    extern __shared__ unsigned char smem_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *mbar = reinterpret_cast<uint64_t *>(smem + SM::kData);  // [warp][stage]
    volatile int *cta_abort = reinterpret_cast<volatile int *>(mbar + kStages * kWarps);

    const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z / A.nqt, qt = blockIdx.z % A.nqt;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int quad = lane & 3, row = lane >> 2;
    const int P = A.P, G = A.G;
    int L = A.seq_lens[b];
    if (L < 0) L = 0;
    if (L > A.max_blocks * P) {
        if (split == 0 && kvh == 0 && qt == 0 && tid == 0) atomicOr(A.status, TQ_DEVERR_SEQ_RANGE);
        L = A.max_blocks * P;
    }
    const int q0 = qt * A.qpc;
    const int ncol = min(A.qpc, A.Tq - q0) * G;
    auto col_row = [&](int c) -> size_t {  // output row of column c
        return (static_cast<size_t>(b) * A.Tq + q0 + c / G) * A.Hq + static_cast<size_t>(kvh) * G + c % G;
    };
    auto col_lim = [&](int c) -> int { return max(0, L - A.Tq + q0 + c / G + 1); };  // positions that it sees
    const size_t rows_total = static_cast<size_t>(A.B) * A.Tq * A.Hq;
    const int tok0 = split * A.pages_per_split * P;
    const int tok1 = min(col_lim(ncol - 1), tok0 + A.pages_per_split * P);
    if (tok0 >= tok1) {
        if (A.splits == 1) {
            for (int e = tid; e < ncol * (D / 2); e += kThreads)
                reinterpret_cast<uint32_t *>(A.out + col_row(e / (D / 2)) * D)[e % (D / 2)] = 0u;
        } else if (tid < ncol) {
            float *ml = A.ml + (static_cast<size_t>(split) * rows_total + col_row(tid)) * 2;
            ml[0] = -INFINITY;
            ml[1] = 0.f;
        }
        return;
    }
    const int nrounds = (tok1 - tok0 + kTok - 1) / kTok;

    if (tid < kStages * kWarps)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(&mbar[tid]))));
    if (tid == 0) *cta_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();

    const uint32_t sbase = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    auto stage_off = [&](int st) -> uint32_t { return static_cast<uint32_t>((warp * kStages + st) * SM::kStage); };
    auto mbar_addr = [&](int st) -> uint32_t {
        return static_cast<uint32_t>(__cvta_generic_to_shared(&mbar[warp * kStages + st]));
    };
    const int32_t *table = A.block_table + static_cast<int64_t>(b) * A.max_blocks;
    auto round_tok = [&](int rr) -> int { return tok0 + (kWarps * rr + warp) * kTok; };
    auto fetch_id = [&](int rr, int half) -> int {  // block of a round's 16-token half, -1 past the split
        const int t = round_tok(rr) + 16 * half;
        return t < tok1 ? __ldg(table + (t >> A.pshift)) : -1;
    };
    auto good = [&](int blk) -> bool { return blk >= 0 && blk < A.num_blocks; };
    auto issue = [&](int rr, int st, const int (&blk)[2]) {  // lane 0: the round's pages into a stage
        const int t = round_tok(rr);
        const int boxes = P == 16 ? 2 : 1;
        uint32_t bytes = 0;
#pragma unroll
        for (int p = 0; p < 2; ++p)
            if (p < boxes && good(blk[p])) bytes += static_cast<uint32_t>(2 * P * D);
            else if (p < boxes && t + 16 * p < tok1) atomicOr(A.status, TQ_DEVERR_BLOCK_RANGE);
        const uint32_t mb = mbar_addr(st);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // this warp's accesses of the stage are done
        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(mb), "r"(bytes) : "memory");
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (p >= boxes || !good(blk[p])) continue;
            const int y = static_cast<int>((static_cast<int64_t>(blk[p]) * A.Hkv + kvh) * P) + (P == 32 ? (t & 31) : 0);
            const uint32_t dk = sbase + stage_off(st) + p * 16 * 128;
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
    auto drain = [&](int st, uint32_t par) {
        const long long t0 = clock64();
        while (!mbar_try(mbar_addr(st), par) && clock64() - t0 < kDrainLimit) {
        }
    };

    const int my_rounds = (nrounds - warp + kWarps - 1) / kWarps;  // rounds warp, warp + kWarps, ...
    int ids[2] = {-1, -1}, ids1[2] = {-1, -1};  // blocks of the round to compute and of the next one
    if (my_rounds > 0) {
        ids[0] = fetch_id(0, 0);
        ids[1] = fetch_id(0, 1);
        if (lane == 0) issue(0, 0, ids);
    }
    // a zero limit tests the first copy at once, while it cannot be done: the way to the timeout path
    const bool first_ok = A.wait_limit > 0 || my_rounds == 0 || mbar_test(mbar_addr(0), 0);
    if (my_rounds > 1) {
        ids1[0] = fetch_id(1, 0);
        ids1[1] = fetch_id(1, 1);
    }

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
            for (int i = 0; i < 2; ++i) {
                w[s][i] = cv ? __ldg(qr + 8 * s + 4 * i + quad) : make_uint2(0u, 0u);
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
        if (ex < -100) ex = -100;
        if (ex > 120) ex = 120;
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
        lim[e] = c < ncol ? col_lim(c) : 0;
    }

    float o[MT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
    float m_run[2] = {-INFINITY, -INFINITY};  // columns 2 quad + e
    float l_run[2] = {0.f, 0.f};              // this lane's tokens' share of the denominators
    const int mi = lane >> 3, ri = lane & 7;
    const int krow = ri + 8 * (mi & 1), kch = mi >> 1;  // keys: matrices (rows 0-7 | 8-15) x (chunk c | c + 1)

    auto scale_of = [&](const float *p, int blk) -> float {
        return good(blk) ? __ldg(p + static_cast<int64_t>(blk) * A.Hkv + kvh) : 0.f;
    };
    float ks[2], vs[2];  // scales of the round to compute
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        ks[h] = scale_of(A.k_scales, ids[h]);
        vs[h] = scale_of(A.v_scales, ids[h]);
    }
    for (int c = 0; c < my_rounds; ++c) {
        const int st = c & 1;
        __syncwarp();  // every lane is done with the stage the next copy overwrites
        float ks1[2] = {0.f, 0.f}, vs1[2] = {0.f, 0.f};
        int ids2[2] = {-1, -1};
        if (c + 1 < my_rounds) {
            if (lane == 0) issue(c + 1, st ^ 1, ids1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                ks1[h] = scale_of(A.k_scales, ids1[h]);
                vs1[h] = scale_of(A.v_scales, ids1[h]);
                if (c + 2 < my_rounds) ids2[h] = fetch_id(c + 2, h);
            }
        }
        {
            const uint32_t par = (c >> 1) & 1;
            bool ok = true;
            if (A.wait_limit <= 0) {
                ok = c == 0 ? first_ok : mbar_test(mbar_addr(st), par);
            } else {
                const long long t0 = clock64();
                while (!mbar_try(mbar_addr(st), par))
                    if (clock64() - t0 > A.wait_limit) {
                        ok = false;
                        break;
                    }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                if (lane == 0) {
                    atomicOr(A.status, TQ_DEVERR_TIMEOUT);
                    *cta_abort = 1;
                }
                drain(st, par);
                if (c + 1 < my_rounds) drain(st ^ 1, ((c + 1) >> 1) & 1);
                break;
            }
        }
        const int t = round_tok(c);
        int nv[2];  // visible tokens of each half (of the column that sees most)
#pragma unroll
        for (int h = 0; h < 2; ++h) nv[h] = good(ids[h]) ? max(0, min(16, tok1 - t - 16 * h)) : 0;
        const uint32_t kbase = sbase + stage_off(st), vbase = kbase + SM::kTileBytes;
        if (nv[0] + nv[1] < kTok) {  // rows behind the end or of a bad page hold anything: zero the values
            unsigned char *vz = smem + stage_off(st) + SM::kTileBytes;
            for (int e = lane; e < kTok * (D / 16); e += 32) {
                const int rr = e / (D / 16), cc = e % (D / 16);
                if ((rr & 15) >= nv[rr >> 4])
                    *reinterpret_cast<uint4 *>(vz + (cc / 8) * kBoxBytes + rr * 128 + (cc % 8) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            __syncwarp();
        }
        // ---- scores ----
        float sc[2][4] = {};
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const uint32_t at = kbase + (s >> 2) * kBoxBytes + krow * 128 + (((2 * (s & 3) + kch) ^ (krow & 7)) << 4);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4(at + h * 16 * 128, a0, a1, a2, a3);
                mma_e4m3(sc[h], a0, a1, a2, a3, qh[s][0], qh[s][1]);
                mma_e4m3(sc[h], a0, a1, a2, a3, ql[s][0], ql[s][1]);
            }
        }
        // ---- mask, online softmax (base 2): this lane holds tokens row, row + 8 of each half, columns 2 quad + e ----
        float y[2][2][2], lv[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            lv[h] = log2_scale(vs[h]);
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int i = row + 8 * r;
                    const bool seen = i < nv[h] && t + 16 * h + i < lim[e];
                    y[h][r][e] = seen ? fmaf(sc[h][2 * r + e], fac[e] * ks[h], lv[h]) : -INFINITY;
                }
        }
        float alpha[2], shift[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mt = fmaxf(fmaxf(y[0][0][e], y[0][1][e]), fmaxf(y[1][0][e], y[1][1][e]));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 4));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 8));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
            const float m_new = fmaxf(m_run[e], mt);
            const bool none = m_new == -INFINITY;  // nothing seen so far (or only NaN)
            alpha[e] = none ? 1.f : fast_exp2(m_run[e] - m_new);
            shift[e] = none ? kPShift : kPShift - m_new;
            m_run[e] = m_new;
            l_run[e] *= alpha[e];
        }
        if (alpha[0] != 1.f || alpha[1] != 1.f) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                o[mt][0] *= alpha[0]; o[mt][1] *= alpha[1]; o[mt][2] *= alpha[0]; o[mt][3] *= alpha[1];
            }
        }
        // ---- P as the B operand: byte pairs (high, low) of a token and column, transposed
        // to (column `row`; tokens 2 quad, 2 quad + 1 | + 8, + 9), then high and low bytes apart ----
        uint32_t bh[2], bl[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float down = fast_exp2(kLShift - kPShift - lv[h]);
            uint32_t tr[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float p0 = fast_exp2(y[h][r][0] + shift[0]), p1 = fast_exp2(y[h][r][1] + shift[1]);
                l_run[0] = fmaf(p0, down, l_run[0]);
                l_run[1] = fmaf(p1, down, l_run[1]);
                const uint32_t hi = e4m3x2_rest(p0, p1), lo = e4m3x2(p0, p1);
                tr[r] = movmatrix_trans(__byte_perm(hi, lo, 0x5140));
            }
            bh[h] = __byte_perm(tr[0], tr[1], 0x6420);
            bl[h] = __byte_perm(tr[0], tr[1], 0x7531);
        }
        // ---- O[coordinate][column] += V^T P: the m-tile's rows are its even coordinates, then its odd ones ----
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t r0, r1, r2, r3;
            ldsm_x4_trans(vbase + (mt >> 3) * kBoxBytes + lane * 128 + (((mt & 7) ^ ri) << 4), r0, r1, r2, r3);
            const uint32_t a0 = __byte_perm(r0, r1, 0x6420), a1 = __byte_perm(r0, r1, 0x7531);
            const uint32_t a2 = __byte_perm(r2, r3, 0x6420), a3 = __byte_perm(r2, r3, 0x7531);
            mma_e4m3(o[mt], a0, a1, a2, a3, bh[0], bh[1]);
            mma_e4m3(o[mt], a0, a1, a2, a3, bl[0], bl[1]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            ks[h] = ks1[h];
            vs[h] = vs1[h];
            ids[h] = ids1[h];
            ids1[h] = ids2[h];
        }
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
    const float down = fast_exp2(-kPShift), ldown = fast_exp2(-kLShift);
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
            const float f = r_m[w * 8 + c] == -INFINITY ? 1.f : fast_exp2(r_m[w * 8 + c] - ref);
            acc = fmaf(f, r_o[(w * D + j) * 8 + c], acc);
            l = fmaf(f, r_l[w * 8 + c], l);
        }
        acc *= down;
        l *= ldown;
        if (dead) {
            M = -INFINITY;
            acc = l = 0.f;
        }
        const size_t orow = col_row(c);
        if (A.splits == 1) {
            A.out[orow * D + j] = float_to_bf16_bits(l == 0.f ? 0.f : acc / l);
        } else {
            const size_t pr = static_cast<size_t>(split) * rows_total + orow;
            A.acc[pr * D + j] = acc;
            if (j == 0) {
                A.ml[2 * pr] = M;
                A.ml[2 * pr + 1] = l;
            }
        }
    }
}

// Merges the splits of an output row: o = sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s.
// One warp per row, D / 32 coordinates per lane; a split that saw nothing (l = 0) has
// no partial to read.  A NaN of any split stays one.
template <int D>
__global__ void __launch_bounds__(128) merge_fp8_kernel(const float *__restrict__ ml, const float *__restrict__ acc,
                                                        uint16_t *__restrict__ out, int64_t rows, int splits)
{
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    float M = -INFINITY;
    for (int s = lane; s < splits; s += 32) M = fmaxf(M, __ldg(ml + (s * rows + row) * 2));
    M = warp_max(M);
    const float ref = M == -INFINITY ? 0.f : M;
    float n[E] = {}, den = 0.f;
    for (int s0 = 0; s0 < splits; s0 += 32) {
        float w = 0.f, l = 0.f;
        if (s0 + lane < splits) {
            const float2 v = __ldg(reinterpret_cast<const float2 *>(ml) + (s0 + lane) * rows + row);
            l = v.y;
            w = v.y == 0.f ? 0.f : (v.x == -INFINITY ? 1.f : fast_exp2(v.x - ref));
        }
        den += warp_sum(l == 0.f ? 0.f : w * l);
        const unsigned some = __ballot_sync(0xffffffffu, l != 0.f);
        const int k1 = min(32, splits - s0);
#pragma unroll 4
        for (int k = 0; k < k1; ++k) {
            const float wk = __shfl_sync(0xffffffffu, w, k);
            if (!(some >> k & 1u)) continue;
            const float *p = acc + ((s0 + k) * rows + row) * D + lane * E;
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
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint32_t *dst = reinterpret_cast<uint32_t *>(out + row * D + lane * E);
#pragma unroll
    for (int i = 0; i < E; i += 2)
        dst[i / 2] = float_to_bf16_bits(n[i] * inv) | (static_cast<uint32_t>(float_to_bf16_bits(n[i + 1] * inv)) << 16);
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

size_t workspace_bytes(int d, int64_t rows, int splits)
{
    if (splits <= 1) return 0;
    return align256(static_cast<size_t>(splits) * rows * 2 * sizeof(float)) +
           align256(static_cast<size_t>(splits) * rows * d * sizeof(float));
}

template <int D>
cudaError_t launch(const CUtensorMap &tk, const CUtensorMap &tv, const Args &a, bool tc, cudaStream_t st)
{
    cudaError_t e;
    if (tc) {
        e = launch_prefill_tc(tk, tv, D, a, st);
    } else {
        const size_t smem = Fp8Smem<D>::kBytes;
        e = ensure_smem_attr(reinterpret_cast<const void *>(attention_fp8_kernel<D>), smem);
        if (e != cudaSuccess) return e;
        attention_fp8_kernel<D><<<dim3(a.splits, a.Hkv, a.B * a.nqt), Fp8Smem<D>::kThreads, smem, st>>>(tk, tv, a);
        e = cudaGetLastError();
    }
    if (e != cudaSuccess || a.splits == 1) return e;
    const int64_t rows = static_cast<int64_t>(a.B) * a.Tq * a.Hq;
    merge_fp8_kernel<D><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, st>>>(a.ml, a.acc, a.out, rows, a.splits);
    return cudaGetLastError();
}

int clamp_splits(long long splits, long long most)
{
    if (splits > most) splits = most;
    if (splits > 256) splits = 256;
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
    // whole 32-token rounds per split, so that a split never begins inside a round's page pair
    const int ppr = kTok / P;
    a.pages_per_split = ((max_blocks + splits - 1) / splits + ppr - 1) / ppr * ppr;
    a.ml = static_cast<float *>(workspace);
    a.acc = reinterpret_cast<float *>(static_cast<char *>(workspace) +
                                      align256(static_cast<size_t>(splits) * rows * 2 * sizeof(float)));
    a.out = out;
    a.status = c.status;
    a.wait_limit = c.wait_limit;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    e = c.d == 128 ? launch<128>(tk, tv, a, tc, st) : launch<256>(tk, tv, a, tc, st);
    if (e != cudaSuccess) return api_error(TQ_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return TQ_OK;
}

}  // namespace
}  // namespace tq

extern "C" int tq_decode_splits_fp8(tq_handle h, int batch, int num_kv_heads, int max_blocks_per_seq, int page_size)
{
    if (!h || batch < 1 || num_kv_heads < 1 || max_blocks_per_seq < 1 || page_size < 1) return 1;
    const long long units = static_cast<long long>(batch) * num_kv_heads;
    const long long ctas = 8LL * tq::handle_codec(h).num_sms;
    const long long tiles = (static_cast<long long>(max_blocks_per_seq) * page_size + 127) / 128;
    return tq::clamp_splits((ctas + units - 1) / units, tiles);
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
    // one CTA per SM: about two waves, each split at least 512 tokens
    const long long most = (static_cast<long long>(max_blocks_per_seq) * page_size + 511) / 512;
    return tq::clamp_splits((2LL * tq::handle_codec(h).num_sms + units - 1) / units, most);
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
