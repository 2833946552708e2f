// tq_latent_narrow.cu -- attention over latent pages for sequences of up to 64 (query token, head) rows: one CTA per SM, tiles
// of 64 tokens.
//
//   S[r][t] = <q_r, [c_t | r_t]>      M = 64 rows (tensor-memory lanes 32 i .. 32 i + 15), N = 64 tokens
//   O^T[j][r] += sum_t c_t[j] P[r][t]  M = 128 coordinates (DL / 128 times), N = the rows rounded up to 16
// with P as in tq_latent.cu.  The second product is the transposed one: its A operand, the latents along coordinates, is the
// tile as it lies for the first, and DL x 64 sums are DL / 2 columns of tensor memory, where 64 x DL would be all of it.  P goes
// over the tile's rotated part, which the scores are done with.
//
// Few rows leave a tile bound by HBM: 64 x D x 2 bytes at an SM's share take ~3000 cycles, the products ~2100 (M = 64 runs at
// half the rate).  Against the pairs of tq_latent.cu (where half of the 128 rows would be idle) a tile needs nothing of
// another CTA and its chain from the last byte to the stage's release is shorter, so the two stages (four at DL = 256) keep
// more in flight.  Measured against the pairs for every call: 32 sequences of 1k to 8k of 64 heads 50.4 us instead of 50.7, 2 x
// 131k of 32 heads 61.5 instead of 64.5 (4.9 TB/s, 72% of the measured copy rate), 190 of up to 900 of 40 heads at DL = 256 26.5
// instead of 32.7, one of 500 of 8 heads 9.6 instead of 10.9 (a call in a graph, inputs that together pass L2).  P in one bf16
// term as there, so that a row's accuracy does not hang on how many there are.
//
// What bounds it: a tile takes 1.88 us between start and end where all SMs stream (HBM alone: 1.65); and beside the tiles ~7 us
// from the launch to the first scores and 3 to 6 for output and join.
// The loops over a tile's groups are not unrolled: the shorter code is worth 0.5 us (49.3 -> 48.7); the pairs' kernel, unrolled,
// is the faster one (568 against 574 us for chunks of 256 tokens).
//
// Warps: 8 softmax and output; 1 issue of the scores; 1 issue of P.V; 1 loads of tiles; 1 loads of Q.  Waits, shares of the work
// and pieces as in tq_latent.cu.
#include "tq_latent.cuh"
#include "tq_umma.cuh"

namespace tq {
namespace latent {
namespace {

constexpr int kTok = 64;  // tokens of a tile
constexpr int kThreads = kSoft + 128;

template <int DL>
struct Cfg {
    static constexpr int D = DL + kRope;
    static constexpr int NBLK = D / 64;           // blocks of 64 coordinates; the last one is the rotated part
    static constexpr int NX = DL / 128;           // P.V products of 128 coordinates
    static constexpr int NS = DL == 512 ? 2 : 4;  // stages
    static constexpr int GB = DL == 512 ? 3 : 5;  // blocks of a group, which has a barrier of its own
    static constexpr int NG = NBLK / GB;
    static_assert(NG * GB == NBLK, "whole groups");
    static constexpr uint32_t kBlk = 64 * 128;
    static constexpr uint32_t kOct = NBLK * 1024;  // eight tokens of a stage: NBLK blocks of 8 x 128 bytes
    static constexpr uint32_t kStage = NBLK * kBlk;
    static constexpr uint32_t kQOff = 0;
    static constexpr uint32_t kKOff = NBLK * kBlk;
    static constexpr uint32_t kBarOff = kKOff + NS * kStage;
    static constexpr int bQFull = 0;                 // Q landed
    static constexpr int bQFree = 1;                 // the piece's scores are done: Q may be overwritten
    static constexpr int bKFull = 2;                 // [NS][NG] blocks landed
    static constexpr int bSFull = bKFull + NS * NG;  // [2] scores in tensor memory
    static constexpr int bPFull = bSFull + 2;        // [2] P written, its scores read, O rescaled
    static constexpr int bPvDone = bPFull + 2;       // [NS] O += P V done: the stage is free
    static constexpr int bEnd = bPvDone + NS;        // [2] all MMAs issued by a warp are done
    static constexpr int kBars = bEnd + 2;
    static constexpr uint32_t kMiscOff = kBarOff + 8 * kBars;  // tensor-memory base, abort, NaN flag
    static constexpr uint32_t kOkOff = kMiscOff + 64;          // [8] a bit per 8 tokens of a tile
    static constexpr uint32_t kXOff = (kOkOff + 32 + 15) / 16 * 16;  // [2][64] exchange between the halves of a row
    static constexpr uint32_t kFacOff = kXOff + 4 * 128;       // [64] factors of the rows
    static constexpr uint32_t kPlanOff = kFacOff + 4 * 64;
    static constexpr uint32_t kSmem = kPlanOff + 32 + 8 * (kThreads / 32 + 3);
    static constexpr uint32_t kTmS = 0, kTmO = 128;  // [2] 64 columns; [NX] 64 columns
    static_assert(kSmem <= 232448, "shared memory");
};

__device__ __forceinline__ void mma_bf16(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi, uint32_t id, int acc)
{
    umma::mma_f16_lohi(d, a_lo, a_hi, b_lo, b_hi, id, acc);
}

// 32 columns of the 16 lanes that a 64-row product fills: word 4 j + e (+ 2) is row lane / 4 (+ 8), column 8 j + 2 (lane % 4) + e.
__device__ __forceinline__ void ld_rows(uint32_t taddr, float (&v)[16])
{
    uint32_t r[16];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr)
                 : "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

template <int DL>
__global__ void __launch_bounds__(kThreads, 1)
    latent_narrow_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmQ, const Args A)
{
    using C = Cfg<DL>;
    constexpr int NS = C::NS, NG = C::NG, NBLK = C::NBLK, NX = C::NX;
    extern __shared__ __align__(1024) unsigned char smem[];  // dynamic shared memory begins on a 1024-byte boundary
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int worker = blockIdx.x;
    const uint32_t sbase = saddr(smem);
    uint64_t *mbar = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    volatile int *misc = reinterpret_cast<volatile int *>(smem + C::kMiscOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kMiscOff);
    volatile int *abort_flag = misc + 1;  // misc[2]: something not finite was hidden
    volatile uint32_t *okmask = reinterpret_cast<volatile uint32_t *>(smem + C::kOkOff);
    float *xch = reinterpret_cast<float *>(smem + C::kXOff), *fac = reinterpret_cast<float *>(smem + C::kFacOff);
    int4 *jobs = reinterpret_cast<int4 *>(smem + C::kPlanOff);
    long long *plan = reinterpret_cast<long long *>(smem + C::kPlanOff + 32);  // see tq_latent.cu

    if (warp == kSoftWarps) umma::tmem_alloc(tmem_slot, 512);
    if (tid == 0) {
        umma::mbar_init(&mbar[C::bQFull], 1);
        umma::mbar_init(&mbar[C::bQFree], 1);
        for (int i = 0; i < NS * NG; ++i) umma::mbar_init(&mbar[C::bKFull + i], 1);
        for (int i = 0; i < NS; ++i) umma::mbar_init(&mbar[C::bPvDone + i], 1);
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(&mbar[C::bSFull + i], 1);
            umma::mbar_init(&mbar[C::bPFull + i], kSoftWarps);
            umma::mbar_init(&mbar[C::bEnd + i], 1);
        }
        for (int i = 1; i < 4; ++i) misc[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        A.done[worker] = 0;
        plan[kThreads / 32 + 2] = clock64();
    }
    umma::fence_before_sync();
    Dealer<kNarrowRows, kTok, kThreads> dealer;
    Share<kNarrowRows, kTok> share = dealer.deal(A, worker, blockIdx.x == 0, plan, jobs);
    umma::fence_after_sync();
    const uint32_t tbase = *tmem_slot;
    auto grid = cooperative_groups::this_grid();
    auto zeroed = grid.barrier_arrive();  // waited for before the first count
    dealer.find_jobs(A, jobs);

    // bounded waits, see tq_latent.cu
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
    auto wait_bar = [&](int i, uint32_t par) -> bool { return __all_sync(0xffffffffu, wait_one(i, par)); };
    auto drain = [&](int i, uint32_t par) {
        const long long t0 = clock64();
        while (!umma::mbar_try_wait(&mbar[i], par) && clock64() - t0 < kDrainLimit) {
        }
    };
    const int rows16 = (min(A.R, kNarrowRows) + 15) / 16 * 16;  // columns of O^T

    if (warp < kSoftWarps) {
        // ================= softmax, P, output =================
        // rows r0 and r0 + 8, tokens 32 g + 8 j + 2 (lane % 4) + {0, 1}; of O^T the coordinates of lanes 32 (warp % 4) .. in
        // half g of the products
        const int quad = warp & 3, g = warp >> 2, r0 = 16 * quad + (lane >> 2);
        const uint32_t lane_base = tbase + (static_cast<uint32_t>(32 * quad) << 16);
        const float c = fabsf(A.sm_scale) * kLog2e;
        const float slack = kSlack / c;
        const bool flip = A.sm_scale < 0.f;
        bool bad = false, dead = false;  // this warp's wait failed; all know
        int it = 0;
        Piece p, next;
        for (bool more = share.next(A, p); more; p = next) {
            const bool whole_unit = p.t0 == 0 && p.t1 == p.tiles;
            const size_t at = static_cast<size_t>(p.b) * A.R;
            const size_t slot = (2 * worker + (p.t0 == 0 ? 1 : 0)) * static_cast<size_t>(kNarrowRows);
            auto limit = [&](int row) -> int { return A.Tq == 1 || row >= A.R ? p.n : max(0, p.L - A.Tq + row / A.Hq + 1); };
            const int lim0 = limit(0);  // tokens that every row sees
            int lim[2];
            float m_run[2], m_most[2], l_run[2];  // reference; what does not move it yet; denominator
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                lim[e] = limit(r0 + 8 * e);
                m_run[e] = m_most[e] = -INFINITY;
                l_run[e] = 0.f;
            }
            bool far_ref = false;
            float shift[2] = {-kMargin, -kMargin};
            const int it0 = it;
            for (int i = p.t0; i < p.t1 && !dead; ++i, ++it) {
                bad |= !wait_bar(C::bSFull + (it & 1), (it >> 1) & 1);
                umma::fence_after_sync();
                float s[16];
                __syncwarp();
                ld_rows(lane_base + C::kTmS + 64 * (it & 1) + 32 * g, s);
                umma::fence_before_sync();
                const uint32_t ok4 = okmask[it & 7] >> (4 * g) & 15u;
                const int base = i * kTok + 32 * g + 2 * (lane & 3);
                const bool whole = __all_sync(0xffffffffu, min(lim[0], lim[1]) >= (i + 1) * kTok) && ok4 == 15u;
                auto hidden = [&](int k) -> bool {  // word k
                    return base + 8 * (k >> 2) + (k & 1) >= lim[k >> 1 & 1] || !(ok4 >> (k >> 2) & 1u);
                };
                if (flip) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) s[k] = -s[k];
                }
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (hidden(k)) s[k] = -INFINITY;
                }
                float top[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    top[e] = max3(max3(max3(s[2 * e], s[2 * e + 1], s[2 * e + 4]), s[2 * e + 5], s[2 * e + 8]),
                                  max3(s[2 * e + 9], s[2 * e + 12], s[2 * e + 13]), -INFINITY);
                }
                if (any_of_softmax(bad || top[0] > m_most[0] || top[1] > m_most[1])) {
                    if (any_of_softmax(bad)) {
                        dead = true;
                        break;
                    }
                    bool need = false;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
                        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
                        if ((lane & 3) == 0) xch[64 * g + r0 + 8 * e] = top[e];
                    }
                    any_of_softmax(false);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        top[e] = fmaxf(top[e], xch[64 * (g ^ 1) + r0 + 8 * e]);
                        const bool above = top[e] > m_most[e], moves = m_run[e] != -INFINITY && above;
                        const float al = moves ? fast_exp2((m_run[e] - top[e]) * c) : 1.f;
                        if (above) m_run[e] = top[e], m_most[e] = __fadd_rd(top[e], slack);
                        l_run[e] *= al;
                        need |= moves && r0 + 8 * e < A.R;
                        if (g == 0 && (lane & 3) == 0) fac[r0 + 8 * e] = al;
                    }
                    far_ref = __any_sync(0xffffffffu, (m_run[0] != -INFINITY && fabsf(m_run[0]) * c > kFar) ||
                                                          (m_run[1] != -INFINITY && fabsf(m_run[1]) * c > kFar));
#pragma unroll
                    for (int e = 0; e < 2; ++e) shift[e] = far_ref || m_run[e] == -INFINITY ? -kMargin : fmaf(-m_run[e], c, -kMargin);
                    if (any_of_softmax(need)) {  // there was a tile before
                        bad |= !wait_bar(C::bPvDone + (it - 1) % NS, ((it - 1) / NS) & 1);  // O is at rest
                        umma::fence_after_sync();
#pragma unroll 1
                        for (int x = g * (NX / 2); x < (g + 1) * (NX / 2); ++x)
#pragma unroll 1
                            for (int ch = 0; ch < rows16; ch += 16) {
                                float o[16];
                                __syncwarp();
                                umma::ld16(lane_base + C::kTmO + 64 * x + ch, o);
                                uint32_t w[16];
#pragma unroll
                                for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * fac[ch + k]);
                                umma::st16(lane_base + C::kTmO + 64 * x + ch, w);
                            }
                        umma::wait_st();
                        umma::fence_before_sync();
                    }
                }
                const uint32_t st = sbase + C::kKOff + (it % NS) * C::kStage;
                if (__builtin_expect(far_ref, 0)) {
#pragma unroll
                    for (int k = 0; k < 16; ++k) s[k] -= m_run[k >> 1 & 1] == -INFINITY ? 0.f : m_run[k >> 1 & 1];
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int k = 4 * j + 2 * e;
                        uint32_t w = bf16x2_of(fast_exp2(fmaf(s[k], c, shift[e])), fast_exp2(fmaf(s[k + 1], c, shift[e])));
                        if (!whole) {  // hidden: zero also where c is 0 or the reference infinite
                            if (hidden(k)) w &= 0xffff0000u;
                            if (hidden(k + 1)) w &= 0x0000ffffu;
                        }
                        l_run[e] += __uint_as_float(w << 16) + __uint_as_float(w & 0xffff0000u);
                        // row r of P: 64 tokens in 128 bytes of the rotated part's block, 16-byte chunks swizzled
                        const int r = r0 + 8 * e;
                        const uint32_t ad = st + (r >> 3) * C::kOct + (NBLK - 1) * 1024 + (r & 7) * 128 + (((4 * g + j) ^ (r & 7)) << 4) + 4 * (lane & 3);
                        asm volatile("st.shared.b32 [%0], %1;" ::"r"(ad), "r"(w) : "memory");
                    }
                const int rem_n = p.n - i * kTok, rem_0 = lim0 - i * kTok;
                if (rem_n < kTok || rem_0 < min(rem_n, kTok)) {
                    // values that some row must not see, see tq_latent.cu
                    constexpr int kChunks = DL / 8;
                    const int f = max(rem_0, 0);
                    for (int e = tid; e < (kTok - f) * kChunks; e += kSoft) {
                        const int t = f + e / kChunks, x = e % kChunks;
                        const uint32_t ad = st + (t >> 3) * C::kOct + (x >> 3) * 1024 + (t & 7) * 128 + (((x & 7) ^ (t & 7)) << 4);
                        if (t >= rem_n) {
                            sts128(ad, make_uint4(0u, 0u, 0u, 0u));
                            continue;
                        }
                        const uint4 v = lds128(ad);
                        uint32_t q[4] = {v.x, v.y, v.z, v.w};
                        bool found = false;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((q[k] & 0x7f80u) == 0x7f80u) q[k] &= 0xffff0000u, found = true;
                            if ((q[k] & 0x7f800000u) == 0x7f800000u) q[k] &= 0x0000ffffu, found = true;
                        }
                        if (found) {
                            sts128(ad, make_uint4(q[0], q[1], q[2], q[3]));
                            misc[2] = 1;
                        }
                    }
                }
                umma::fence_proxy_async();
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(saddr(&mbar[C::bPFull + (it & 1)])) : "memory");
            }
            more = share.next(A, next);  // while the last products run
            if (p.t0 < p.t1 && !dead) {
                bad |= !wait_bar(C::bPvDone + (it - 1) % NS, ((it - 1) / NS) & 1);
                umma::fence_after_sync();
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 1);
                    l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 2);
                    if ((lane & 3) == 0) xch[64 * g + r0 + 8 * e] = l_run[e];
                }
                dead = any_of_softmax(bad);
                if (!dead) {
                    if (g == 0 && (lane & 3) == 0) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int r = r0 + 8 * e;
                            const float l = l_run[e] + xch[64 + r];
                            fac[r] = l == 0.f ? 0.f : 1.f / l;
                            if (!whole_unit && r < A.R) A.ml[slot + r] = make_float2(m_run[e], l);
                        }
                    }
                    const bool nan = misc[2] != 0;
                    any_of_softmax(false);
                    const int32_t *table = A.block_table + static_cast<int64_t>(p.b) * A.max_blocks;
#pragma unroll 1
                    for (int x = g * (NX / 2); x < (g + 1) * (NX / 2); ++x) {
                        const int j = 128 * x + 32 * quad + lane;  // this lane's coordinate
#pragma unroll 1
                        for (int ch = 0; ch < rows16; ch += 16) {
                            float o[16];
                            __syncwarp();
                            umma::ld16(lane_base + C::kTmO + 64 * x + ch, o);
                            if (nan) {  // rows that see a token whose coordinate j is not finite
                                for (int t = lim0; t < p.n; ++t) {
                                    const int blk = __ldg(table + (t >> A.pshift));
                                    if (blk < 0 || blk >= A.num_blocks) continue;
                                    const uint16_t v = A.pool[(static_cast<int64_t>(blk) * A.P + (t & (A.P - 1))) * C::D + j];
                                    if ((v & 0x7f80u) != 0x7f80u) continue;
#pragma unroll
                                    for (int k = 0; k < 16; ++k)
                                        if (t < limit(ch + k)) o[k] = __uint_as_float(0x7fffffffu);
                                }
                            }
                            __syncwarp();
                            if (whole_unit) {
#pragma unroll
                                for (int k = 0; k < 16; k += 2) {
                                    // two lanes exchange, so that each has two neighbouring coordinates of one of two rows
                                    const float u0 = o[k] * fac[ch + k], u1 = o[k + 1] * fac[ch + k + 1];
                                    const float v = __shfl_xor_sync(0xffffffffu, lane & 1 ? u0 : u1, 1);
                                    const int r = ch + k + (lane & 1);
                                    if (r < A.R)
                                        *reinterpret_cast<uint32_t *>(A.out + (at + r) * DL + (j & ~1)) = lane & 1 ? bf16x2_of(v, u1) : bf16x2_of(u0, v);
                                }
                            } else {
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    if (ch + k < A.R) A.acc[(slot + ch + k) * DL + j] = o[k];
                            }
                        }
                    }
                    umma::fence_before_sync();
                    any_of_softmax(false);  // the factors and the flag have been read
                    if (tid == 0) misc[2] = 0;
                }
            }
            if (dead || p.tiles == 0) {  // nothing counts: zeros, or a piece without weight
                it = it0 + p.t1 - p.t0;
                if (p.tiles == 0 || whole_unit) {
                    uint4 *dst = reinterpret_cast<uint4 *>(A.out + at * DL);
                    for (int k = tid; k < A.R * (DL / 8); k += kSoft) dst[k] = make_uint4(0u, 0u, 0u, 0u);
                } else if (tid < A.R) {
                    A.ml[slot + tid] = make_float2(-INFINITY, kNothing);
                }
            }
        }
    } else if (warp == kSoftWarps) {
        // ================= issue of the scores =================
        if (umma::elect_one()) {
            constexpr uint32_t id = umma::idesc_bf16(64, kTok, false);
            const uint64_t d0 = umma::make_desc_sw128(sbase + C::kQOff, 16, 1024), dk = umma::make_desc_sw128(sbase + C::kKOff, 16, C::kOct);
            const uint32_t q_lo = static_cast<uint32_t>(d0), hi = static_cast<uint32_t>(d0 >> 32);
            const uint32_t kd_lo = static_cast<uint32_t>(dk), hi_k = static_cast<uint32_t>(dk >> 32);
            bool ok = true;
            int it = 0, sg = 0;
            Piece p;
            while (ok && share.next(A, p)) {
                if (p.tiles == 0) continue;
                ok = wait_one(C::bQFull, sg & 1);
                ++sg;
                for (int i = p.t0; ok && i < p.t1; ++i, ++it) {
                    if (it >= 2 && !(ok = wait_one(C::bPFull + (it & 1), ((it >> 1) - 1) & 1))) break;  // these columns are read
                    const uint32_t k_lo = kd_lo + (it % NS) * (C::kStage / 16);
                    const uint32_t ds = tbase + C::kTmS + 64 * (it & 1);
#pragma unroll
                    for (int b = 0; b < NBLK; ++b) {
                        if (b % C::GB == 0) {
                            if (!(ok = wait_one(C::bKFull + (it % NS) * NG + b / C::GB, (it / NS) & 1))) break;
                            umma::fence_after_sync();
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16(ds, q_lo + b * (C::kBlk / 16) + 2 * k, hi, k_lo + b * 64 + 2 * k, hi_k, id, b + k > 0);
                    }
                    if (ok) umma::commit(&mbar[C::bSFull + (it & 1)]);
                }
                if (ok) umma::commit(&mbar[C::bQFree]);
            }
            umma::commit(&mbar[C::bEnd]);
            drain(C::bEnd, 0);
        }
        __syncwarp();
    } else if (warp == kSoftWarps + 1) {
        // ================= issue of P.V =================
        if (umma::elect_one()) {
            const uint32_t id = umma::idesc_bf16(128, rows16, false) | (1u << 15);  // A along coordinates
            const uint64_t dp = umma::make_desc_sw128(sbase + C::kKOff + (NBLK - 1) * 1024, 16, C::kOct),
                           dv = umma::make_desc_sw128(sbase + C::kKOff, 1024, C::kOct);
            const uint32_t lo_p = static_cast<uint32_t>(dp), hi_p = static_cast<uint32_t>(dp >> 32);
            const uint32_t lo_v = static_cast<uint32_t>(dv), hi_v = static_cast<uint32_t>(dv >> 32);
            bool ok = true;
            int it = 0;
            Piece p;
            while (ok && share.next(A, p)) {
                for (int i = p.t0; ok && i < p.t1; ++i, ++it) {
                    if (!(ok = wait_one(C::bPFull + (it & 1), (it >> 1) & 1))) break;
                    umma::fence_after_sync();
                    const uint32_t st = (it % NS) * (C::kStage / 16);
#pragma unroll 1
                    for (int x = 0; x < NX; ++x)
#pragma unroll
                        for (int t = 0; t < kTok / 16; ++t)
                            mma_bf16(tbase + C::kTmO + 64 * x, lo_v + st + t * (2 * C::kOct / 16) + x * 128, hi_v, lo_p + st + 2 * t, hi_p, id,
                                     i > p.t0 || t > 0);
                    umma::commit(&mbar[C::bPvDone + it % NS]);
                }
            }
            umma::commit(&mbar[C::bEnd + 1]);
            drain(C::bEnd + 1, 0);
        }
        __syncwarp();
    } else if (warp == kSoftWarps + 2) {
        // ================= loads of tiles: boxes of eight tokens, a lane looks up one =================
        const int nowhere = static_cast<int>(A.num_blocks) << A.pshift;  // a row behind the pool: reads zeros
        const uint32_t k_full = saddr(&mbar[C::bKFull]);
        constexpr bool kPrefetch = NS == 2;  // with four stages it costs 2 % (190 sequences of up to 900 tokens 32.5 -> 33 us)
        int it = 0, issued = 0;
        bool ok = true;
        Piece p;
        while (ok && share.next(A, p)) {
            const int32_t *table = A.block_table + static_cast<int64_t>(p.b) * A.max_blocks;
            auto fetch_id = [&](int i) -> int {
                const int pos = i * kTok + 8 * (lane & 7);
                return i < p.t1 && pos < p.n ? __ldg(table + (pos >> A.pshift)) : -1;
            };
            int blk = fetch_id(p.t0);
            for (int i = p.t0; i < p.t1; ++i, ++it) {
                const int pos = i * kTok + 8 * (lane & 7);
                const bool good = blk >= 0 && blk < A.num_blocks;
                if (!good && pos < p.n) atomicOr(A.status, TQ_DEVERR_BLOCK_RANGE);
                const uint32_t valid = __ballot_sync(0xffffffffu, good || pos >= p.n) & 255u;
                const int y = good ? (blk << A.pshift) + (pos & (A.P - 1)) : nowhere;
                int row[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) row[k] = __shfl_sync(0xffffffffu, y, k);
                if (it >= NS && !(ok = wait_bar(C::bPvDone + it % NS, (it / NS - 1) & 1))) break;
                if (umma::elect_one()) {
                    okmask[it & 7] = valid;
                    const uint32_t st = sbase + C::kKOff + (it % NS) * C::kStage;
                    const uint32_t full = k_full + 8 * NG * (it % NS);
#pragma unroll 1
                    for (int x = 0; x < NG; ++x) {
                        asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full + 8 * x), "r"(8 * 1024 * C::GB) : "memory");
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                                         ::"r"(st + k * C::kOct + x * (C::GB * 1024)), "l"(reinterpret_cast<uint64_t>(&tmK)), "r"(0), "r"(row[k]), "r"(C::GB * x), "r"(full + 8 * x)
                                         : "memory");
                    }
                }
                __syncwarp();
                issued = it + 1;
                blk = fetch_id(i + 1);
                if (kPrefetch) prefetch_rows<C::D>(A, i * kTok + NS * kTok + 8 * (lane & 7), fetch_id(i + NS), lane < 8);
            }
        }
        for (int t = max(0, issued - NS); t < issued; ++t)
            for (int x = 0; x < NG; ++x) drain(C::bKFull + (t % NS) * NG + x, (t / NS) & 1);
    } else {
        // ================= loads of Q =================
        int sg = 0;
        bool ok = true;
        Piece p;
        while (ok && share.next(A, p)) {
            if (p.tiles == 0) continue;
            if (sg > 0 && !(ok = wait_bar(C::bQFree, (sg - 1) & 1))) break;
            if (umma::elect_one()) {
                const uint32_t full = saddr(&mbar[C::bQFull]);
                asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full), "r"(NBLK * C::kBlk) : "memory");
                asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                             ::"r"(sbase + C::kQOff), "l"(reinterpret_cast<uint64_t>(&tmQ)), "r"(0), "r"(p.b * A.R), "r"(0), "r"(full)
                             : "memory");
            }
            __syncwarp();
            ++sg;
        }
        if (sg > 0) drain(C::bQFull, (sg - 1) & 1);
    }

    // copies and MMAs in flight have ended: the warps that issued them have waited
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    __syncwarp();
    if (warp == kSoftWarps) umma::tmem_dealloc(tbase, 512);
    grid.barrier_wait(std::move(zeroed));
    join<DL, kNarrowRows, kThreads>(A, jobs, worker, 0, 1, plan[kThreads / 32 + 2], *reinterpret_cast<Merge *>(smem));
}

template <int DL>
cudaError_t launch(const CUtensorMap &tk, const CUtensorMap &tq, const Args &a, cudaStream_t st)
{
    return launch_together(latent_narrow_kernel<DL>, 1, kThreads, Cfg<DL>::kSmem, st, a, tk, tq);
}

}  // namespace

int narrow_group(int dl) { return dl == 512 ? Cfg<512>::GB : Cfg<256>::GB; }

cudaError_t launch_narrow(const CUtensorMap &tk, const CUtensorMap &tq, int dl, const Args &a, cudaStream_t st)
{
    return dl == 512 ? launch<512>(tk, tq, a, st) : launch<256>(tk, tq, a, st);
}

}  // namespace latent
}  // namespace tq
