// tq_latent.cu -- attention over latent pages: every head's keys and values are one shared row [c | r] a token.
//
//   S[r][t] = <q_r, [c_t | r_t]>    r: (query token, head) rows of a sequence, D = DL + 64 coordinates
//   O[r][j] = sum_t P[r][t] c_t[j]  j < DL
// with y = sm_scale log2(e) S, P = 2^(y - m) rounded to bf16 (m as kMargin says), the denominator the fp32 sum of the rounded P.
//
// All heads read the same rows, so a tile of 128 tokens serves 128 rows: 2 (D + DL) 128 flops against 2 D bytes a token,
// 242 flop/B at DL = 512.  O is 128 x 512 in fp32, all of an SM's tensor memory; so a pair of CTAs (a cluster of two)
// shares a tile, M = 128 across the pair (cta_group::2): a CTA holds 64 rows of Q, O and P, and of each tile
//   for the scores   its own 64 tokens, all D coordinates (half of B's rows), in blocks of 64 tokens x 64 coordinates;
//   for P.V          all 128 tokens of its own DL/2 coordinates (half of B's columns).
// Both products take B from the same offsets in the two CTAs.  Block b of a stage holds the CTA's own tokens' coordinates
// 64 b .. 64 b + 63 for the scores; then the half of the blocks that are the other CTA's coordinates are dead, and the
// other CTA's tokens of this CTA's coordinates are loaded over them (from L2, where the other CTA has just brought them):
// blocks 0 .. NO - 1 hold the tile's first 64 tokens in both CTAs, NO .. 2 NO - 1 the last 64.  So a stage is 64 x D and two
// stages fit beside Q (four at DL = 256).
//
// Work is dealt to the pairs in equal shares of 128-token tiles, in the order of the units (sequence, block of 128 rows):
// every CTA finds its share from the lengths.  The pairs that share a unit leave their sums in the workspace and join them at
// their ends, each a part of the rows.
//
// P.V goes through the tokens, and at the middle hands back the blocks and the half of P that only the first 64 of them use (with
// all at the end 571 instead of 551 us in the second case below).
//
// P is one bf16 term: a second one for its remainder would be a second value product, half of a tile's tensor work again, and its
// buffers have no room beside the stages.  It adds 4 to 9% to the error that the output's own rounding leaves (16% for a few
// hundred tokens).
//
// Measured (a call in a graph): 1024 tokens behind 15k of 128 heads, DL = 512: 2.85 ms, 1.59 PFLOP/s, 83% of the measured bf16
// rate; 256 tokens of 4 sequences of 2k to 8k, 64 heads: 552 us, 1.55 PFLOP/s.  A tile's products take ~2180 cycles of the tensor
// pipe, but read 2875 cycles' worth of shared memory: that bounds a tile, ~3050 cycles.  Decode of 8 x 32k tokens of 128 heads:
// 74.5 us, 4.1 TB/s; 4 tokens of 24 sequences of 1k to 9k, 32 heads: 51 us; there start (~7 us to the first scores), the chain load
// - scores - softmax - P.V through two stages, and the join take what is above HBM's time.  At DL = 256 the softmax warps bound a
// tile: ~1900 cycles against 1150 of the products.
//
// Warps (one CTA per SM): 8, a thread per row and quarter of the tile's tokens: softmax, P, output; 1 issue of the scores and 1
// of P.V (in the pair's first CTA, for both); 1 loads of the tiles; 1 loads of Q and over the dead blocks.
// Every wait on a barrier in shared memory, and the join's for other workers' pieces, is bounded by the handle's wait limit (see
// join); a timeout sets TQ_DEVERR_TIMEOUT and stops the CTA, whose rows then carry no weight, or are zeros where the join gave
// up; copies and MMAs in flight finish before the pair ends.  The barrier over the grid has no limit and needs none: a block
// arrives at it before it waits for anything but its own threads and its cluster's start, and all blocks run at once.
#include <climits>
#include <cmath>

#include "tq_latent.cuh"
#include "tq_umma.cuh"

namespace tq {
namespace latent {
namespace {

constexpr int kTile = 128;       // tokens of a tile, rows of a unit
constexpr int kHalf = 64;        // a CTA's tokens and rows
constexpr int kThreads = kSoft + 128;

template <int DL>
struct Cfg {
    static constexpr int D = DL + kRope;
    static constexpr int NBLK = D / 64;      // blocks of a stage; the last one is the rotated part
    static constexpr int NO = DL / 128;      // blocks of the CTA's own coordinates
    static constexpr int NX = DL / 256;      // P.V products of 256 coordinates (128 of each CTA)
    static constexpr int NS = DL == 512 ? 2 : 4;  // stages
    static constexpr int NP = DL == 512 ? 1 : 2;  // buffers of P's first half (the second goes over the rotated part)
    static constexpr int GB = DL == 512 ? 3 : 5;  // blocks of a group, which has a barrier of its own
    static constexpr int NG = NBLK / GB;
    static_assert(NG * GB == NBLK, "whole groups");
    static constexpr int kHalfGroups = NO / GB;  // groups of the first half of the tokens' values alone
    static constexpr uint32_t kBlk = 64 * 128;
    static constexpr uint32_t kOct = NBLK * 1024; // eight tokens of a stage: NBLK blocks of 8 x 128 bytes
    static constexpr uint32_t kStage = NBLK * kBlk;
    static constexpr uint32_t kQOff = 0;
    static constexpr uint32_t kKOff = NBLK * kBlk;
    static constexpr uint32_t kPOff = kKOff + NS * kStage;
    static constexpr uint32_t kBarOff = kPOff + NP * kBlk;
    // barriers; (L) the pair's first CTA's counts for both
    static constexpr int bQFull = 0;                // (L) Q landed
    static constexpr int bKFull = 1;                // (L) [NS][NG] own tokens' blocks landed
    static constexpr int bVFull = bKFull + NS * NG; // [NS] the other tokens' blocks landed
    static constexpr int bSFull = bVFull + NS;      // [2] scores in tensor memory
    static constexpr int bPFull = bSFull + 2;       // (L) [2] P written, its scores read, O rescaled
    static constexpr int bPvDone = bPFull + 2;      // [NS] O += P V done: the stage is free
    static constexpr int bPvHalf = bPvDone + NS;    // [NS] and those of the first half of its tokens
    static constexpr int bEnd = bPvHalf + NS;       // (L) [2] teardown: all MMAs issued by a warp are done
    static constexpr int kBars = bEnd + 2;
    static constexpr uint32_t kMiscOff = kBarOff + 8 * kBars;   // tensor-memory base, abort, issued counts, NaN flags
    static constexpr uint32_t kOkOff = kMiscOff + 64;           // [8] a bit per 8 tokens of a tile: behind the end, or on a valid page
    static constexpr uint32_t kXOff = kOkOff + 32;              // [kSoft] exchange between the four threads of a row
    static constexpr uint32_t kPlanOff = (kXOff + 4 * kSoft + 15) / 16 * 16;  // scan and plan
    static constexpr uint32_t kSmem = kPlanOff + 32 + 8 * (kThreads / 32 + 3);
    static constexpr uint32_t kTmS = 0, kTmO = 256;  // [2] 64 columns; DL / 2 columns
    static_assert(kSmem <= 232448, "shared memory");
};

template <int DL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ CUtensorMap tmQ, const Args A)
{
    using C = Cfg<DL>;
    constexpr int NS = C::NS, NG = C::NG, NBLK = C::NBLK, NO = C::NO;
    extern __shared__ __align__(1024) unsigned char smem[];  // dynamic shared memory begins on a 1024-byte boundary
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t rank = umma::cluster_rank();
    const int pair = blockIdx.x >> 1;
    const uint32_t sbase = saddr(smem);
    uint64_t *mbar = reinterpret_cast<uint64_t *>(smem + C::kBarOff);
    volatile int *misc = reinterpret_cast<volatile int *>(smem + C::kMiscOff);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kMiscOff);
    volatile int *abort_flag = misc + 1;
    // misc[2..3] groups of tiles and [4..5] Qs whose copies this and the other CTA issued; [6..7] NaN flags by a piece's parity
    volatile uint32_t *okmask = reinterpret_cast<volatile uint32_t *>(smem + C::kOkOff);
    float *xch = reinterpret_cast<float *>(smem + C::kXOff);
    int4 *jobs = reinterpret_cast<int4 *>(smem + C::kPlanOff);
    long long *plan = reinterpret_cast<long long *>(smem + C::kPlanOff + 32);  // warps' sums; then the first unit's first cost, and the unit; when the block began

    if (warp == kSoftWarps) umma::tmem_alloc_pair(tmem_slot, 512);
    if (tid == 0) {
        umma::mbar_init(&mbar[C::bQFull], 2);
        for (int i = 0; i < NS * NG; ++i) umma::mbar_init(&mbar[C::bKFull + i], 2);
        for (int i = 0; i < NS; ++i) {
            umma::mbar_init(&mbar[C::bVFull + i], 1);
            umma::mbar_init(&mbar[C::bPvDone + i], 1);
            umma::mbar_init(&mbar[C::bPvHalf + i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            umma::mbar_init(&mbar[C::bSFull + i], 1);
            umma::mbar_init(&mbar[C::bPFull + i], 2 * kSoftWarps);
            umma::mbar_init(&mbar[C::bEnd + i], 1);
        }
        for (int i = 1; i < 8; ++i) misc[i] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (rank == 0) A.done[pair] = 0;
        plan[kThreads / 32 + 2] = clock64();
    }

    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    Dealer<kTile, kTile, kThreads> dealer;
    Share<kTile, kTile> share = dealer.deal(A, pair, blockIdx.x == 0, plan, jobs);
    umma::cluster_sync();
    auto grid = cooperative_groups::this_grid();
    auto zeroed = grid.barrier_arrive();  // waited for before the first count
    dealer.find_jobs(A, jobs);
    const uint32_t tbase = *tmem_slot;

    // bounded waits, by a warp and by one thread: they give up on the CTA's abort flag or after the wait limit (then raising
    // the flag and the status bit); a zero limit tests once
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
    auto leader = [&](int i) -> uint32_t { return umma::peer_addr(saddr(&mbar[i]), 0); };
    auto drain = [&](int i, uint32_t par) {
        const long long t0 = clock64();
        while (!umma::mbar_try_wait(&mbar[i], par) && clock64() - t0 < kDrainLimit) {
        }
    };

    if (warp < kSoftWarps) {
        // ================= a quarter of a row's tokens: softmax, P, output =================
        // row r, half h of the tile's tokens (and of the coordinates), columns 32 g .. of that half
        const int r = tid & 63, h = (tid >> 6) & 1, g = tid >> 7;
        const uint32_t lane_base = tbase + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const float c = fabsf(A.sm_scale) * kLog2e;
        const float slack = kSlack / c;
        const uint32_t flip = A.sm_scale < 0.f ? 0x80000000u : 0u;
        const int *table = nullptr;
        const bool sectors = (reinterpret_cast<uintptr_t>(A.out) & 31) == 0;  // rows begin on 32 bytes
        bool bad = false, dead = false;  // this warp's wait failed; all know
        int it = 0, sg = 0;
        Piece p, next;
        for (bool more = share.next(A, p); more; p = next) {
            const int row = p.rt * kTile + static_cast<int>(rank) * kHalf + r;
            const bool valid = row < A.R;
            const size_t at = static_cast<size_t>(p.b) * A.R + row;
            const bool whole_unit = p.t0 == 0 && p.t1 == p.tiles;
            const size_t slot = (2 * pair + (p.t0 == 0 ? 1 : 0)) * static_cast<size_t>(kTile) + rank * kHalf + r;
            table = A.block_table + static_cast<int64_t>(p.b) * A.max_blocks;
            const int lim0 = max(0, p.L - A.Tq + (A.Tq == 1 ? 0 : p.rt * kTile / A.Hq) + 1);  // tokens that every row sees
            const int lim = A.Tq == 1 || !valid ? p.n : max(0, p.L - A.Tq + row / A.Hq + 1);
            float m_run = -INFINITY, m_most = -INFINITY, l_run = 0.f;  // reference; what does not move it yet
            bool far_ref = false;
            float base = -kMargin;
            const int it0 = it;
            for (int i = p.t0; i < p.t1 && !dead; ++i, ++it) {
                bad |= !wait_bar(C::bSFull + (it & 1), (it >> 1) & 1);
                umma::fence_after_sync();
                float sf[32];
                __syncwarp();
                umma::ld32(lane_base + C::kTmS + 64 * (it & 1) + 32 * g, sf);
                umma::fence_before_sync();
                const int rem = lim - i * kTile - h * kHalf - 32 * g;  // of these tokens, those that the row sees
                const uint32_t ok4 = okmask[it & 7] >> (8 * h + 4 * g) & 15u;
                const bool whole = __all_sync(0xffffffffu, rem >= 32 && ok4 == 15u);
                if (flip) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) sf[k] = -sf[k];
                }
                if (!whole) {
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (k >= rem || !(ok4 >> (k >> 3) & 1u)) sf[k] = -INFINITY;
                }
                float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    m0 = max3(m0, sf[k], sf[k + 1]);
                    m1 = max3(m1, sf[k + 2], sf[k + 3]);
                }
                float top = fmaxf(m0, m1);
                if (any_of_softmax(bad || top > m_most)) {
                    if (any_of_softmax(bad)) {
                        dead = true;
                        break;
                    }
                    xch[tid] = top;
                    any_of_softmax(false);
                    top = fmaxf(fmaxf(top, xch[tid ^ 64]), fmaxf(xch[tid ^ 128], xch[tid ^ 192]));
                    const bool moves = top > m_most, need = valid && m_run != -INFINITY && moves;
                    const float al = need ? fast_exp2((m_run - top) * c) : 1.f;
                    if (moves) m_run = top, m_most = __fadd_rd(top, slack);
                    far_ref = __any_sync(0xffffffffu, m_run != -INFINITY && fabsf(m_run) * c > kFar);
                    base = far_ref || m_run == -INFINITY ? -kMargin : fmaf(-m_run, c, -kMargin);
                    if (__any_sync(0xffffffffu, need)) {  // need: there was a tile before
                        bad |= !wait_bar(C::bPvDone + (it - 1) % NS, ((it - 1) / NS) & 1);  // O is at rest
                        umma::fence_after_sync();
                        const uint32_t to = lane_base + C::kTmO + g * (DL / 4);
#pragma unroll 1
                        for (int ch = 0; ch < DL / 4; ch += 32) {
                            float o[32];
                            __syncwarp();
                            umma::ld32(to + ch, o);
                            uint32_t w[32];
#pragma unroll
                            for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(o[k] * al);
                            umma::st32(to + ch, w);
                        }
                        umma::wait_st();
                        umma::fence_before_sync();
                        l_run *= al;
                    }
                }
                if (far_ref) {
                    const float ref = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        const float2 d = unpack2(add2(pack2(sf[k], sf[k + 1]), pack2(-ref, -ref)));
                        sf[k] = d.x;
                        sf[k + 1] = d.y;
                    }
                }
                const uint64_t c2 = pack2(c, c), base2 = pack2(base, base);
                uint64_t sum0 = 0, sum1 = 0;
                uint32_t w[16];
#pragma unroll
                for (int k = 0; k < 32; k += 4) {
                    float2 x0 = unpack2(fma2(pack2(sf[k], sf[k + 1]), c2, base2));
                    float2 x1 = unpack2(fma2(pack2(sf[k + 2], sf[k + 3]), c2, base2));
                    x0.x = fast_exp2(x0.x);
                    x0.y = fast_exp2(x0.y);
                    x1.x = fast_exp2(x1.x);
                    x1.y = fast_exp2(x1.y);
                    w[k / 2] = bf16x2_of(x0.x, x0.y);
                    w[k / 2 + 1] = bf16x2_of(x1.x, x1.y);
                }
                if (!whole) {  // hidden: zero also where c is 0 or the reference infinite
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if (k >= rem || !(ok4 >> (k >> 3) & 1u)) w[k / 2] &= k & 1 ? 0x0000ffffu : 0xffff0000u;
                }
#pragma unroll
                for (int k = 0; k < 16; k += 2) {
                    sum0 = add2(sum0, pack2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u)));
                    sum1 = add2(sum1, pack2(__uint_as_float(w[k + 1] << 16), __uint_as_float(w[k + 1] & 0xffff0000u)));
                }
                const float2 sum = unpack2(add2(sum0, sum1));
                l_run += sum.x + sum.y;
                // P: the first half's buffer is free when an earlier tile's P.V is done, the rotated part with these scores
                if (h == 0 && it >= C::NP) bad |= !wait_bar(C::bPvHalf + (it - C::NP) % NS, ((it - C::NP) / NS) & 1);
                const uint32_t st = sbase + C::kKOff + (it % NS) * C::kStage;
                const uint32_t pd = h == 0 ? sbase + C::kPOff + (it % C::NP) * C::kBlk + r * 128
                                           : st + (r >> 3) * C::kOct + (NBLK - 1) * 1024 + (r & 7) * 128;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    sts128(pd + (((4 * g + k) ^ (r & 7)) << 4), make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
                bad |= !wait_bar(C::bVFull + it % NS, (it / NS) & 1);
                const int rem_n = p.n - i * kTile, rem_0 = lim0 - i * kTile;
                if (rem_n < kTile || rem_0 < min(rem_n, kTile)) {
                    // Values that some row must not see: 0 times NaN or infinity would reach it.  Tokens behind the last one
                    // become zeros.  Of those that only some rows see, what is not finite becomes zero, and the rows that
                    // see it get their NaN at the end.
                    const int f = max(rem_0, 0);
                    for (int e = tid; e < (kTile - f) * 8 * NO; e += kSoft) {
                        const int t = f + e / (8 * NO), x = e % (8 * NO);
                        const uint32_t ad = st + ((t & 63) >> 3) * C::kOct + ((t >> 6) * NO + (x >> 3)) * 1024 + (t & 7) * 128 + (((x & 7) ^ (t & 7)) << 4);
                        if (t >= rem_n) {
                            sts128(ad, make_uint4(0u, 0u, 0u, 0u));
                            continue;
                        }
                        uint4 v = lds128(ad);
                        uint32_t q[4] = {v.x, v.y, v.z, v.w};
                        bool found = false;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            if ((q[k] & 0x7f80u) == 0x7f80u) q[k] &= 0xffff0000u, found = true;
                            if ((q[k] & 0x7f800000u) == 0x7f800000u) q[k] &= 0x0000ffffu, found = true;
                        }
                        if (found) {
                            sts128(ad, make_uint4(q[0], q[1], q[2], q[3]));
                            const uint32_t flag = sbase + C::kMiscOff + 4 * (6 + (sg & 1));
                            for (uint32_t to = 0; to < 2; ++to)
                                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(umma::peer_addr(flag, to)), "r"(1u) : "memory");
                            asm volatile("fence.acq_rel.cluster;" ::: "memory");
                        }
                    }
                }
                umma::fence_proxy_async();
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) umma::cluster_arrive(leader(C::bPFull + (it & 1)));
            }
            more = share.next(A, next);  // while the last products run
            if (p.t0 < p.t1 && !dead) {
                bad |= !wait_bar(C::bPvDone + (it - 1) % NS, ((it - 1) / NS) & 1);
                umma::fence_after_sync();
                xch[tid] = l_run;
                dead = any_of_softmax(bad);
                if (!dead) {
                    l_run = (l_run + xch[tid ^ 64]) + (xch[tid ^ 128] + xch[tid ^ 192]);
                    const bool nan = misc[6 + (sg & 1)] != 0;
                    const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
#pragma unroll 1
                    for (int ch = g * (DL / 4); ch < (g + 1) * (DL / 4); ch += 32) {
                        __syncwarp();
                        // columns 128 x .. of the first lanes are coordinates 128 x .., of the last ones DL / 2 + 128 x ..
                        const int j0 = h * (DL / 2) + ch;
                        float o[32];
                        umma::ld32(lane_base + C::kTmO + ch, o);
                        if (nan && valid) {
                            for (int t = lim0; t < lim; ++t) {
                                const int blk = __ldg(table + (t >> A.pshift));
                                if (blk < 0 || blk >= A.num_blocks) continue;
                                const uint16_t *src = A.pool + (static_cast<int64_t>(blk) * A.P + (t & (A.P - 1))) * C::D + j0;
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    if ((src[k] & 0x7f80u) == 0x7f80u) o[k] = __uint_as_float(0x7fffffffu);
                            }
                        }
                        if (valid && whole_unit) {
                            uint16_t *dst = A.out + at * DL + j0;
#pragma unroll
                            for (int k = 0; k < 32; k += 16) {
                                float v[8];
#pragma unroll
                                for (int m = 0; m < 8; ++m) v[m] = __uint_as_float(bf16x2_of(o[k + 2 * m] * inv, o[k + 2 * m + 1] * inv));
                                if (sectors) {
                                    stg256(reinterpret_cast<float *>(dst + k), v);
                                } else {
                                    reinterpret_cast<float4 *>(dst + k)[0] = make_float4(v[0], v[1], v[2], v[3]);
                                    reinterpret_cast<float4 *>(dst + k)[1] = make_float4(v[4], v[5], v[6], v[7]);
                                }
                            }
                        } else if (valid) {
#pragma unroll
                            for (int k = 0; k < 32; k += 8) {
                                const float v[8] = {o[k], o[k + 1], o[k + 2], o[k + 3], o[k + 4], o[k + 5], o[k + 6], o[k + 7]};
                                stg256(A.acc + slot * DL + j0 + k, v);
                            }
                        }
                    }
                    umma::fence_before_sync();
                    if (!whole_unit && valid && tid < 64) A.ml[slot] = make_float2(m_run, l_run);
                    any_of_softmax(false);  // the exchange and the flag have been read
                    if (tid == 0) misc[6 + (sg & 1)] = 0;
                }
            }
            if (dead || p.tiles == 0) {  // nothing counts: zeros, or a piece without weight
                it = it0 + p.t1 - p.t0;
                if (valid && (p.tiles == 0 || whole_unit)) {
                    uint4 *dst = reinterpret_cast<uint4 *>(A.out + at * DL + (2 * h + g) * (DL / 4));
                    for (int k = 0; k < DL / 32; ++k) dst[k] = make_uint4(0u, 0u, 0u, 0u);
                } else if (valid && tid < 64) {
                    A.ml[slot] = make_float2(-INFINITY, kNothing);
                }
            }
            if (p.tiles) ++sg;
        }
    } else if (warp == kSoftWarps) {
        // ================= issue of the scores, for both CTAs =================
        if (rank == 0 && umma::elect_one()) {
            constexpr uint32_t id = umma::idesc_bf16(128, kTile, false);
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
                            umma::mma_f16_pair(ds, q_lo + b * (C::kBlk / 16) + 2 * k, hi, k_lo + b * 64 + 2 * k, hi_k, id,
                                               b + k > 0);
                    }
                    if (ok) umma::commit_pair(&mbar[C::bSFull + (it & 1)]);
                }
            }
            umma::commit_pair(&mbar[C::bEnd]);
            drain(C::bEnd, 0);
        }
        __syncwarp();
    } else if (warp == kSoftWarps + 1) {
        // ================= issue of P.V, for both CTAs =================
        if (rank == 0 && umma::elect_one()) {
            constexpr uint32_t id = umma::idesc_bf16(128, 256, true);
            const uint64_t dp = umma::make_desc_sw128(sbase, 16, 1024), dr = umma::make_desc_sw128(sbase, 16, C::kOct),
                           dv = umma::make_desc_sw128(sbase, 1024, C::kOct);
            const uint32_t lo_p = static_cast<uint32_t>(dp), hi_p = static_cast<uint32_t>(dp >> 32);
            const uint32_t lo_r = static_cast<uint32_t>(dr), hi_r = static_cast<uint32_t>(dr >> 32);
            const uint32_t lo_v = static_cast<uint32_t>(dv), hi_v = static_cast<uint32_t>(dv >> 32);
            bool ok = true;
            int it = 0;
            Piece p;
            while (ok && share.next(A, p)) {
                for (int i = p.t0; ok && i < p.t1; ++i, ++it) {
                    if (!(ok = wait_one(C::bPFull + (it & 1), (it >> 1) & 1))) break;
                    umma::fence_after_sync();
                    const uint32_t st = (C::kKOff + (it % NS) * C::kStage) / 16;
#pragma unroll
                    for (int t = 0; t < 8; ++t)  // 16 tokens
#pragma unroll
                        for (int x = 0; x < C::NX; ++x) {
                            const uint32_t pa = 2 * (t & 3) + (t < 4 ? lo_p + (C::kPOff + (it % C::NP) * C::kBlk) / 16
                                                                     : lo_r + st + (NBLK - 1) * 64);
                            const uint32_t va = lo_v + st + (t & 3) * (2 * C::kOct / 16) + ((t >> 2) * NO + 2 * x) * 64;
                            umma::mma_f16_pair(tbase + C::kTmO + 128 * x, pa, t < 4 ? hi_p : hi_r, va, hi_v, id, i > p.t0 || t > 0);
                            if (t == 3 && x == C::NX - 1) umma::commit_pair(&mbar[C::bPvHalf + it % NS]);
                        }
                    umma::commit_pair(&mbar[C::bPvDone + it % NS]);
                }
            }
            umma::commit_pair(&mbar[C::bEnd + 1]);
            drain(C::bEnd + 1, 0);
        }
        __syncwarp();
    } else if (warp == kSoftWarps + 2) {
        // ================= loads: the tiles' own tokens =================
        // Eight tokens are a box (all their coordinates lie side by side in the pool): lane j looks up the tile's tokens
        // 8 j .. 8 j + 7.  Block ids are read a tile ahead, behind the copies, so that no release waits for them.
        const int nowhere = static_cast<int>(A.num_blocks) << A.pshift;  // a row behind the pool: reads zeros
        int it = 0;
        bool ok = true;
        const uint32_t k_full = leader(C::bKFull);
        const bool far = NS == 2 && A.RT == 1;  // several row blocks read the same tiles, which are in L2 then
        Piece p;
        while (ok && share.next(A, p)) {
            if (p.tiles == 0) continue;
            const int32_t *table = A.block_table + static_cast<int64_t>(p.b) * A.max_blocks;
            auto fetch_id = [&](int i) -> int {
                const int pos = i * kTile + 8 * (lane & 15);
                return i < p.t1 && pos < p.n ? __ldg(table + (pos >> A.pshift)) : -1;
            };
            int blk = fetch_id(p.t0);
            for (int i = p.t0; i < p.t1; ++i, ++it) {
                const int pos = i * kTile + 8 * (lane & 15);
                const bool good = blk >= 0 && blk < A.num_blocks;
                if (rank == 0 && !good && pos < p.n) atomicOr(A.status, TQ_DEVERR_BLOCK_RANGE);
                const uint32_t valid = __ballot_sync(0xffffffffu, good || pos >= p.n) & 0xffffu;
                const int y = good ? (blk << A.pshift) + (pos & (A.P - 1)) : nowhere;
                int row[8];
#pragma unroll
                for (int g = 0; g < 8; ++g) row[g] = __shfl_sync(0xffffffffu, y, 8 * static_cast<int>(rank) + g);
                const uint32_t st = sbase + C::kKOff + (it % NS) * C::kStage;
                const uint32_t full = k_full + 8 * NG * (it % NS);
#pragma unroll
                for (int x = 0; x < NG; ++x) {
                    if (it >= NS && (x == 0 || x == C::kHalfGroups) && !(ok = wait_bar((x < C::kHalfGroups ? C::bPvHalf : C::bPvDone) + it % NS, (it / NS - 1) & 1))) break;
                    if (umma::elect_one()) {
                        if (x == 0) okmask[it & 7] = valid;
                        umma::cluster_arrive_expect(full + 8 * x, 8 * 1024 * C::GB);
#pragma unroll
                        for (int g = 0; g < 8; ++g)
                            asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                                         ::"r"(st + g * C::kOct + x * (C::GB * 1024)), "l"(reinterpret_cast<uint64_t>(&tmK)), "r"(0), "r"(row[g]), "r"(C::GB * x), "r"(full + 8 * x)
                                         : "memory");
                        misc[2] = it * NG + x + 1;
                    }
                    __syncwarp();
                }
                if (!ok) break;
                blk = fetch_id(i + 1);
                if (far) prefetch_rows<C::D>(A, (i + NS) * kTile + 8 * (lane & 15), fetch_id(i + NS), lane < 16 && lane >> 3 == static_cast<int>(rank));
            }
        }
    } else {
        // ================= loads: Q, and the other CTA's tokens of the own coordinates =================
        const int nowhere = static_cast<int>(A.num_blocks) << A.pshift;
        const int other = 1 - static_cast<int>(rank);
        const uint32_t q_full = leader(C::bQFull);
        int it = 0, issued = 0;
        bool ok = true;
        Piece p;
        while (ok && share.next(A, p)) {
            if (p.tiles == 0) continue;
            // Q: the scores of the piece before are done, this warp has waited for the last of them
            const int first = p.rt * kTile + static_cast<int>(rank) * kHalf;
            const int qy = first < A.R ? p.b * A.R + first : A.B * A.R;
            if (umma::elect_one()) {
                umma::cluster_arrive_expect(q_full, NBLK * C::kBlk);
                asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                             ::"r"(sbase + C::kQOff), "l"(reinterpret_cast<uint64_t>(&tmQ)), "r"(0), "r"(qy), "r"(0), "r"(q_full)
                             : "memory");
                misc[4] = misc[4] + 1;
            }
            __syncwarp();
            const int32_t *table = A.block_table + static_cast<int64_t>(p.b) * A.max_blocks;
            auto fetch_row = [&](int i) -> int {  // lane: tokens 8 (lane % 8) .. of the other half
                const int pos = i * kTile + other * kHalf + 8 * (lane & 7);
                const int blk = pos < p.n ? __ldg(table + (pos >> A.pshift)) : -1;
                return blk >= 0 && blk < A.num_blocks ? (blk << A.pshift) + (pos & (A.P - 1)) : nowhere;
            };
            int y = fetch_row(p.t0);
            for (int i = p.t0; i < p.t1; ++i, ++it) {
                int row[8];
#pragma unroll
                for (int g = 0; g < 8; ++g) row[g] = __shfl_sync(0xffffffffu, y, g);
                if (!(ok = wait_bar(C::bSFull + (it & 1), (it >> 1) & 1))) break;
                if (umma::elect_one()) {
                    const uint32_t full = saddr(&mbar[C::bVFull + it % NS]);
                    const uint32_t st = sbase + C::kKOff + (it % NS) * C::kStage + other * NO * 1024;
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full), "r"(NO * C::kBlk) : "memory");
#pragma unroll
                    for (int g = 0; g < 8; ++g)
                        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                                     ::"r"(st + g * C::kOct), "l"(reinterpret_cast<uint64_t>(&tmV)), "r"(0), "r"(row[g]),
                                       "r"(static_cast<int>(rank) * NO), "r"(full)
                                     : "memory");
                }
                __syncwarp();
                issued = it + 1;
                y = i + 1 < p.t1 ? fetch_row(i + 1) : 0;
            }
        }
        for (int t = max(0, issued - NS); t < issued; ++t) drain(C::bVFull + t % NS, (t / NS) & 1);
    }

    // ---- teardown: what either CTA has in flight lands before the pair ends, also when a wait gave up ----
    __syncwarp();
    if (warp >= kSoftWarps + 2 && lane == 0) {  // tell the other CTA how far this one came
        const int w = warp == kSoftWarps + 2 ? 2 : 4;
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(umma::peer_addr(sbase + C::kMiscOff + 4 * (w + 1), rank ^ 1u)), "r"(misc[w]) : "memory");
    }
    umma::fence_before_sync();
    umma::cluster_sync();
    umma::fence_after_sync();
    if (tid == 0) {
        // a barrier that only the other CTA has announced copies on gets this CTA's arrival, so that its phase ends with them
        for (int t = misc[2]; t < misc[3]; ++t) umma::cluster_arrive(leader(C::bKFull + t % (NS * NG)));
        for (int t = misc[4]; t < misc[5]; ++t) umma::cluster_arrive(leader(C::bQFull));
        if (rank == 0) {
            const int groups = max(misc[2], misc[3]), qs = max(misc[4], misc[5]);
            for (int t = max(0, groups - NS * NG); t < groups; ++t) drain(C::bKFull + t % (NS * NG), t / (NS * NG) & 1);
            if (qs > 0) drain(C::bQFull, (qs - 1) & 1);
        } else {
            // the first CTA's commits arrive here too, and none may find this CTA gone: its last ones, on these
            drain(C::bEnd, 0);
            drain(C::bEnd + 1, 0);
        }
    }
    __syncthreads();
    umma::cluster_sync();
    __syncwarp();
    if (warp == kSoftWarps) umma::tmem_dealloc_pair(tbase, 512);
    grid.barrier_wait(std::move(zeroed));
    join<DL, kTile, kThreads>(A, jobs, pair, static_cast<int>(rank), 2, plan[kThreads / 32 + 2], *reinterpret_cast<Merge *>(smem));
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }
// Pairs of CTAs, or CTAs: the pieces of either take the same room.
int pairs_of(int num_sms) { return num_sms / 2 < kMaxWorkers / 2 ? num_sms / 2 : kMaxWorkers / 2; }
static_assert(kTile == 2 * kNarrowRows, "rows of a pair's unit and of a CTA's");

size_t workspace_bytes(int dl, int pairs)
{
    const size_t rows = static_cast<size_t>(2) * pairs * kTile;
    return align256(kMaxWorkers * sizeof(int)) + align256(rows * sizeof(float2)) + rows * dl * sizeof(float);
}

template <int DL>
cudaError_t launch(const CUtensorMap &tk, const CUtensorMap &tv, const CUtensorMap &tq, const Args &a, cudaStream_t st)
{
    return launch_together(latent_kernel<DL>, 2, kThreads, Cfg<DL>::kSmem, st, a, tk, tv, tq);
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

tq_status attend(const char *who, tq_handle h, const uint16_t *q, const uint16_t *pool, const int32_t *block_table,
                 const int32_t *seq_lens, int batch, int q_tokens, int Hq, int dl, int P, int max_blocks, int64_t num_blocks,
                 float sm_scale, void *workspace, size_t ws_bytes, uint16_t *out, void *stream)
{
    if (!h) return api_error(TQ_ERR_INVALID_ARG, "%s: NULL handle", who);
    const Codec &c = handle_codec(h);
    if (dl != 256 && dl != 512) return api_error(TQ_ERR_UNSUPPORTED, "%s: latent_dim %d not in {256, 512}", who, dl);
    if (P != 16 && P != 32 && P != 64) return api_error(TQ_ERR_UNSUPPORTED, "%s: page_size %d not in {16, 32, 64}", who, P);
    if (batch < 0 || q_tokens < 1 || Hq < 1 || max_blocks < 1 || num_blocks < 1)
        return api_error(TQ_ERR_INVALID_ARG, "%s: bad sizes", who);
    if (!std::isfinite(sm_scale)) return api_error(TQ_ERR_INVALID_ARG, "%s: sm_scale not finite", who);
    if (!std::isfinite(sm_scale * kLog2e))  // scores are taken in powers of two
        return api_error(TQ_ERR_UNSUPPORTED, "%s: sm_scale out of range", who);
    if (max_blocks > (1 << 30) / P) return api_error(TQ_ERR_UNSUPPORTED, "%s: more than 2^30 positions", who);
    if (num_blocks > ((int64_t(1) << 31) - 1) / P)
        return api_error(TQ_ERR_UNSUPPORTED, "%s: pool of %lld blocks is too large", who, static_cast<long long>(num_blocks));
    const int64_t rows = static_cast<int64_t>(q_tokens) * Hq;
    const int64_t units = (rows + kTile - 1) / kTile * batch, tiles = static_cast<int64_t>(max_blocks) * P / kNarrowRows + 2;
    // counted in 32 bits: rows, units, and the tiles of one worker's share
    if (rows >= (int64_t(1) << 31) - kTile || rows * batch >= (int64_t(1) << 31) || units >= (int64_t(1) << 30) ||
        units * tiles / (c.num_sms > 2 ? c.num_sms / 2 : 1) >= (int64_t(1) << 30))
        return api_error(TQ_ERR_UNSUPPORTED, "%s: too many sequences x query tokens in one call", who);
    if (batch == 0) return TQ_OK;
    if (!q || !pool || !block_table || !seq_lens || !out) return api_error(TQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (!aligned(q, 16) || !aligned(pool, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(workspace, 256) ||
        !aligned(out, 16))
        return api_error(TQ_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    Args a{};
    const int pairs = pairs_of(c.num_sms);
    if (pairs < 1) return api_error(TQ_ERR_UNSUPPORTED, "%s: no pair of SMs", who);
    const bool narrow = rows <= kNarrowRows;
    a.workers = narrow ? 2 * pairs : pairs;
    a.least_workers = static_cast<int>(units * (tiles + kUnitCost) / (3 << 29)) + 1;
    const size_t need = workspace_bytes(dl, pairs);
    if (ws_bytes < need || !workspace)
        return api_error(TQ_ERR_INVALID_ARG, "%s: workspace %zu bytes < %zu needed", who, workspace ? ws_bytes : 0, need);
    // the runtime keeps an error until it is asked for: left there, the library's next launch would report it as its own
    auto failed = [who](const char *what, cudaError_t e) -> tq_status {
        cudaGetLastError();
        return api_error(TQ_ERR_CUDA, "%s: %s: %s", who, what, cudaGetErrorString(e));
    };
    CUtensorMap tk, tv, tq;
    cudaError_t e = cudaSuccess;
    const int d = dl + kRope;
    const int group = narrow ? narrow_group(dl) : dl == 512 ? Cfg<512>::GB : Cfg<256>::GB;
    if (!encode_row_blocks_map(&tk, pool, d, num_blocks * P, 8, group, &e) ||
        (!narrow && !encode_row_blocks_map(&tv, pool, d, num_blocks * P, 8, dl / 128, &e)) ||
        !encode_row_blocks_map(&tq, q, d, rows * batch, kHalf, d / 64, &e))
        return failed("cuTensorMapEncodeTiled", e);
    a.pool = pool;
    a.block_table = block_table;
    a.seq_lens = seq_lens;
    a.B = batch;
    a.Tq = q_tokens;
    a.Hq = Hq;
    a.R = static_cast<int>(rows);
    a.RT = narrow ? 1 : static_cast<int>((rows + kTile - 1) / kTile);
    a.P = P;
    a.pshift = P == 16 ? 4 : P == 32 ? 5 : 6;
    a.max_blocks = max_blocks;
    a.few = (narrow ? batch : units) <= 32 && units * tiles < (1 << 23);
    a.num_blocks = num_blocks;
    a.sm_scale = sm_scale;
    a.done = static_cast<int *>(workspace);
    a.ml = reinterpret_cast<float2 *>(static_cast<char *>(workspace) + align256(kMaxWorkers * sizeof(int)));
    a.acc = reinterpret_cast<float *>(reinterpret_cast<char *>(a.ml) + align256(static_cast<size_t>(2) * pairs * kTile * sizeof(float2)));
    a.out = out;
    a.status = c.status;
    a.wait_limit = c.wait_limit;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (narrow) e = launch_narrow(tk, tq, dl, a, st);
    else e = dl == 512 ? launch<512>(tk, tv, tq, a, st) : launch<256>(tk, tv, tq, a, st);
    if (e != cudaSuccess) return failed("launch", e);
    return TQ_OK;
}

}  // namespace
}  // namespace latent
}  // namespace tq

extern "C" size_t tq_workspace_bytes_latent(tq_handle h, int batch, int q_tokens, int num_q_heads, int latent_dim)
{
    if (!h || batch < 1 || q_tokens < 1 || num_q_heads < 1 || (latent_dim != 256 && latent_dim != 512)) return 0;
    return tq::latent::workspace_bytes(latent_dim, tq::latent::pairs_of(tq::handle_codec(h).num_sms));
}

extern "C" tq_status tq_decode_attention_latent(tq_handle h, const uint16_t *q, const uint16_t *pool, const int32_t *block_table,
                                                const int32_t *seq_lens, int batch, int num_q_heads, int latent_dim,
                                                int page_size, int max_blocks_per_seq, int64_t num_blocks, float sm_scale,
                                                void *workspace, size_t ws_bytes, uint16_t *out, void *stream)
{
    return tq::latent::attend("tq_decode_attention_latent", h, q, pool, block_table, seq_lens, batch, 1, num_q_heads, latent_dim,
                              page_size, max_blocks_per_seq, num_blocks, sm_scale, workspace, ws_bytes, out, stream);
}

extern "C" tq_status tq_prefill_attention_latent(tq_handle h, const uint16_t *q, const uint16_t *pool, const int32_t *block_table,
                                                 const int32_t *seq_lens, int batch, int q_tokens, int num_q_heads,
                                                 int latent_dim, int page_size, int max_blocks_per_seq, int64_t num_blocks,
                                                 float sm_scale, void *workspace, size_t ws_bytes, uint16_t *out, void *stream)
{
    return tq::latent::attend("tq_prefill_attention_latent", h, q, pool, block_table, seq_lens, batch, q_tokens, num_q_heads,
                              latent_dim, page_size, max_blocks_per_seq, num_blocks, sm_scale, workspace, ws_bytes, out, stream);
}
