// tq_append_latent.cu -- appending tokens to latent pages: a token's latent vector, normalised where a weight is given,
// and its rotated key part side by side in one row; the query heads' parts rotated on the way.
//
//   c' = c w / sqrt(mean(c^2) + eps), sums and products in fp32, rounded once
//   (x, y) -> (x cos - y sin, y cos + x sin), every product and sum rounded once in fp32
//
// Bound: HBM, in one pass.  Blocks for the pool rows (a warp each), then blocks for the query heads; everything that does not
// depend on a token's slot and position is loaded with them.  Measured (a call in a graph): 8192 tokens of 128 heads, DL = 512:
// 53 us, 5.5 TB/s (80% of the measured copy rate; a block a token, its row first: 66); 4,687 ragged tokens of 20 heads at
// DL = 256: 8.9 us; 8 tokens of 64 heads: 2.7 us, which is the launch and three latencies (slot, cosines, store).
#include <cmath>
#include <cuda_runtime.h>

#include "tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kRope = TQ_LATENT_ROPE_DIM;
constexpr int kUnits = kRope / 16;      // units of eight pairs in a row
constexpr int kThreads = 256;
constexpr int kLanes = kThreads / kUnits;  // heads side by side

struct LatentArgs {
    const uint16_t *latent, *k, *q;
    int64_t T;
    int Hq;
    int64_t ls, ks, qs, qh, os, oh;  // strides in elements: tokens, and heads of q and q_out
    const uint16_t *weight;
    float eps;
    const int64_t *positions;
    const float *rope;
    int64_t rope_rows;
    int interleaved;
    const int64_t *slots;
    int64_t num_slots;
    uint16_t *pool, *q_out;
    unsigned *status;
    bool small;  // (token, four heads) are counted in 32 bits
};

__device__ __forceinline__ uint4 ld_row(const void *p)  // plain: q may be rewritten in place
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void unpack8(const uint4 &w, float (&x)[8])
{
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(v[i] << 16);
        x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8])
{
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(v[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// A unit's cosines and sines, and the turn of its two chunks of eight coordinates.
struct Turn {
    float c[8], s[8];
    __device__ __forceinline__ void load(const float *row, int u)
    {
        const float4 *pc = reinterpret_cast<const float4 *>(row + 8 * u), *ps = reinterpret_cast<const float4 *>(row + kRope / 2 + 8 * u);
        *reinterpret_cast<float4 *>(c) = __ldg(pc);
        *reinterpret_cast<float4 *>(c + 4) = __ldg(pc + 1);
        *reinterpret_cast<float4 *>(s) = __ldg(ps);
        *reinterpret_cast<float4 *>(s + 4) = __ldg(ps + 1);
    }
    static __device__ __forceinline__ void pair(float &x, float &y, float c, float s)
    {
        const float a = x, b = y;
        x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
    }
    __device__ __forceinline__ void turn(uint4 &wa, uint4 &wb, int interleaved) const
    {
        float a[8], b[8];
        unpack8(wa, a);
        unpack8(wb, b);
        if (interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                pair(a[2 * i], a[2 * i + 1], c[i], s[i]);
                pair(b[2 * i], b[2 * i + 1], c[4 + i], s[4 + i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) pair(a[i], b[i], c[i], s[i]);
        }
        wa = pack8(a);
        wb = pack8(b);
    }
};

// Whether a token is written: its slot lies in the pool and its position in the table.
__device__ __forceinline__ bool token_ok(const LatentArgs &A, int64_t slot, int64_t pos, bool report)
{
    if (slot < 0) return false;
    if (slot >= A.num_slots) {
        if (report) atomicOr(A.status, TQ_DEVERR_SLOT_RANGE);
        return false;
    }
    if (A.rope && (pos < 0 || pos >= A.rope_rows)) {
        if (report) atomicOr(A.status, TQ_DEVERR_POSITION);
        return false;
    }
    return true;
}

// A warp's pool row: DL / 32 coordinates of the latent a lane, in registers between the sum and the scaling.
template <int DL>
__device__ __forceinline__ void pool_row(const LatentArgs &A, int64_t t, int lane)
{
    constexpr int N = DL / 256;  // chunks of eight coordinates a lane
    const int u = lane % kUnits;
    const int j0 = A.interleaved ? 16 * u : 8 * u, j1 = A.interleaved ? 16 * u + 8 : kRope / 2 + 8 * u;
    uint4 w[N], g[N], ka, kb;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        w[i] = ld_row(A.latent + t * A.ls + 8 * (lane + 32 * i));
        if (A.weight) g[i] = ld_pinned(A.weight + 8 * (lane + 32 * i));
    }
    if (lane < kUnits) {
        ka = ld_row(A.k + t * A.ks + j0);
        kb = ld_row(A.k + t * A.ks + j1);
    }
    const int64_t slot = ld_pinned_s64(A.slots + t);
    const int64_t pos = A.rope ? ld_pinned_s64(A.positions + t) : 0;
    if (!token_ok(A, slot, pos, lane == 0)) return;
    Turn tn{};
    if (A.rope && lane < kUnits) tn.load(A.rope + pos * kRope, u);
    uint16_t *dst = A.pool + slot * (DL + kRope);
    if (A.weight) {
        float x[N][8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            unpack8(w[i], x[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fmaf(x[i][k], x[i][k], sum);
        }
        float total = warp_sum(sum), eps = A.eps;
        // Squares past fp32's range, or in its lowest part with no eps above them: the same with c times a power of two (all
        // lanes agree).
        const float s = !(total < INFINITY) ? 0x1p-80f : total < 0x1p-100f && eps < 0x1p-80f ? 0x1p100f : 1.f;
        if (s != 1.f) {
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    x[i][k] *= s;
                    sum = fmaf(x[i][k], x[i][k], sum);
                }
            total = warp_sum(sum);
            eps = eps * s * s;
        }
        const float inv = 1.f / sqrtf(total * (1.f / DL) + eps);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float y[8];
            unpack8(g[i], y);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] *= x[i][k] * inv;
            w[i] = pack8(y);
        }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) *reinterpret_cast<uint4 *>(dst + 8 * (lane + 32 * i)) = w[i];
    if (lane < kUnits) {
        if (A.rope) tn.turn(ka, kb, A.interleaved);
        *reinterpret_cast<uint4 *>(dst + DL + j0) = ka;
        *reinterpret_cast<uint4 *>(dst + DL + j1) = kb;
    }
}

// row_blocks blocks for the pool rows, a warp each, then blocks for the queries: thread i's unit of heads r, r + n, r + 2 n and
// r + 3 n of token i / n, r = i % n, n = ceil(Hq / 4), all of them on their way with the token's slot and position.
constexpr int kHeads = 4;
template <int DL>
__global__ void __launch_bounds__(kThreads) append_latent_kernel(const LatentArgs A, const unsigned row_blocks)
{
    const int tid = threadIdx.x;
    if (blockIdx.x < row_blocks) {
        const int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + tid / 32;
        if (t < A.T) pool_row<DL>(A, t, tid % 32);
        return;
    }
    const int n = (A.Hq + kHeads - 1) / kHeads, u = tid % kUnits;
    const int64_t i = static_cast<int64_t>(blockIdx.x - row_blocks) * kLanes + tid / kUnits;
    const int64_t t = A.small ? static_cast<uint32_t>(i) / static_cast<uint32_t>(n) : i / n;
    if (t >= A.T) return;
    const int r = static_cast<int>(i - t * n);
    const int j0 = A.interleaved ? 16 * u : 8 * u, j1 = A.interleaved ? 16 * u + 8 : kRope / 2 + 8 * u;
    const uint16_t *src = A.q + t * A.qs;
    uint4 a[kHeads], b[kHeads];
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
        if (r + k * n < A.Hq) {
            a[k] = ld_row(src + (r + k * n) * A.qh + j0);
            b[k] = ld_row(src + (r + k * n) * A.qh + j1);
        }
    const int64_t slot = ld_pinned_s64(A.slots + t);
    const int64_t pos = A.rope ? ld_pinned_s64(A.positions + t) : 0;
    if (!token_ok(A, slot, pos, false)) return;  // what is wrong is reported with the pool row
    Turn tn{};
    if (A.rope) tn.load(A.rope + pos * kRope, u);
    uint16_t *dst = A.q_out + t * A.os;
#pragma unroll
    for (int k = 0; k < kHeads; ++k)
        if (r + k * n < A.Hq) {
            if (A.rope) tn.turn(a[k], b[k], A.interleaved);
            *reinterpret_cast<uint4 *>(dst + (r + k * n) * A.oh + j0) = a[k];
            *reinterpret_cast<uint4 *>(dst + (r + k * n) * A.oh + j1) = b[k];
        }
}

template <int DL>
cudaError_t launch(const LatentArgs &a, cudaStream_t st)
{
    const int64_t rows = (a.T + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t q = a.q ? (a.T * ((a.Hq + kHeads - 1) / kHeads) + kLanes - 1) / kLanes : 0;
    append_latent_kernel<DL><<<static_cast<unsigned>(rows + q), kThreads, 0, st>>>(a, static_cast<unsigned>(rows));
    return cudaGetLastError();
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace
}  // namespace tq

extern "C" tq_status tq_append_latent(tq_handle h, const uint16_t *latent, const uint16_t *k_rope, const uint16_t *q, int64_t T,
                                      int latent_dim, int num_q_heads, int64_t latent_stride, int64_t k_stride,
                                      int64_t q_stride_tok, int64_t q_stride_head, const uint16_t *norm_weight, float norm_eps,
                                      const int64_t *positions, const float *rope, int64_t rope_rows, int style,
                                      const int64_t *slot_mapping, uint16_t *pool, int page_size, int64_t num_blocks,
                                      uint16_t *q_out, int64_t qo_stride_tok, int64_t qo_stride_head, void *stream)
{
    using tq::aligned;
    using tq::api_error;
    const char *who = "tq_append_latent";
    if (!h) return api_error(TQ_ERR_INVALID_ARG, "%s: NULL handle", who);
    if (latent_dim != 256 && latent_dim != 512)
        return api_error(TQ_ERR_UNSUPPORTED, "%s: latent_dim %d not in {256, 512}", who, latent_dim);
    if (page_size != 16 && page_size != 32 && page_size != 64)
        return api_error(TQ_ERR_UNSUPPORTED, "%s: page_size %d not in {16, 32, 64}", who, page_size);
    if (!q) num_q_heads = 0;
    if (T < 0 || num_blocks < 1 || (q && num_q_heads < 1))
        return api_error(TQ_ERR_INVALID_ARG, "%s: T=%lld num_q_heads=%d num_blocks=%lld", who, static_cast<long long>(T), num_q_heads,
                         static_cast<long long>(num_blocks));
    if (style != TQ_ROPE_HALF && style != TQ_ROPE_INTERLEAVED)
        return api_error(TQ_ERR_UNSUPPORTED, "%s: unknown rotation style %d", who, style);
    if ((q == nullptr) != (q_out == nullptr)) return api_error(TQ_ERR_INVALID_ARG, "%s: q and q_out go together", who);
    if (norm_weight && !(norm_eps >= 0.f && std::isfinite(norm_eps)))
        return api_error(TQ_ERR_INVALID_ARG, "%s: norm_eps must be finite and >= 0", who);
    if (T >= (int64_t(1) << 30) || num_q_heads > (1 << 18) || T * num_q_heads >= (int64_t(1) << 36)) return api_error(TQ_ERR_UNSUPPORTED, "%s: too many tokens or heads in one call", who);
    if (num_blocks > ((int64_t(1) << 31) - 1) / page_size)
        return api_error(TQ_ERR_UNSUPPORTED, "%s: pool of %lld blocks is too large", who, static_cast<long long>(num_blocks));
    if (T == 0) return TQ_OK;
    if (!latent || !k_rope || !slot_mapping || !pool || (rope && !positions))
        return api_error(TQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (rope && rope_rows < 1) return api_error(TQ_ERR_INVALID_ARG, "%s: empty rope table", who);
    if (!aligned(latent, 16) || !aligned(k_rope, 16) || !aligned(q, 16) || !aligned(norm_weight, 16) || !aligned(pool, 16) ||
        !aligned(q_out, 16) || !aligned(rope, 16) || !aligned(slot_mapping, 8) || !aligned(positions, 8))
        return api_error(TQ_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    const int r = TQ_LATENT_ROPE_DIM;
    const int64_t most = int64_t(1) << 40;
    auto bad = [&](int64_t s, int64_t least) { return s < least || s > most || s % 8; };
    if (bad(latent_stride, latent_dim) || bad(k_stride, r) ||
        (q && (bad(q_stride_tok, r) || bad(q_stride_head, r) || bad(qo_stride_tok, r) || bad(qo_stride_head, r))))
        return api_error(TQ_ERR_INVALID_ARG, "%s: strides must be multiples of 8 elements, no less than a row", who);
    // no offset passes 2^60 elements: T - 1 tokens of a stride up to 2^59, and fewer than 2^18 heads of a stride up to 2^40
    const int64_t widest = T > 1 ? (int64_t(1) << 59) / (T - 1) : most;
    if (latent_stride > widest || k_stride > widest || (q && (q_stride_tok > widest || qo_stride_tok > widest)))
        return api_error(TQ_ERR_UNSUPPORTED, "%s: rows too far apart", who);
    if (q && T > 1 && num_q_heads > 1 && qo_stride_tok < (num_q_heads - 1) * qo_stride_head + r && qo_stride_head < (T - 1) * qo_stride_tok + r)
        return api_error(TQ_ERR_INVALID_ARG, "%s: rows of q_out overlap", who);
    // in place: a thread rewrites what it has read itself, not what another one is still to read
    if (q && q_out == q && ((T > 1 && qo_stride_tok != q_stride_tok) || (num_q_heads > 1 && qo_stride_head != q_stride_head)))
        return api_error(TQ_ERR_INVALID_ARG, "%s: q_out is q with other strides", who);
    const tq::Codec &c = tq::handle_codec(h);
    const tq::LatentArgs a{latent, k_rope, q, T, num_q_heads, latent_stride, k_stride, q_stride_tok, q_stride_head, qo_stride_tok,
                           qo_stride_head, norm_weight, norm_eps, positions, rope, rope_rows, style == TQ_ROPE_INTERLEAVED,
                           slot_mapping, num_blocks * page_size, pool, q_out, c.status, T * num_q_heads < (int64_t(1) << 31)};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = latent_dim == 512 ? tq::launch<512>(a, st) : tq::launch<256>(a, st);
    if (e != cudaSuccess) return api_error(TQ_ERR_CUDA, "%s: launch: %s", who, cudaGetErrorString(e));
    return TQ_OK;
}
