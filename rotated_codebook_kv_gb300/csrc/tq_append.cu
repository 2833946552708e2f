// tq_append.cu -- appending rotated keys and values to plain bf16 pages or to e4m3
// pages with one scale per (page, kv head).
//
// The rotation by position turns the coordinate pair (x, y) by the angle whose cosine
// c and sine s stand in the token's row of the rope table: x' = x c - y s,
// y' = y c + x s, every product and sum rounded once in fp32 (no fused multiply-add),
// so that a page's scale does not depend on how the products are contracted.
//
// Work is cut into units of 16 coordinates of one row (32 bytes of bf16): a rotated
// unit i is the eight pairs 8 i .. 8 i + 7 (two 16-byte chunks, rot_dim / 2 apart or
// adjacent by the style), the others are 16 coordinates that pass through.
#include <cmath>
#include <cuda_runtime.h>

#include "tq.h"
#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace {

constexpr int kUnit = 16;        // coordinates of a unit
constexpr int kThreads = 256;
constexpr int kWindow = 32;      // tokens looked back and ahead of a run's first token
constexpr int kMinExp = -100;    // least exponent of a page's scale

struct AppendArgs {
    const uint16_t *q, *k, *v;
    int64_t T;
    int Hq, Hkv;
    int64_t qs, ks, vs;            // token strides, elements
    const int64_t *positions;
    const float *rope;
    int64_t rope_rows;
    int r, interleaved;            // rot_dim, style
    const int64_t *slots;
    int P, pshift;                 // page size, its logarithm
    int64_t num_slots;             // num_blocks * P
    uint16_t *q_out;
    void *k_pool, *v_pool;
    float *k_scales, *v_scales;
    unsigned *status;
};

// First coordinates of a unit's two 8-wide chunks.
__device__ __forceinline__ void unit_chunks(int u, int r, int interleaved, int &j0, int &j1)
{
    const bool pair = u < r / kUnit;
    j0 = (pair && !interleaved) ? 8 * u : kUnit * u;
    j1 = (pair && !interleaved) ? r / 2 + 8 * u : kUnit * u + 8;
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
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        v[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

struct Turn {
    float c[8], s[8];
};

// The eight (cosine, sine) of a rotated unit.
__device__ __forceinline__ Turn load_turn(const float *__restrict__ row, int u, int r)
{
    Turn t;
    const float4 *c = reinterpret_cast<const float4 *>(row + 8 * u);
    const float4 *s = reinterpret_cast<const float4 *>(row + r / 2 + 8 * u);
    *reinterpret_cast<float4 *>(t.c) = __ldg(c);
    *reinterpret_cast<float4 *>(t.c + 4) = __ldg(c + 1);
    *reinterpret_cast<float4 *>(t.s) = __ldg(s);
    *reinterpret_cast<float4 *>(t.s + 4) = __ldg(s + 1);
    return t;
}

__device__ __forceinline__ void turn_pair(float &x, float &y, float c, float s)
{
    const float a = x, b = y;
    x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
    y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// Rotates the unit's two chunks.
__device__ __forceinline__ void turn_unit(float (&a)[8], float (&b)[8], const Turn &t, int interleaved)
{
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            turn_pair(a[2 * i], a[2 * i + 1], t.c[i], t.s[i]);
            turn_pair(b[2 * i], b[2 * i + 1], t.c[4 + i], t.s[4 + i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) turn_pair(a[i], b[i], t.c[i], t.s[i]);
    }
}

// Whether token t is written: its slot lies in the pool and its position in the table.
// One caller per token reports what is wrong.
__device__ __forceinline__ bool token_ok(const AppendArgs &A, int64_t t, int64_t slot, int64_t &pos, bool report)
{
    pos = 0;
    if (slot < 0) return false;
    if (slot >= A.num_slots) {
        if (report) atomicOr(A.status, TQ_DEVERR_SLOT_RANGE);
        return false;
    }
    if (A.r) {
        pos = __ldg(A.positions + t);
        if (pos < 0 || pos >= A.rope_rows) {
            if (report) atomicOr(A.status, TQ_DEVERR_POSITION);
            return false;
        }
    }
    return true;
}

// Rows row0, row0 + step, ... of one token: the Hq query rows and, with KV, the key and
// value rows, into q_out and the bf16 pools.  A thread keeps one unit of every row it takes, so
// the token's cosines and sines are loaded once.
template <int D, bool KV>
__device__ __forceinline__ void token_rows(const AppendArgs &A, int64_t t, int row0, int step, int u)
{
    const int64_t slot = __ldg(A.slots + t);
    int64_t pos;
    if (!token_ok(A, t, slot, pos, row0 == 0 && u == 0)) return;
    const bool pair = u < A.r / kUnit;
    int j0, j1;
    unit_chunks(u, A.r, A.interleaved, j0, j1);
    Turn tn{};
    if (pair) tn = load_turn(A.rope + pos * A.r, u, A.r);
    const int rows = A.Hq + (KV ? 2 * A.Hkv : 0);
    const int64_t blk = slot >> A.pshift;
    const int o = static_cast<int>(slot & (A.P - 1));
    auto source = [&](int row) -> const uint16_t * {
        if (row < A.Hq) return A.q + t * A.qs + static_cast<int64_t>(row) * D;
        if (row < A.Hq + A.Hkv) return A.k + t * A.ks + static_cast<int64_t>(row - A.Hq) * D;
        return A.v + t * A.vs + static_cast<int64_t>(row - A.Hq - A.Hkv) * D;
    };
    auto finish = [&](int row, uint4 wa, uint4 wb) {
        uint16_t *dst;
        bool turn = pair;
        if (row < A.Hq) {
            dst = A.q_out + (t * A.Hq + row) * D;
        } else {
            const int hk = row - A.Hq;
            const bool val = hk >= A.Hkv;
            uint16_t *pool = static_cast<uint16_t *>(val ? A.v_pool : A.k_pool);
            dst = pool + ((blk * A.Hkv + (val ? hk - A.Hkv : hk)) * A.P + o) * D;
            turn = pair && !val;
        }
        if (turn) {
            float a[8], b[8];
            unpack8(wa, a);
            unpack8(wb, b);
            turn_unit(a, b, tn, A.interleaved);
            wa = pack8(a);
            wb = pack8(b);
        }
        *reinterpret_cast<uint4 *>(dst + j0) = wa;
        *reinterpret_cast<uint4 *>(dst + j1) = wb;
    };
    for (int row = row0; row < rows; row += 2 * step) {
        const bool two = row + step < rows;
        const uint16_t *s0 = source(row), *s1 = source(two ? row + step : row);
        const uint4 a0 = ld_pinned(s0 + j0), b0 = ld_pinned(s0 + j1);
        uint4 a1{}, b1{};
        if (two) {
            a1 = ld_pinned(s1 + j0);
            b1 = ld_pinned(s1 + j1);
        }
        finish(row, a0, b0);
        if (two) finish(row + step, a1, b1);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_bf16_kernel(const AppendArgs A)
{
    constexpr int U = D / kUnit;           // units of a row
    constexpr int RL = kThreads / U;       // rows in flight
    const int u = threadIdx.x % U, rl = threadIdx.x / U;
    token_rows<D, true>(A, blockIdx.x, blockIdx.y * RL + rl, RL * gridDim.y, u);
}

__device__ __forceinline__ float pow2_scale(float amax)
{
    // least e with amax <= 448 2^e = 1.75 2^(e + 8)
    const uint32_t b = __float_as_uint(amax);
    int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (e < kMinExp) e = kMinExp;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Two values to e4m3, nearest even, saturating (a NaN stays one): x in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float x, float y)
{
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(y), "f"(x));
    return h;
}

__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv)
{
    const uint32_t a = e4m3x2(x[0] * inv, x[1] * inv) | (e4m3x2(x[2] * inv, x[3] * inv) << 16);
    const uint32_t b = e4m3x2(x[4] * inv, x[5] * inv) | (e4m3x2(x[6] * inv, x[7] * inv) << 16);
    return make_uint2(a, b);
}

__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio)
{
    uint32_t out = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h2;
        const uint16_t c = static_cast<uint16_t>(w >> (16 * i));
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
        out |= e4m3x2(f.x * ratio, f.y * ratio) << (16 * i);
    }
    return out;
}

__device__ __forceinline__ float finite_abs(float x)
{
    const float a = fabsf(x);
    return a <= 3.402823466e38f ? a : 0.f;
}

// Query rows of a token (blocks below q_blocks), then the pages: a block takes the
// runs (consecutive tokens on consecutive slots of one page) that begin among its
// `chunk` tokens, threads 0-127 their keys, 128-255 their values.
template <int D, int UP>
__global__ void __launch_bounds__(kThreads) append_fp8_kernel(const AppendArgs A, const int q_blocks, const int chunk)
{
    constexpr int U = D / kUnit;
    if (blockIdx.x < q_blocks) {
        constexpr int RL = kThreads / U;
        const int per = gridDim.y;
        token_rows<D, false>(A, blockIdx.x, blockIdx.y * RL + threadIdx.x / U, RL * per, threadIdx.x % U);
        return;
    }
    constexpr int kHalf = kThreads / 2;
    constexpr int kMaxChunk = 16;
    __shared__ int64_t win[kWindow + kMaxChunk + kWindow];
    __shared__ float red[kThreads / 32];
    __shared__ int s_len[kMaxChunk];
    const int tid = threadIdx.x;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x - q_blocks) * chunk;
    const int P = A.P;
    for (int i = tid; i < 2 * kWindow + chunk; i += kThreads) {
        const int64_t t = t0 - kWindow + i;
        int64_t s = (t >= 0 && t < A.T) ? __ldg(A.slots + t) : -1;
        if (s >= A.num_slots) {
            if (i >= kWindow && i < kWindow + chunk && blockIdx.y == 0) atomicOr(A.status, TQ_DEVERR_SLOT_RANGE);
            s = -1;
        }
        win[i] = s;
    }
    __syncthreads();
    if (tid < chunk) {  // length of the run that begins at this token, 0 where none does
        const int64_t *w = win + kWindow + tid;
        const int64_t s = w[0];
        int len = 0;
        if (s >= 0 && !((s & (P - 1)) != 0 && w[-1] == s - 1)) {
            const int64_t page = s >> A.pshift;
            bool clash = false;
            for (int i = 1; i <= kWindow; ++i) clash |= w[-i] >= 0 && (w[-i] >> A.pshift) == page;
            if (clash) {
                if (blockIdx.y == 0) atomicOr(A.status, TQ_DEVERR_SLOT_ORDER);
            } else {
                const int most = P - static_cast<int>(s & (P - 1));
                len = 1;
                while (len < most && w[len] == s + len) ++len;
            }
        }
        s_len[tid] = len;
    }
    __syncthreads();
    const bool val = tid >= kHalf;
    const int ht = tid & (kHalf - 1);
    const uint16_t *src = val ? A.v : A.k;
    const int64_t stride = val ? A.vs : A.ks;
    unsigned char *pool = static_cast<unsigned char *>(val ? A.v_pool : A.k_pool);
    float *scales = val ? A.v_scales : A.k_scales;
    for (int c = 0; c < chunk; ++c) {
        const int len = s_len[c];
        if (len == 0) continue;
        const int64_t t = t0 + c, slot = win[kWindow + c], page = slot >> A.pshift;
        const int o = static_cast<int>(slot & (P - 1));
        for (int h = blockIdx.y; h < A.Hkv; h += gridDim.y) {
            const int64_t rec = page * A.Hkv + h;
            const float old = o > 0 ? scales[rec] : 0.f;
            uint4 wa[UP], wb[UP];
            bool live[UP];
            int64_t pos[UP];
#pragma unroll
            for (int i = 0; i < UP; ++i) {
                const int e = ht + i * kHalf, row = e / U, u = e % U;
                pos[i] = 0;
                live[i] = row < len;
                if (live[i] && A.r) {
                    pos[i] = __ldg(A.positions + t + row);
                    if (pos[i] < 0 || pos[i] >= A.rope_rows) {
                        if (u == 0 && h == 0 && !val) atomicOr(A.status, TQ_DEVERR_POSITION);
                        live[i] = false;
                    }
                }
                if (live[i]) {
                    int j0, j1;
                    unit_chunks(u, A.r, A.interleaved, j0, j1);
                    const uint16_t *p = src + (t + row) * stride + static_cast<int64_t>(h) * D;
                    wa[i] = ld_pinned(p + j0);
                    wb[i] = ld_pinned(p + j1);
                }
            }
            float a[UP][8], b[UP][8];
            float amax = 0.f;
#pragma unroll
            for (int i = 0; i < UP; ++i) {
                if (!live[i]) continue;
                const int u = (ht + i * kHalf) % U;
                unpack8(wa[i], a[i]);
                unpack8(wb[i], b[i]);
                if (!val && u < A.r / kUnit)
                    turn_unit(a[i], b[i], load_turn(A.rope + pos[i] * A.r, u, A.r), A.interleaved);
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fmaxf(finite_abs(a[i][j]), finite_abs(b[i][j])));
            }
            amax = warp_max(amax);
            __syncthreads();  // the last pass's readers of `red` are done
            if ((tid & 31) == 0) red[tid >> 5] = amax;
            __syncthreads();
            const float *rw = red + (val ? kHalf / 32 : 0);
            amax = fmaxf(fmaxf(rw[0], rw[1]), fmaxf(rw[2], rw[3]));
            const float need = pow2_scale(amax);
            const bool keep = o > 0 && old > 0.f && old <= 3.402823466e38f;  // the page's rows and scale so far
            const float scale = keep ? fmaxf(old, need) : need;
            const float inv = 1.f / scale;
            unsigned char *base = pool + rec * P * D;
            if (keep && scale > old) {  // code the earlier rows anew
                const float ratio = old * inv;
                for (int e = ht; e < o * (D / 16); e += kHalf) {
                    uint4 *p = reinterpret_cast<uint4 *>(base) + e;
                    const uint4 w = *p;
                    *p = make_uint4(recode4(w.x, ratio), recode4(w.y, ratio), recode4(w.z, ratio), recode4(w.w, ratio));
                }
            }
#pragma unroll
            for (int i = 0; i < UP; ++i) {
                if (!live[i]) continue;
                const int e = ht + i * kHalf, row = e / U, u = e % U;
                int j0, j1;
                unit_chunks(u, A.r, A.interleaved, j0, j1);
                unsigned char *p = base + static_cast<int64_t>(o + row) * D;
                *reinterpret_cast<uint2 *>(p + j0) = codes8(a[i], inv);
                *reinterpret_cast<uint2 *>(p + j1) = codes8(b[i], inv);
            }
            if (ht == 0 && !(keep && scale == old)) scales[rec] = scale;
        }
    }
}

template <int D>
cudaError_t launch_bf16(const AppendArgs &a, cudaStream_t st)
{
    constexpr int RL = kThreads / (D / kUnit);
    const int rows = a.Hq + 2 * a.Hkv;
    // few tokens: a block per RL rows, for latency; many: the rows of a token in one block
    const unsigned gy = a.T < 1024 ? static_cast<unsigned>((rows + RL - 1) / RL) : 1u;
    append_bf16_kernel<D><<<dim3(static_cast<unsigned>(a.T), gy), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch_fp8(const AppendArgs &a, cudaStream_t st)
{
    // few tokens: every token may begin a page's run, so a block each; many: 16 tokens,
    // among which about one run begins
    const int chunk = a.T < 1024 ? 1 : 16;
    const int q_blocks = a.Hq ? static_cast<int>(a.T) : 0;
    const unsigned gy = static_cast<unsigned>(a.Hkv < 65535 ? a.Hkv : 65535);
    const dim3 grid(static_cast<unsigned>(q_blocks + (a.T + chunk - 1) / chunk), gy);
    if (a.P == 16) append_fp8_kernel<D, 16 * (D / kUnit) / (kThreads / 2)><<<grid, kThreads, 0, st>>>(a, q_blocks, chunk);
    else append_fp8_kernel<D, 32 * (D / kUnit) / (kThreads / 2)><<<grid, kThreads, 0, st>>>(a, q_blocks, chunk);
    return cudaGetLastError();
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// The checks that both entry points share; *run is false where there is nothing to do.
tq_status check(const char *who, tq_handle h, AppendArgs *a, int64_t num_blocks, int style, size_t cell, bool *run)
{
    *run = false;
    if (!h) return api_error(TQ_ERR_INVALID_ARG, "%s: NULL handle", who);
    const Codec &c = handle_codec(h);
    const int d = c.d;
    if (a->P != 16 && a->P != 32) return api_error(TQ_ERR_UNSUPPORTED, "%s: page_size %d not in {16, 32}", who, a->P);
    if (!a->q) a->Hq = 0;
    if (a->T < 0 || a->Hkv < 1 || num_blocks < 1 || (a->q && a->Hq < 1))
        return api_error(TQ_ERR_INVALID_ARG, "%s: T=%lld num_q_heads=%d num_kv_heads=%d num_blocks=%lld", who,
                         static_cast<long long>(a->T), a->Hq, a->Hkv, static_cast<long long>(num_blocks));
    if (a->r < 0 || a->r > d || a->r % kUnit)
        return api_error(TQ_ERR_UNSUPPORTED, "%s: rot_dim %d is not a multiple of 16 in 0..%d", who, a->r, d);
    if (style != TQ_ROPE_HALF && style != TQ_ROPE_INTERLEAVED)
        return api_error(TQ_ERR_UNSUPPORTED, "%s: unknown rotation style %d", who, style);
    if ((a->q == nullptr) != (a->q_out == nullptr))
        return api_error(TQ_ERR_INVALID_ARG, "%s: q and q_out go together", who);
    if (a->Hq > (1 << 20) || a->Hkv > (1 << 20))
        return api_error(TQ_ERR_UNSUPPORTED, "%s: more than 2^20 heads", who);
    // grid size, and byte offsets within a pool
    if (a->T >= (int64_t(1) << 30)) return api_error(TQ_ERR_UNSUPPORTED, "%s: too many tokens in one call", who);
    if (num_blocks > (int64_t(1) << 50) / (static_cast<int64_t>(a->Hkv) * a->P * d * static_cast<int64_t>(cell)))
        return api_error(TQ_ERR_UNSUPPORTED, "%s: pool of %lld blocks is too large", who,
                         static_cast<long long>(num_blocks));
    if (a->T == 0) return TQ_OK;
    if (!a->k || !a->v || !a->slots || !a->k_pool || !a->v_pool || (a->r && (!a->rope || !a->positions)))
        return api_error(TQ_ERR_INVALID_ARG, "%s: NULL pointer", who);
    if (a->r && a->rope_rows < 1) return api_error(TQ_ERR_INVALID_ARG, "%s: empty rope table", who);
    if (!aligned(a->q, 16) || !aligned(a->k, 16) || !aligned(a->v, 16) || !aligned(a->k_pool, 16) ||
        !aligned(a->v_pool, 16) || !aligned(a->q_out, 16) || !aligned(a->rope, 16) || !aligned(a->slots, 8) ||
        !aligned(a->positions, 8))
        return api_error(TQ_ERR_INVALID_ARG, "%s: misaligned pointer", who);
    const int64_t kv = static_cast<int64_t>(a->Hkv) * d;
    if (a->ks < kv || a->vs < kv || a->ks % 8 || a->vs % 8 ||
        (a->q && (a->qs < static_cast<int64_t>(a->Hq) * d || a->qs % 8)))
        return api_error(TQ_ERR_INVALID_ARG, "%s: token strides must be >= heads*head_dim and multiples of 8 elements",
                         who);
    a->interleaved = style == TQ_ROPE_INTERLEAVED;
    a->pshift = a->P == 16 ? 4 : 5;
    a->num_slots = num_blocks * a->P;
    a->status = c.status;
    *run = true;
    return TQ_OK;
}

}  // namespace
}  // namespace tq

extern "C" tq_status tq_append_kv_bf16(tq_handle h, const uint16_t *q, const uint16_t *k, const uint16_t *v, int64_t T,
                                       int num_q_heads, int num_kv_heads, int64_t q_stride_tok, int64_t k_stride_tok,
                                       int64_t v_stride_tok, const int64_t *positions, const float *rope,
                                       int64_t rope_rows, int rot_dim, int style, const int64_t *slot_mapping,
                                       uint16_t *k_pool, uint16_t *v_pool, int page_size, int64_t num_blocks,
                                       uint16_t *q_out, void *stream)
{
    tq::AppendArgs a{q, k, v, T, num_q_heads, num_kv_heads, q_stride_tok, k_stride_tok, v_stride_tok, positions, rope,
                     rope_rows, rot_dim, 0, slot_mapping, page_size, 0, 0, q_out, k_pool, v_pool, nullptr, nullptr,
                     nullptr};
    bool run;
    const tq_status s = tq::check("tq_append_kv_bf16", h, &a, num_blocks, style, 2, &run);
    if (s != TQ_OK || !run) return s;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = tq::handle_codec(h).d == 128 ? tq::launch_bf16<128>(a, st) : tq::launch_bf16<256>(a, st);
    if (e != cudaSuccess) return tq::api_error(TQ_ERR_CUDA, "tq_append_kv_bf16: launch: %s", cudaGetErrorString(e));
    return TQ_OK;
}

extern "C" tq_status tq_append_kv_fp8(tq_handle h, const uint16_t *q, const uint16_t *k, const uint16_t *v, int64_t T,
                                      int num_q_heads, int num_kv_heads, int64_t q_stride_tok, int64_t k_stride_tok,
                                      int64_t v_stride_tok, const int64_t *positions, const float *rope,
                                      int64_t rope_rows, int rot_dim, int style, const int64_t *slot_mapping,
                                      uint8_t *k_pool, uint8_t *v_pool, float *k_scales, float *v_scales,
                                      int page_size, int64_t num_blocks, uint16_t *q_out, void *stream)
{
    tq::AppendArgs a{q, k, v, T, num_q_heads, num_kv_heads, q_stride_tok, k_stride_tok, v_stride_tok, positions, rope,
                     rope_rows, rot_dim, 0, slot_mapping, page_size, 0, 0, q_out, k_pool, v_pool, k_scales, v_scales,
                     nullptr};
    bool run;
    const tq_status s = tq::check("tq_append_kv_fp8", h, &a, num_blocks, style, 1, &run);
    if (s != TQ_OK || !run) return s;
    if (!k_scales || !v_scales) return tq::api_error(TQ_ERR_INVALID_ARG, "tq_append_kv_fp8: NULL pointer");
    if (!tq::aligned(k_scales, 4) || !tq::aligned(v_scales, 4))
        return tq::api_error(TQ_ERR_INVALID_ARG, "tq_append_kv_fp8: misaligned pointer");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = tq::handle_codec(h).d == 128 ? tq::launch_fp8<128>(a, st) : tq::launch_fp8<256>(a, st);
    if (e != cudaSuccess) return tq::api_error(TQ_ERR_CUDA, "tq_append_kv_fp8: launch: %s", cudaGetErrorString(e));
    return TQ_OK;
}
