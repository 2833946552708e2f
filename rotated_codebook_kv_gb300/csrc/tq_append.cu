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
//
// Bound: HBM, in one pass (every row is read and written once, a page's earlier rows only where its scale grows).
// Measured on a GB300 (copy 6783 GB/s): to bf16 pages 15,500 tokens of 16 query and 8 kv heads of 256 87 us = 5.8 TB/s, two
// rows of a thread in flight; to 8-bit pages 32k tokens of 32 query and 8 kv heads of 128 148 us = 5.1 TB/s, of which the
// query rows take ~90 (6.0 TB/s) and the pages ~60, bound by the latency of a chain (slots, rows, maximum, codes) and
// the instructions of the rotation and the codes.  A step's few tokens: 11 us, the host's checks and launch
// (1.7 to bf16 pages and 3.4 to 8-bit ones by graph replay).
// Tried for the pages and slower when they stood at 163: rows through shared memory by asynchronous copies (166-172 us;
// ragged chunks 53 against 45), page and query blocks in turn instead of one after the other (184; every fourth block 152,
// but ragged chunks 48).
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
    bool small;                    // query rows are counted in 32 bits
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

// Whether a token is written: its slot lies in the pool and its position in the table.
// One caller per token reports what is wrong.
__device__ __forceinline__ bool token_ok(const AppendArgs &A, int64_t slot, int64_t pos, bool report)
{
    if (slot < 0) return false;
    if (slot >= A.num_slots) {
        if (report) atomicOr(A.status, TQ_DEVERR_SLOT_RANGE);
        return false;
    }
    if (A.r && (pos < 0 || pos >= A.rope_rows)) {
        if (report) atomicOr(A.status, TQ_DEVERR_POSITION);
        return false;
    }
    return true;
}

// 16 bytes of a row that this launch may rewrite in place (a query): a plain load, pinned like ld_pinned (whose
// non-coherent path asks for memory that nobody writes meanwhile).  A thread loads what it writes before it writes it.
__device__ __forceinline__ uint4 ld_query(const void *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

// One unit of a row, rotated by tn where `turn`, to bf16.
__device__ __forceinline__ void put_unit(uint16_t *dst, int j0, int j1, uint4 wa, uint4 wb, bool turn, const Turn &tn,
                                         int interleaved)
{
    if (turn) {
        float a[8], b[8];
        unpack8(wa, a);
        unpack8(wb, b);
        turn_unit(a, b, tn, interleaved);
        wa = pack8(a);
        wb = pack8(b);
    }
    *reinterpret_cast<uint4 *>(dst + j0) = wa;
    *reinterpret_cast<uint4 *>(dst + j1) = wb;
}

// Rows row0, row0 + step, ... of one token, its query, key and value rows, into q_out and the bf16 pools.  A thread keeps
// one unit of every row it takes, so the token's cosines and sines are loaded once.
template <int D>
__device__ __forceinline__ void token_rows(const AppendArgs &A, int64_t t, int row0, int step, int u)
{
    const int64_t slot = ld_pinned_s64(A.slots + t);
    const int64_t pos = A.r ? ld_pinned_s64(A.positions + t) : 0;
    const int rows = A.Hq + 2 * A.Hkv;
    int j0, j1;
    unit_chunks(u, A.r, A.interleaved, j0, j1);
    if (!token_ok(A, slot, pos, row0 == 0 && u == 0)) return;
    const bool pair = u < A.r / kUnit;
    Turn tn{};
    if (pair) tn = load_turn(A.rope + pos * A.r, u, A.r);
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
        put_unit(dst, j0, j1, wa, wb, turn, tn, A.interleaved);
    };
    for (int row = row0; row < rows; row += 2 * step) {  // two rows on their way at a time
        const bool two = row + step < rows;
        const uint16_t *s0 = source(row), *s1 = source(two ? row + step : row);
        const uint4 a0 = ld_query(s0 + j0), b0 = ld_query(s0 + j1);
        uint4 a1{}, b1{};
        if (two) {
            a1 = ld_query(s1 + j0);
            b1 = ld_query(s1 + j1);
        }
        finish(row, a0, b0);
        if (two) finish(row + step, a1, b1);
    }
}

// The query rows alone: thread i's unit of rows r, r + n, r + 2 n and r + 3 n of token i / n, r = i % n, n = ceil(Hq / 4).
// All of them are on their way with the token's slot and position, and share its cosines and sines.
constexpr int kQueryRows = 4;
template <int D>
__device__ __forceinline__ void query_rows(const AppendArgs &A, int64_t i, int u)
{
    const int n = (A.Hq + kQueryRows - 1) / kQueryRows;
    const int64_t t = A.small ? static_cast<uint32_t>(i) / static_cast<uint32_t>(n) : i / n;
    if (t >= A.T) return;
    const int r = static_cast<int>(i - t * n);
    int j0, j1;
    unit_chunks(u, A.r, A.interleaved, j0, j1);
    const uint16_t *src = A.q + t * A.qs + static_cast<int64_t>(r) * D;
    uint4 w[kQueryRows][2];
#pragma unroll
    for (int k = 0; k < kQueryRows; ++k)
        if (r + k * n < A.Hq) {
            w[k][0] = ld_query(src + k * n * D + j0);
            w[k][1] = ld_query(src + k * n * D + j1);
        }
    const int64_t slot = ld_pinned_s64(A.slots + t);
    const int64_t pos = A.r ? ld_pinned_s64(A.positions + t) : 0;
    if (!token_ok(A, slot, pos, false)) return;  // what is wrong is reported with the pages
    Turn tn{};
    const bool pair = u < A.r / kUnit;
    if (pair) tn = load_turn(A.rope + pos * A.r, u, A.r);
    uint16_t *dst = A.q_out + (t * A.Hq + r) * D;
#pragma unroll
    for (int k = 0; k < kQueryRows; ++k)
        if (r + k * n < A.Hq) put_unit(dst + k * n * D, j0, j1, w[k][0], w[k][1], pair, tn, A.interleaved);
}

template <int D>
__global__ void __launch_bounds__(kThreads) append_bf16_kernel(const AppendArgs A)
{
    constexpr int U = D / kUnit;           // units of a row
    constexpr int RL = kThreads / U;       // rows in flight
    const int u = threadIdx.x % U, rl = threadIdx.x / U;
    token_rows<D>(A, blockIdx.x, blockIdx.y * RL + rl, RL * gridDim.y, u);
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

// kv_blocks blocks (gridDim.y of each over the heads) for the pages, then blocks for the query rows.
//
// A block finds the runs (consecutive tokens on consecutive slots of one page) that begin among its `chunk` tokens; groups
// of its warps take items (run, kv head, keys or values) in turn.  A page's scale needs its rows twice, for the maximum
// and for the codes: a group has two or four warps, so that each lane holds few units, rotated, in registers
// between; a group meets at a barrier of its own.
//
// At head dim 128 a lane holds two units, with three blocks on an SM, at 256 four with two (when chosen, 32k tokens 150 us against 163 at
// 128, and 208 against 216 at 256; chunks of 200 to 1500 tokens 83 against 91, and 132 against 111).
constexpr int units_held(int d) { return d == 128 ? 2 : 4; }
constexpr int group_warps(int d, int p) { return p * (d / kUnit) / (32 * units_held(d)); }
template <int D, int P>
__global__ void __launch_bounds__(kThreads, D == 128 ? 3 : 2)
    append_fp8_kernel(const AppendArgs A, const int kv_blocks, const int chunk)
{
    constexpr int U = D / kUnit;
    constexpr int NK = units_held(D);           // units of an item per lane: the lane's unit of rows row0, row0 + kRowStep, ...
    constexpr int W = group_warps(D, P);        // warps of a group
    constexpr int kGroups = kThreads / 32 / W;
    constexpr int kRowStep = 32 * W / U;
    if (blockIdx.x >= kv_blocks) {
        constexpr int RL = kThreads / U;
        const int64_t i = (static_cast<int64_t>(blockIdx.x - kv_blocks) * gridDim.y + blockIdx.y) * RL;
        query_rows<D>(A, i + threadIdx.x / U, threadIdx.x % U);
        return;
    }
    constexpr int kMaxChunk = 32;
    __shared__ int64_t win[kWindow + kMaxChunk + kWindow];
    __shared__ int s_at[kMaxChunk], s_len[kMaxChunk], s_runs;
    __shared__ float s_max[kGroups][2][W];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
    for (int i = tid; i < 2 * kWindow + kMaxChunk; i += kThreads) {
        const int64_t t = t0 - kWindow + i;
        int64_t s = (t >= 0 && t < A.T) ? __ldg(A.slots + t) : -1;
        if (s >= A.num_slots) {
            if (i >= kWindow && i < kWindow + chunk && blockIdx.y == 0) atomicOr(A.status, TQ_DEVERR_SLOT_RANGE);
            s = -1;
        }
        win[i] = s;
    }
    __syncthreads();
    if (warp == 0) {
        // lane i: token i of the chunk and the one 32 on; a token continues a run where its slot follows the one before
        const int64_t *w = win + kWindow + lane;
        const int64_t v = w[0], ahead = w[32];
        const bool more = v >= 0 && v == w[-1] + 1 && (v & (P - 1));
        const uint64_t cont = __ballot_sync(0xffffffffu, more) |
                              static_cast<uint64_t>(__ballot_sync(0xffffffffu, ahead >= 0 && ahead == w[31] + 1 && (ahead & (P - 1)))) << 32;
        unsigned starts = __ballot_sync(0xffffffffu, lane < chunk && v >= 0 && !more);
        const int len = __ffsll(~(cont >> lane >> 1));  // the run that begins here: this token and those that continue it
        for (unsigned left = starts; left; left &= left - 1) {
            const int i = __ffs(left) - 1;
            const int64_t page = __shfl_sync(0xffffffffu, v, i) / P, other = win[kWindow + i - 1 - lane];
            if (__any_sync(0xffffffffu, other >= 0 && other / P == page)) {  // the page stands earlier in the call, too
                starts &= ~(1u << i);
                if (lane == 0 && blockIdx.y == 0) atomicOr(A.status, TQ_DEVERR_SLOT_ORDER);
            }
        }
        if (starts >> lane & 1u) {
            const int n = __popc(starts & ((1u << lane) - 1u));
            s_at[n] = lane;
            s_len[n] = len;
        }
        if (lane == 0) s_runs = __popc(starts);
    }
    __syncthreads();
    const int group = warp / W, gl = tid % (32 * W);
    const int u = gl % U, row0 = gl / U;
    int j0, j1;
    unit_chunks(u, A.r, A.interleaved, j0, j1);
    const int gy = static_cast<int>(gridDim.y);
    const int heads = (A.Hkv - static_cast<int>(blockIdx.y) + gy - 1) / gy;
    int flip = 0;
    for (int it = group; it < 2 * heads * s_runs; it += kGroups, flip ^= 1) {
        const int run = it / (2 * heads), x = it - run * (2 * heads);
        const bool val = x >= heads;
        const int h = static_cast<int>(blockIdx.y) + (val ? x - heads : x) * gy;
        const int len = s_len[run];
        const int64_t t = t0 + s_at[run], slot = win[kWindow + s_at[run]];
        const int o = static_cast<int>(slot & (P - 1));
        const int64_t rec = slot / P * A.Hkv + h;
        const int64_t stride = val ? A.vs : A.ks;
        const uint16_t *src = (val ? A.v : A.k) + t * stride + static_cast<int64_t>(h) * D;
        float *scale_at = (val ? A.v_scales : A.k_scales) + rec;
        unsigned char *base = static_cast<unsigned char *>(val ? A.v_pool : A.k_pool) + rec * P * D;
        const bool pair = !val && u < A.r / kUnit;
        uint4 wa[NK], wb[NK];
        int64_t pos[NK];
#pragma unroll
        for (int n = 0; n < NK; ++n) {
            const int row = row0 + n * kRowStep;
            pos[n] = -1;
            if (row < len) {
                wa[n] = ld_pinned(src + row * stride + j0);
                wb[n] = ld_pinned(src + row * stride + j1);
                pos[n] = A.r ? ld_pinned_s64(A.positions + t + row) : 0;
            }
        }
        const float old = o > 0 ? *scale_at : 0.f;
        float a[NK][8], b[NK][8];
        float amax = -1.f;  // stays below zero where no token of the run is written
        unsigned live = 0;  // units that are written
#pragma unroll
        for (int n = 0; n < NK; ++n) {
            if (row0 + n * kRowStep >= len) continue;
            if (A.r && (pos[n] < 0 || pos[n] >= A.rope_rows)) {
                if (h == 0 && !val && u == 0) atomicOr(A.status, TQ_DEVERR_POSITION);
                continue;
            }
            live |= 1u << n;
            unpack8(wa[n], a[n]);
            unpack8(wb[n], b[n]);
            if (pair) turn_unit(a[n], b[n], load_turn(A.rope + pos[n] * A.r, u, A.r), A.interleaved);
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max3(amax, finite_abs(a[n][j]), finite_abs(b[n][j]));
        }
        amax = warp_max(amax);
        if (lane == 0) s_max[group][flip][warp % W] = amax;
        // two sets, so that the next item's do not wait for this one's readers
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(32 * W) : "memory");
#pragma unroll
        for (int k = 0; k < W; ++k) amax = fmaxf(amax, s_max[group][flip][k]);
        if (amax < 0.f) continue;  // the page stays as it was
        const float need = pow2_scale(amax);
        const bool keep = o > 0 && old >= 0.f && old <= 3.402823466e38f;  // the page's rows and scale so far
        const float scale = keep ? fmaxf(old, need) : need;
        const float inv = 1.f / scale;
        if (keep && scale > old) {  // code the earlier rows anew
            const float ratio = old * inv;
            for (int e = gl; e < o * (D / 16); e += 32 * W) {
                uint4 *p = reinterpret_cast<uint4 *>(base) + e;
                const uint4 w = *p;
                *p = make_uint4(recode4(w.x, ratio), recode4(w.y, ratio), recode4(w.z, ratio), recode4(w.w, ratio));
            }
        }
#pragma unroll
        for (int n = 0; n < NK; ++n)
            if (live >> n & 1u) {
                unsigned char *p = base + (o + row0 + n * kRowStep) * D;
                *reinterpret_cast<uint2 *>(p + j0) = codes8(a[n], inv);
                *reinterpret_cast<uint2 *>(p + j1) = codes8(b[n], inv);
            }
        if (gl == 0 && !(keep && scale == old)) *scale_at = scale;
    }
}

template <int D>
cudaError_t launch_bf16(const AppendArgs &a, cudaStream_t st)
{
    constexpr int RL = kThreads / (D / kUnit);
    const int rows = a.Hq + 2 * a.Hkv;
    // Few tokens: a block per RL rows, for latency.  Many: the rows of a token in one block, which reads slot and position
    // once.  The limit is where either fills the GPU's SMs several times over.
    const unsigned gy = a.T < 1024 ? static_cast<unsigned>((rows + RL - 1) / RL) : 1u;
    append_bf16_kernel<D><<<dim3(static_cast<unsigned>(a.T), gy), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int D, int P>
cudaError_t launch_fp8(const AppendArgs &a, int num_sms, cudaStream_t st)
{
    // Few tokens: every one may begin a page's run, so a block for each.  Many: a page's rows of tokens per block (about
    // one run begins among them).  A block takes an item for each of its groups at a time, so further blocks over the
    // heads only where there would be fewer than four blocks an SM (eight: 32k tokens on pages of 32 152 us against 144).
    const int chunk = a.T < 1024 ? 1 : P;
    const int64_t kv = (a.T + chunk - 1) / chunk;
    constexpr int kGroups = kThreads / 32 / group_warps(D, P);
    const int64_t want = (4LL * num_sms + kv - 1) / kv, most = (2LL * a.Hkv + kGroups - 1) / kGroups;
    const int gy = static_cast<int>(want < most ? want : most < 65535 ? most : 65535);
    const int64_t per = static_cast<int64_t>(kThreads / (D / kUnit)) * gy;
    const int64_t q = (a.T * ((a.Hq + kQueryRows - 1) / kQueryRows) + per - 1) / per;
    append_fp8_kernel<D, P><<<dim3(static_cast<unsigned>(kv + q), gy), kThreads, 0, st>>>(a, static_cast<int>(kv), chunk);
    return cudaGetLastError();
}

cudaError_t launch_fp8(const AppendArgs &a, int d, int num_sms, cudaStream_t st)
{
    if (d == 128) return a.P == 16 ? launch_fp8<128, 16>(a, num_sms, st) : launch_fp8<128, 32>(a, num_sms, st);
    return a.P == 16 ? launch_fp8<256, 16>(a, num_sms, st) : launch_fp8<256, 32>(a, num_sms, st);
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
    if (a->Hq > (1 << 18) || a->Hkv > (1 << 18))
        return api_error(TQ_ERR_UNSUPPORTED, "%s: more than 2^18 heads", who);
    // grid sizes, and byte offsets within a pool
    if (a->T >= (int64_t(1) << 30) || a->T * (a->Hq + 2 * a->Hkv) >= (int64_t(1) << 34))
        return api_error(TQ_ERR_UNSUPPORTED, "%s: too many tokens in one call", who);
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
    a->small = a->T * a->Hq < (int64_t(1) << 31);
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
                     nullptr, false};
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
                     nullptr, false};
    bool run;
    const tq_status s = tq::check("tq_append_kv_fp8", h, &a, num_blocks, style, 1, &run);
    if (s != TQ_OK || !run) return s;
    if (!k_scales || !v_scales) return tq::api_error(TQ_ERR_INVALID_ARG, "tq_append_kv_fp8: NULL pointer");
    if (!tq::aligned(k_scales, 4) || !tq::aligned(v_scales, 4))
        return tq::api_error(TQ_ERR_INVALID_ARG, "tq_append_kv_fp8: misaligned pointer");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const tq::Codec &c = tq::handle_codec(h);
    const cudaError_t e = tq::launch_fp8(a, c.d, c.num_sms, st);
    if (e != cudaSuccess) return tq::api_error(TQ_ERR_CUDA, "tq_append_kv_fp8: launch: %s", cudaGetErrorString(e));
    return TQ_OK;
}
