// tq_fp8.cuh -- what the attention kernels over 8-bit pages share: arguments, scale and
// e4m3 helpers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "tq_device.cuh"
#include "tq_internal.h"

namespace tq {
namespace fp8 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLShift = 4.f;  // denominators are summed as 2^4 p / vs: vs in 2^-100 .. 2^120 neither overflows nor flushes
// The prefill's denominators are sums of 2^-10 P / vs, P up to 2^15: vs in 2^-100 .. 2^120 neither overflows (4 million tokens)
// nor flushes.
constexpr float kSumUnit = 0x1p-10f;

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// log2 of a page scale, exact for powers of two; below 2^-100 (an empty scale) as 2^-100.
__device__ __forceinline__ float log2_scale(float s)
{
    const uint32_t b = __float_as_uint(fmaxf(s, 7.888609052210118e-31f));
    float m;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(m) : "f"(__uint_as_float((b & 0x7fffffu) | 0x3f800000u)));
    return static_cast<float>(static_cast<int>(b >> 23) - 127) + m;
}

// (x, y) to e4m3 (x in the low byte) and what is left of them.
__device__ __forceinline__ uint32_t e4m3x2_rest(float &x, float &y)
{
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(y), "f"(x));
    uint32_t h2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(c));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h2));
    x -= f.x;
    y -= f.y;
    return c;
}

// Two halves to e4m3 and what is left of them (exact).
__device__ __forceinline__ uint32_t e4m3x2_rest(__half2 &x)
{
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
    uint32_t b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"(c));
    x = __hsub2(x, *reinterpret_cast<const __half2 *>(&b));
    return c;
}

__device__ __forceinline__ uint32_t e4m3x2(__half2 x)
{
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(*reinterpret_cast<const uint32_t *>(&x)));
    return c;
}

__device__ __forceinline__ uint32_t e4m3x2(float x, float y)
{
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(y), "f"(x));
    return c;
}

// NaN among 16 value codes of a token that not every query token sees: 0 times NaN would carry it to those that do not.
// Taken out of the products and noted as the coordinate's first such token; the rows that see it get their NaN at the end.
__device__ __forceinline__ void hide_nan(uint4 &w, int *nan_at, int token)
{
    uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t nan = ((v[i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;  // the codes 0x7f and 0xff
        while (nan) {
            const int byte = __ffs(nan) / 8 - 1;
            atomicMin(nan_at + 4 * i + byte, token);
            v[i] &= ~(0xffu << (8 * byte));
            nan &= nan - 1;
        }
    }
    w = make_uint4(v[0], v[1], v[2], v[3]);
}

struct Args {
    const uint16_t *q;
    const float *k_scales, *v_scales;
    const int32_t *block_table, *seq_lens;
    int B, Hq, Hkv, G, P, pshift, max_blocks;
    int64_t num_blocks;
    float sm_scale;
    int splits, pages_per_split;
    int whole;         // prefill: units (sequence, kv head, query block) that are not cut
    int Tq, qpc, nqt;  // query tokens per sequence, per CTA, and CTAs over them
    float *ml, *acc;   // [splits][B][Tq][Hq][2], [splits][B][Tq][Hq][D]; unused with one split
    int *pieces;       // [B][Hkv] pieces of a unit (decode)
    uint16_t *out;
    unsigned *status;
    long long wait_limit;
};

// The tcgen05 kernel: 128 (head dim 256) or 256 (head dim 128) columns, (query token, head) pairs, per CTA.
// prefill_tc_columns: that number for a head dim; launch_prefill_tc sets no argument of `a` itself.
int prefill_tc_columns(int d);
cudaError_t launch_prefill_tc(const CUtensorMap &tk, const CUtensorMap &tv, int d, const Args &a, cudaStream_t st);

}  // namespace fp8
}  // namespace tq
