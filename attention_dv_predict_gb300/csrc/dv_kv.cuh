// dv_kv.cuh -- device helpers of the KV-cache operators (sm_103a).
#pragma once

#include "dv_common.cuh"
#include "dv_kv.h"

namespace dv {
namespace {

// ---------------------------------------------------------------------------
// 8-bit rows.  A row of D values is held as codes c in [-127, 127] and one
// binary32 scale s: value = c s, with
//   s = max(amax |x| / 127, 2^-126),   c = rint(x / s)
// (both quotients rounded to binary32, ties of rint to even).  The floor
// keeps s normal, so that x / s and c s have full precision.  A row that
// holds a NaN or an infinity has s = NaN and codes 0: it reads back as NaN.

DV_DEV float quant_scale(float amax)
{
    return amax <= 3.402823466e38f ? fmaxf(__fdiv_rn(amax, 127.f), 1.1754943508e-38f)
                                   : __int_as_float(0x7fc00000);
}

// x / s rounded to a code (s not NaN; |x| <= amax).
DV_DEV int quant_code(float x, float s) { return __float2int_rn(__fdiv_rn(x, s)); }

// |a| and |b|, larger first; a NaN stays one.
DV_DEV float amax2(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

DV_DEV unsigned pack_codes(int a, int b, int c, int d)
{
    return (a & 0xff) | (b & 0xff) << 8 | (c & 0xff) << 16 | (unsigned)d << 24;
}

// Four consecutive values of a cached row (i: a multiple of 4), without its scale.
DV_DEV float4 ld_cached4(const void *base, int dtype, size_t i)
{
    if (dtype == DV_F32)
        return __ldcg(reinterpret_cast<const float4 *>(static_cast<const float *>(base) + i));
    if (dtype == DV_F16) {
        const uint2 u =
            __ldcg(reinterpret_cast<const uint2 *>(static_cast<const __half *>(base) + i));
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    const unsigned u = __ldcg(reinterpret_cast<const unsigned *>(static_cast<const int8_t *>(base) + i));
    return make_float4((int8_t)u, (int8_t)(u >> 8), (int8_t)(u >> 16), (int8_t)(u >> 24));
}

DV_DEV float ld_row(const KvRowsArgs &r, long long i)
{
    return r.f16 ? __half2float(static_cast<const __half *>(r.p)[i])
                 : static_cast<const float *>(r.p)[i];
}

// Four consecutive values of a row given by the caller (16-byte aligned for
// binary32, 8-byte for binary16).
DV_DEV float4 ld_row4(const KvRowsArgs &r, long long i)
{
    if (!r.f16)
        return *reinterpret_cast<const float4 *>(static_cast<const float *>(r.p) + i);
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const __half *>(r.p) + i);
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

// ---------------------------------------------------------------------------
// Mean key of one complete block, by the whole CTA (blockDim a multiple of
// 32, >= D / 4; barriers inside).  The mean is defined so that its sum is
// exact in binary32 in any order: with n positions and 2^e > amax |k| over
// the block (e >= -100), every key is rounded to a multiple of
// g = n 2^(e - 24), and sums of n such multiples stay below 2^24 g.  Then
// mean = (sum / g) 2^(e - 24), quantised as a row.  The rounding is below
// 2^-17 of the block's largest value for n = 128, far under a code.
// A block with a NaN or an infinity gets codes 0 and scale +inf (it is
// selected first).
struct MeanSmem {
    float red[33];
    float sum[256];
};

DV_DEV float block_amax(float v, float *scratch)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = amax2(v, __shfl_xor_sync(0xffffffffu, v, o));
    if (lane == 0)
        scratch[warp] = v;
    __syncthreads();
    float r = 0.f;
    for (int w = 0; w < nw; ++w)
        r = amax2(r, scratch[w]);
    __syncthreads();
    return r;
}

DV_DEV void block_mean(const KvCacheArgs &c, size_t bh, int j, MeanSmem &sm)
{
    const int D = c.D, n = c.block, lpr = D / 4;  // lanes per row
    const int rows = blockDim.x / lpr, r0 = threadIdx.x / lpr, d0 = (threadIdx.x % lpr) * 4;
    const size_t p0 = bh * (size_t)c.cap + (size_t)j * n;
    const bool on = r0 < rows;  // (blockDim need not be a multiple of lpr)
    float mx = 0.f;
    if (on)
        for (int r = r0; r < n; r += rows) {
            float4 x = ld_cached4(c.k, c.dtype, (p0 + r) * D + d0);
            if (c.dtype == DV_I8) {
                const float s = __ldcg(c.ks + p0 + r);
                x = make_float4(x.x * s, x.y * s, x.z * s, x.w * s);
            }
            mx = amax2(mx, amax2(amax2(x.x, x.y), amax2(x.z, x.w)));
        }
    mx = block_amax(mx, sm.red);
    for (int d = threadIdx.x; d < D; d += blockDim.x)
        sm.sum[d] = 0.f;
    __syncthreads();
    const bool fine = mx <= 3.402823466e38f;
    int e = 0;
    frexpf(fine ? mx : 0.f, &e);
    e = max(e, -100);
    const float inv = ldexpf(1.f / n, 24 - e);  // 1 / g
    if (on && fine) {
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = r0; r < n; r += rows) {
            float4 x = ld_cached4(c.k, c.dtype, (p0 + r) * D + d0);
            if (c.dtype == DV_I8) {
                const float s = __ldcg(c.ks + p0 + r);
                x = make_float4(x.x * s, x.y * s, x.z * s, x.w * s);
            }
            acc.x += rintf(x.x * inv);
            acc.y += rintf(x.y * inv);
            acc.z += rintf(x.z * inv);
            acc.w += rintf(x.w * inv);
        }
        // whole numbers below 2^24: the order of these adds does not matter
        atomicAdd(&sm.sum[d0], acc.x);
        atomicAdd(&sm.sum[d0 + 1], acc.y);
        atomicAdd(&sm.sum[d0 + 2], acc.z);
        atomicAdd(&sm.sum[d0 + 3], acc.w);
    }
    __syncthreads();
    const float step = ldexpf(1.f, e - 24);
    float ma = 0.f;
    for (int d = threadIdx.x; d < D; d += blockDim.x)
        ma = amax2(ma, sm.sum[d] * step);
    ma = block_amax(ma, sm.red);
    const float s = quant_scale(ma);
    const size_t row = bh * (size_t)(c.cap / n) + j;
    for (int d = threadIdx.x; d < D; d += blockDim.x)
        c.mean[row * D + d] = fine ? (int8_t)quant_code(sm.sum[d] * step, s) : (int8_t)0;
    if (threadIdx.x == 0)
        c.mean_scale[row] = fine ? s : INFINITY;
    __syncthreads();
}

}  // namespace
}  // namespace dv
