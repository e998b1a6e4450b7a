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

// (amax / 127 by Markstein's correction: with y = 1 / 127 rounded, q = amax y
// and the exact remainder r = amax - 127 q, q + r y rounds to the quotient
// (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", 1990).  Below 127 2^-126, where r could lose bits,
// the floor decides.)
DV_DEV float quant_scale(float amax)
{
    constexpr float y = 1.f / 127.f;
    const float q = amax * y;
    const float s = fmaf(fmaf(-127.f, q, amax), y, q);
    return amax <= 3.402823466e38f ? fmaxf(s, 1.1754943508e-38f) : __int_as_float(0x7fc00000);
}

// The largest of |a|, |b| (and |c|); a NaN stays one.
DV_DEV float amax3(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
DV_DEV float amax2(float a, float b) { return amax3(a, b, b); }
template <int N>
DV_DEV float amax_of(const float (&x)[N], float mx = 0.f)
{
#pragma unroll
    for (int i = 0; i < N; i += 2)
        mx = amax3(mx, x[i], x[i + 1]);
    return mx;
}

// The low bytes of four words.
DV_DEV unsigned low_bytes(unsigned a, unsigned b, unsigned c, unsigned d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// rint(x / s) where x / s lies near a half, t = x inv being within 2^-15 of
// it: with |x| = (h + r / s) s, h = k + 1/2 and the remainder r exact, the
// rounded quotient is h itself (a tie, to even) while |r| is at most half a
// last place of h times s, and else on r's side of it.  Rows of tiny values
// are scaled up first, where the remainder would lose bits.
DV_DEV float code_at_half(float x, float s, float t)
{
    float ax = fabsf(x);
    if (s < 0x1p-60f) {
        ax *= 0x1p64f;
        s *= 0x1p64f;
    }
    const float k = rintf(fabsf(t) - 0.5f), h = k + 0.5f;
    const float r = fmaf(-h, s, ax);
    float half = __uint_as_float(__float_as_uint(h) & 0x7f800000u) * 0x1p-24f;
    if (k == 0.f && r < 0.f)  // below a power of two the places are half as wide
        half *= 0.5f;
    const float lim = half * s;
    const float c = r > lim ? k + 1.f : r < -lim ? k : 2.f * rintf(0.5f * k + 0.25f);
    return copysignf(c, x);
}

// Codes of N values by products with inv = 1 / s (one Newton step: within
// 2^-24 of it) and the magic number 1.5 2^23, whose low byte then holds the
// code.  x inv is within 127 2^-23 of the true quotient and the rounded
// quotient within 2^-18: both round to the same whole number unless x inv is
// 2^-15 from a half (one value in 16000), where code_at_half decides.
// A division per value made a 2048-token append of the 175B-shaped batch of 8
// compute-bound (with the read back 965 us; now 619, 479 of them the bytes' own).
constexpr float kMagic = 12582912.f;
DV_DEV float quant_inv(float s)  // (s lies in [2^-126, 2^121]: no subnormals)
{
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    return fmaf(inv, fmaf(-s, inv, 1.f), inv);
}
// Four values: their codes' bytes.
DV_DEV unsigned quant4(const float *x, float s, float inv)
{
    float u[4], d[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u[i] = fmaf(x[i], inv, kMagic);
        d[i] = fmaf(x[i], inv, kMagic - u[i]);
    }
    if (amax_of(d) > 0.5f - 0x1p-15f) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (fabsf(d[i]) > 0.5f - 0x1p-15f)
                u[i] = code_at_half(x[i], s, x[i] * inv) + kMagic;
    }
    return low_bytes(__float_as_uint(u[0]), __float_as_uint(u[1]), __float_as_uint(u[2]),
                     __float_as_uint(u[3]));
}

// Pairs of codes as binary16: a code's byte with its sign bit flipped is
// code + 128, which under the byte 0x64 reads 1024 + 128 + code.
DV_DEV unsigned codes_lo(unsigned biased)  // bytes 0, 1
{
    unsigned u = __byte_perm(biased, 0x64646464u, 0x4140), r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x64806480u));
    return r;
}
DV_DEV unsigned codes_hi(unsigned biased)  // bytes 2, 3
{
    unsigned u = __byte_perm(biased, 0x64646464u, 0x4342), r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(u), "r"(0x64806480u));
    return r;
}

DV_DEV float ld_row(const KvRowsArgs &r, long long i)
{
    return r.f16 ? __half2float(static_cast<const __half *>(r.p)[i])
                 : static_cast<const float *>(r.p)[i];
}

// ---------------------------------------------------------------------------
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

// Storage type of a cache, and 16 bytes of it as numbers (without a scale).
template <int DT>
struct Store;
template <>
struct Store<DV_F32> {
    using T = float;
    static constexpr int EPC = 4;
    DV_DEV static void unpack(const uint4 &v, float (&f)[4]) { Elem<float>::unpack(v, f); }
};
template <>
struct Store<DV_F16> {
    using T = __half;
    static constexpr int EPC = 8;
    DV_DEV static void unpack(const uint4 &v, float (&f)[8]) { Elem<__half>::unpack(v, f); }
};
template <>
struct Store<DV_I8> {
    using T = int8_t;
    static constexpr int EPC = 16;
    DV_DEV static void unpack(const uint4 &v, float (&f)[16])
    {
        const unsigned u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned b = u[i] ^ 0x80808080u, lo = codes_lo(b), hi = codes_hi(b);
            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
            const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
            f[4 * i] = x.x;
            f[4 * i + 1] = x.y;
            f[4 * i + 2] = y.x;
            f[4 * i + 3] = y.y;
        }
    }
};

// ---------------------------------------------------------------------------
// Mean key of one complete block, by one warp, from the cached rows (visible
// to it).  The mean is defined so that its sum is exact in any order: with n
// positions and 2^e > amax |k| over the block (e >= -100), every key is
// rounded to a multiple of g = n 2^(e - 24), and sums of n such multiples
// are whole numbers below 2^24 times g.  Then mean = (sum / g) 2^(e - 24),
// quantised as a row.  The rounding is below 2^-17 of the block's largest
// value for n = 128, far under a code.  A block with a NaN or an infinity, or
// whose mean rounds to one, gets codes 0 and scale +inf (it is selected first).
//
// A warp a block and no barrier: the other warps of an append go on with the
// values meanwhile (a mean by the whole CTA, with its barriers, took 210 us
// more of a 2048-token append at the 175B shape, batch 8).

// The last step: the sums acc of EPC dimensions from part * EPC on (the same
// in every lane group of lpr lanes) as the quantised mean of row `row`.
template <int EPC>
DV_DEV void store_mean(const KvCacheArgs &c, size_t row, const int (&acc)[EPC], int e2, bool fine,
                       int part, int lpr)
{
    const float step = ldexpf(1.f, e2 - 24);
    float mean[EPC];
#pragma unroll
    for (int e = 0; e < EPC; ++e)
        mean[e] = (float)acc[e] * step;
    float ma = amax_of(mean);
    for (int o = 1; o < lpr; o <<= 1)
        ma = amax2(ma, __shfl_xor_sync(0xffffffffu, ma, o));
    fine &= ma <= 3.402823466e38f;  // (2^24 units of 2^104: all keys at binary32's end)
    const float s = quant_scale(ma);
    if ((int)(threadIdx.x & 31) < lpr) {
        const float inv = quant_inv(s);
        unsigned *dst = reinterpret_cast<unsigned *>(c.mean + row * c.D + part * EPC);
#pragma unroll
        for (int e = 0; e < EPC / 4; ++e)
            dst[e] = fine ? quant4(mean + 4 * e, s, inv) : 0u;
        if (part == 0)
            c.mean_scale[row] = fine ? s : INFINITY;
    }
}

// Exponent e of the grid for a block whose largest magnitude is mx, and 1 / g.
DV_DEV int mean_exponent(float mx) { int e = 0; frexpf(mx, &e); return max(e, -100); }
// A key over g, rounded to a whole number: |key / g| < 2^20 sits in the magic
// number's low bits (1 / g is a power of two: the product is exact).
DV_DEV int mean_units(float key, float inv_g)
{
    return __float_as_int(fmaf(key, inv_g, kMagic)) - 0x4b400000;
}

template <int DT>
DV_DEV void warp_mean(const KvCacheArgs &c, size_t bh, int j)
{
    using St = Store<DT>;
    constexpr int EPC = St::EPC;
    const int lane = threadIdx.x & 31, lpr = c.D / EPC, part = lane % lpr, r0 = lane / lpr;
    const int rows = 32 / lpr, n = c.block;
    const size_t p0 = bh * (size_t)c.cap + (size_t)j * n;
    const typename St::T *k = static_cast<const typename St::T *>(c.k) + p0 * c.D + part * EPC;
    float mx = 0.f;
#pragma unroll 4
    for (int r = r0; r < n; r += rows) {
        float f[EPC];
        St::unpack(*reinterpret_cast<const uint4 *>(k + (size_t)r * c.D), f);
        const float m = amax_of(f);
        mx = amax2(mx, DT == DV_I8 ? m * c.ks[p0 + r] : m);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        mx = amax2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const bool fine = mx <= 3.402823466e38f;
    const int e2 = mean_exponent(fine ? mx : 0.f);
    const float inv = ldexpf(1.f / n, 24 - e2);  // 1 / g
    int acc[EPC];
#pragma unroll
    for (int e = 0; e < EPC; ++e)
        acc[e] = 0;
    if (fine) {
#pragma unroll 2
        for (int r = r0; r < n; r += rows) {
            float f[EPC];
            St::unpack(*reinterpret_cast<const uint4 *>(k + (size_t)r * c.D), f);
            const float s = DT == DV_I8 ? c.ks[p0 + r] : 1.f;
#pragma unroll
            for (int e = 0; e < EPC; ++e)
                acc[e] += mean_units(DT == DV_I8 ? __fmul_rn(f[e], s) : f[e], inv);
        }
    }
#pragma unroll
    for (int e = 0; e < EPC; ++e)
        for (int o = lpr; o < 32; o <<= 1)
            acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
    store_mean<EPC>(c, bh * (size_t)(c.cap / n) + j, acc, e2, fine, part, lpr);
}

}  // namespace
}  // namespace dv
