// dv_kv_tma.cuh -- barriers, tensor-map copies and small arithmetic shared by
// the KV attention kernels on tensor cores (sm_103a).
#pragma once

#include <cuda_fp16.h>

#include "dv_kv_sched.cuh"

namespace dv {
namespace {

DV_DEV unsigned smem_addr(const void *p) { return (unsigned)__cvta_generic_to_shared(p); }

DV_DEV void bar_init(unsigned bar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
DV_DEV void bar_expect(unsigned bar, int bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
DV_DEV void bar_arrive(unsigned bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// True once the phase with this parity is complete; false after 2^21 polls
// of at most a microsecond each.
constexpr int kKvSpin = 1 << 21;
DV_DEV bool bar_wait(unsigned bar, unsigned parity)
{
    for (int it = 0; it < kKvSpin; ++it) {
        unsigned ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(1000)
            : "memory");
        if (ok)
            return true;
    }
    return false;
}

// Box at (byte x of the rows, position, (row, head)) of a cache side.
DV_DEV void tma_load(unsigned dst, const CUtensorMap *map, int x, int pos, int bh, unsigned bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(pos), "r"(bh), "r"(bar)
        : "memory");
}

DV_DEV void cp4(unsigned dst, const void *src, bool on)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 4 : 0)
                 : "memory");
}
DV_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
DV_DEV void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

DV_DEV uint4 lds16(unsigned a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(a));
    return r;
}
DV_DEV void sts16(unsigned a, unsigned x, unsigned y, unsigned z, unsigned w)
{
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z),
                 "r"(w)
                 : "memory");
}
DV_DEV uint2 lds8(unsigned a)
{
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}

DV_DEV unsigned h2(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&h);
}
// The part of (a, b) that the binary16 pair `hi` leaves.
DV_DEV unsigned h2_rest(float a, float b, unsigned hi)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return h2(a - f.x, b - f.y);
}

DV_DEV float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
DV_DEV float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// Two binary32 operations an instruction.
DV_DEV unsigned long long pack2(float a, float b)
{
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
DV_DEV void unpack2(unsigned long long v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
DV_DEV void add2(float &a, float &b, float c, float d)
{
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a, b)), "l"(pack2(c, d)));
    unpack2(r, a, b);
}
DV_DEV void mul2(float &a, float &b, float c, float d)
{
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a, b)), "l"(pack2(c, d)));
    unpack2(r, a, b);
}
DV_DEV void fma2(float &a, float &b, float c, float d)  // a c + d, b c + d
{
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r)
        : "l"(pack2(a, b)), "l"(pack2(c, c)), "l"(pack2(d, d)));
    unpack2(r, a, b);
}

// A softmax row's reference point.  Weights are w_p = 2^(s_p - m) v_p (s: the
// score in units of log2, v: the value row's scale, 1 in binary16 caches) and
// l = sum 2^(s_p - m), o = sum w_p value_p, so m cancels from o / l and may be
// anything that keeps w in binary16's range.  It is set by a row's first
// weights and moves when a weight or a sum leaves its range: the largest weight
// is then taken to between 2^6 and 2^7, whatever v is.  So the low parts' last
// place, 2^-24, is 2^-30 of the largest weight for value rows of any size down
// to scales of 2^-60, where the shift ends (it keeps l finite: 2^66 a position),
// and no step needs a row's maximum.  (First weights taken to 2^12, nearer to
// the end of the range, moved more often: 64-token trees of 32 x 96 heads x
// 2048 8-bit positions 737 us against 687, rows moving together.)  m is a whole
// number, so that every change of reference scales by a power of two, without
// an error.  m = -inf: nothing seen yet.
constexpr float kWeightMax = 65504.f;  // the largest binary16
constexpr float kSumMax = 0x1p100f;  // 2^(s - m) itself must stay finite where v is tiny
constexpr float kShiftMin = -60.f;
// A reference for the scores' maximum top (over a row) before weights are
// known, and the one to use by the weights' maximum big under it.  Neither is
// below the reference m before.
DV_DEV float ref_from_scores(float m, float top) { return fmaxf(m, floorf(top) - 6.f); }
DV_DEV float ref_new(float m, float m0, float big)
{
    if (!(big <= 3.402823466e38f))  // (the row's result is not finite)
        return m0;
    const int e = (int)(__float_as_uint(big) >> 23) - 127;
    return fmaxf(m, m0 + fmaxf((float)(e - 6), kShiftMin));
}
// 2^d for a whole number d <= 127; 0 below 2^-126 and for NaN (two references
// of rows that see nothing, or whose result is not finite anyway).
DV_DEV float pow2(float d) { return d >= -126.f ? __int_as_float(((int)d + 127) << 23) : 0.f; }
// x 2^d, also where x is large and 2^d below 2^-126: the sums l of rows whose
// value scales lie far apart (zero rows have 2^-126).
DV_DEV float times_pow2(float x, float d)
{
    return x * pow2(fmaxf(d, -126.f)) * pow2(fminf(d + 126.f, 0.f));
}

// Four values of a query row, already scaled for the softmax, as binary16 high
// and low parts {hi01, hi23}, {lo01, lo23} after a power of two takes the
// row's largest element into [2^13, 2^14); *inv undoes it.  The lanes of a
// warp hold the row (v: zeros past its end).
DV_DEV float query_power(float mx, float *inv)
{
    // (mx's exponent field; none for a row that is zero or not finite)
    const int field = (int)(__float_as_uint(mx) >> 23);
    const int e = field == 255 || mx == 0.f ? 0 : min(140 - field, 100);
    *inv = __int_as_float((127 - e) << 23);
    return __int_as_float((127 + e) << 23);
}
struct SplitQ {
    unsigned hi01, hi23, lo01, lo23;
};
DV_DEV SplitQ split_row(float4 v, float scale, float *inv)
{
    v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
    float mx = amax3(amax2(v.x, v.y), v.z, v.w);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        mx = amax2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float al = query_power(mx, inv);
    SplitQ q;
    q.hi01 = h2(v.x * al, v.y * al);
    q.hi23 = h2(v.z * al, v.w * al);
    q.lo01 = h2_rest(v.x * al, v.y * al, q.hi01);
    q.lo23 = h2_rest(v.z * al, v.w * al, q.hi23);
    return q;
}

// Four values at each of N query rows, zeros where at < 0; the loads go out
// together (one branch on the type around them all, not one each).
template <int N>
DV_DEV void ld_queries(const KvRowsArgs &q, const long long (&at)[N], float4 (&v)[N])
{
    if (q.f16) {
        uint2 u[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            u[i] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __half *>(q.p) +
                                                         (at[i] < 0 ? 0 : at[i])));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u[i].x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u[i].y));
            v[i] = make_float4(a.x, a.y, b.x, b.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(q.p) +
                                                          (at[i] < 0 ? 0 : at[i])));
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (at[i] < 0)
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

template <bool BLOCK>
DV_DEV int unit_bh(const KvAttnArgs &a, const Unit &u)
{
    return u.b * a.c.Hkv + (BLOCK ? u.h / (a.H / a.c.Hkv) : u.h);
}

template <class K>
cudaError_t kv_occupancy(K kern, int threads, size_t smem, int *per_sm)
{
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)smem);
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, kern, threads, smem);
    if (e == cudaSuccess && *per_sm < 1)
        e = cudaErrorInvalidConfiguration;
    return e;
}

}  // namespace
}  // namespace dv
