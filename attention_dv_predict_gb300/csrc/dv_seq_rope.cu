// dv_seq_rope.cu -- per-head norms of queries and keys, rotation by position,
// and the store of keys and values in a paged pool, in one pass (sm_103a).
//
// A CTA takes one token and a run of its rows (queries, keys, values); its sines
// and cosines are formed once, from 64-bit fixed-point angles, and stay in
// registers: a lane holds the same 8 dimensions of every row that it meets.  A
// row is read once and written once, so bytes bound it.
#include "dv_common.cuh"
#include "dv_seq.h"

namespace dv {
namespace {

constexpr int kRopeThreads = 256;

template <bool F16>
DV_DEV void ld8(const void *p, long long i, float (&x)[8])
{
    if constexpr (F16) {
        const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(static_cast<const __half *>(p) + i));
        Elem<__half>::unpack(u, x);
    } else {
        const float4 *q = reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i);
        const float4 a = __ldcs(q), b = __ldcs(q + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}
DV_DEV void st8(void *p, long long i, bool f16, const float (&x)[8])
{
    if (f16) {
        __half2 h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
        *reinterpret_cast<uint4 *>(static_cast<__half *>(p) + i) = *reinterpret_cast<uint4 *>(h);
    } else {
        float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        q[0] = make_float4(x[0], x[1], x[2], x[3]);
        q[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// Sine and cosine of `turns` 2^-64 turns.  The quarter turn is taken off in
// whole numbers; what is left, at most an eighth, converts to binary32 with a
// relative error of 2^-24.
DV_DEV void sincos_turns(unsigned long long turns, float *s, float *c)
{
    const unsigned t = (unsigned)(turns >> 32) + ((unsigned)(turns >> 31) & 1u);
    const unsigned q = (t + 0x20000000u) >> 30;
    const float x = (float)(int)(t - (q << 30)) * 0x1p-31f;  // half turns
    float sn, cs;
    sincospif(x, &sn, &cs);
    const float a = q & 1 ? cs : sn, b = q & 1 ? sn : cs;
    *s = q & 2 ? -a : a;
    *c = (q + 1) & 2 ? -b : b;
}

// D / 8 lanes a row; ROWS rows of a lane group on their way at once.
template <bool SRC16, int D>
__global__ void __launch_bounds__(kRopeThreads) k_qk_rope(const SeqRopeArgs a, int rows_per_cta)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = 4;
    __shared__ float s_cos[D / 2], s_sin[D / 2];
    __shared__ float s_row[kRopeThreads / 32][256];
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pos = __ldg(a.pos + t);
    if (pos < 0)
        return;
    const int part = lane % LPR, c0 = part * 8, half = a.rot / 2;
    const int nq = a.H, nk = a.H + a.Hkv, nrows = a.v.p ? nk + a.Hkv : nk;
    const int r0 = blockIdx.y * rows_per_cta, r1 = min(nrows, r0 + rows_per_cta);
    int slot = a.pk ? __ldg(a.slots + t) : -1;
    if (slot >= a.n_pages * a.page) {
        slot = -1;
        if (tid == 0 && blockIdx.y == 0)
            set_status(a.status, DV_ERR_DEVICE_INDEX);
    }
    constexpr int NW = kRopeThreads / 32, STEP = NW * RPW * ROWS;
    float x[ROWS][8];
    // row of lane group g in batch i
    auto row_at = [&](int base, int i) { return base + (i * NW + warp) * RPW + lane / LPR; };
    auto fetch = [&](int base) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = row_at(base, i);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[i][e] = 0.f;
            if (r < r1) {
                const SeqRowsArgs &s = r < nq ? a.q : r < nk ? a.k : a.v;
                const int h = r < nq ? r : r < nk ? r - nq : r - nk;
                ld8<SRC16>(s.p, t * s.st + h * s.sh + c0, x[i]);
            }
        }
    };
    fetch(r0);
    for (int i = tid; i < half; i += kRopeThreads) {
        float s, c;
        sincos_turns(a.steps[i] * (unsigned long long)pos, &s, &c);
        s_sin[i] = s * a.mscale;
        s_cos[i] = c * a.mscale;
    }
    __syncthreads();
    // this lane's angles: element e turns with sine sn[e] (its sign for the
    // pair's first or second), cosine cs[e]
    float sn[8], cs[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = c0 + e;
        const bool turns = c < a.rot;
        const int i = !turns ? 0 : a.interleaved ? c >> 1 : c < half ? c : c - half;
        const bool first = a.interleaved ? !(c & 1) : c < half;
        sn[e] = turns ? (first ? -s_sin[i] : s_sin[i]) : 0.f;
        cs[e] = turns ? s_cos[i] : 1.f;
    }
    // where the other of a pair lies: the same element of another lane, or, for
    // halves that end inside a lane's elements, through shared memory
    const bool by_lane = half % 8 == 0;
    const int other = a.interleaved || c0 >= a.rot ? lane
                      : c0 < half ? lane + half / 8 : lane - half / 8;

    for (int base = r0; base < r1; base += STEP) {
        if (base != r0)
            fetch(base);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int r = row_at(base, i);
            float(&y)[8] = x[i];
            const float *gain = r < nq ? a.q_gain : r < nk ? a.k_gain : nullptr;
            if (a.q_gain || a.k_gain) {  // (a lane without a gain takes part)
                float mean = 0.f;
                if (a.layer) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        mean += y[e];
#pragma unroll
                    for (int o = 1; o < LPR; o <<= 1)
                        mean += __shfl_xor_sync(0xffffffffu, mean, o);
                    mean *= 1.f / D;
                }
                float sq = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sq = fmaf(y[e] - mean, y[e] - mean, sq);
#pragma unroll
                for (int o = 1; o < LPR; o <<= 1)
                    sq += __shfl_xor_sync(0xffffffffu, sq, o);
                if (gain) {
                    const float f = 1.f / sqrtf(sq * (1.f / D) + a.eps);
                    const float4 g0 = __ldg(reinterpret_cast<const float4 *>(gain + c0));
                    const float4 g1 = __ldg(reinterpret_cast<const float4 *>(gain + c0) + 1);
                    const float g[8] = {g0.x, g0.y, g0.z, g0.w, g1.x, g1.y, g1.z, g1.w};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = (y[e] - mean) * f * g[e];
                }
            }
            if (a.rot) {
                float z[8];
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[e] = y[e ^ 1];
                } else if (by_lane) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        z[e] = __shfl_sync(0xffffffffu, y[e], other);
                } else {
                    float *s = s_row[warp] + (lane / LPR) * D;
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        s[c0 + e] = y[e];
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int c = c0 + e;
                        z[e] = c >= a.rot ? 0.f : s[c < half ? c + half : c - half];
                    }
                }
                if (r < nk && c0 < a.rot) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c0 + e < a.rot)
                            y[e] = fmaf(y[e], cs[e], z[e] * sn[e]);
                }
            }
            if (r >= r1)
                continue;
            if (r < nq) {
                st8(a.q_out.p, t * a.q_out.st + r * a.q_out.sh + c0, a.q_out.f16, y);
                continue;
            }
            const int h = r < nk ? r - nq : r - nk;
            if (r < nk && a.k_out.p)
                st8(a.k_out.p, t * a.k_out.st + h * a.k_out.sh + c0, a.k_out.f16, y);
            if (slot >= 0)
                st8(r < nk ? a.pk : a.pv,
                    (((long long)(slot / a.page) * a.Hkv + h) * a.page + slot % a.page) * D + c0,
                    a.f16, y);
        }
    }
}

template <bool SRC16, int D>
cudaError_t launch_rope_d(const SeqRopeArgs &a, cudaStream_t st)
{
    constexpr int PASS = kRopeThreads / 32 * (32 / (D / 8));  // rows a CTA takes at once
    const int nrows = a.H + a.Hkv * (a.v.p ? 2 : 1);
    // Four batches of rows on their way in one CTA where the tokens fill the
    // machine; a batch a CTA where they do not.
    int per = PASS * 4;
    while (per > PASS && (long long)a.T * ((nrows + per - 1) / per) < 152 * 8)
        per -= PASS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.T, (nrows + per - 1) / per);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, k_qk_rope<SRC16, D>, a, per);
}

template <bool SRC16>
cudaError_t launch_rope(const SeqRopeArgs &a, cudaStream_t st)
{
    switch (a.D) {
    case 8: return launch_rope_d<SRC16, 8>(a, st);
    case 16: return launch_rope_d<SRC16, 16>(a, st);
    case 32: return launch_rope_d<SRC16, 32>(a, st);
    case 64: return launch_rope_d<SRC16, 64>(a, st);
    case 128: return launch_rope_d<SRC16, 128>(a, st);
    case 256: return launch_rope_d<SRC16, 256>(a, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_qk_rope(const SeqRopeArgs &a, cudaStream_t st)
{
    return a.q.f16 ? launch_rope<true>(a, st) : launch_rope<false>(a, st);
}

}  // namespace dv
