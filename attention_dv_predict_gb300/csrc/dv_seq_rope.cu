// dv_seq_rope.cu -- per-head norms of queries and keys, rotation by position,
// and the store of keys and values in a paged pool, in one pass (sm_103a).
//
// A warp takes one token and a run of its rows (queries, keys, values): it forms
// the token's sines and cosines from 64-bit fixed-point angles, and then a lane
// holds the same four pairs of every row that it meets, with their angles in
// registers.  A row is read once and written once, so bytes bound it; several
// rows a lane are on their way at once, and no warp waits for another (a CTA a
// token, with its barrier, took 411 us for 16384 tokens of 64 + 8 + 8 binary32
// rows of 128 where the bytes take 149).
#include <climits>

#include "dv_common.cuh"
#include "dv_seq.h"

namespace dv {
namespace {

constexpr int kRopeThreads = 128;

// Four values, as they lie.
template <bool F16>
struct Raw4 {
    DV_DEV static void load(const char *p, uint4 &u)
    {
        if constexpr (F16) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
            u.x = v.x, u.y = v.y;
        } else {
            u = __ldcs(reinterpret_cast<const uint4 *>(p));
        }
    }
    DV_DEV static void get(const uint4 &u, float *x)
    {
        if constexpr (F16) {
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
            x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
        } else {
            x[0] = __uint_as_float(u.x), x[1] = __uint_as_float(u.y);
            x[2] = __uint_as_float(u.z), x[3] = __uint_as_float(u.w);
        }
    }
};
DV_DEV void st4(char *p, bool f16, const float *x)
{
    if (f16) {
        const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
        *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const unsigned *>(&a),
                                                   *reinterpret_cast<const unsigned *>(&b));
    } else {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
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

// D / 8 lanes a row; ROWS rows of a lane group on their way at once.  A token's
// work is cut into runs of `per` rows: query heads (the first q_runs), then KV
// heads (their keys, then their values).  ALL: every dimension turns (rot = D), so no
// pair is asked whether it does and none comes from another lane (177 us for those
// 16384 tokens, against 207 with the code of both).
template <bool SRC16, int D, bool ALL>
__global__ void __launch_bounds__(kRopeThreads, 5)
    k_qk_rope(const SeqRopeArgs a, int runs, int q_runs, int per)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = 4, NW = kRopeThreads / 32;
    constexpr int ES = SRC16 ? 2 : 4;
    __shared__ float s_cos[NW][D / 2], s_sin[NW][D / 2];
    __shared__ float s_row[NW][256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long id = (long long)blockIdx.x * NW + warp;
    const int t = (int)(id / runs), run = (int)(id - (long long)t * runs);
    if (t >= a.T)
        return;
    const int pos = __ldg(a.pos + t);
    if (pos < 0)
        return;
    const bool is_q = run < q_runs;
    const int h0 = (is_q ? run : run - q_runs) * per, h1 = min(is_q ? a.H : a.Hkv, h0 + per);
    const int rot = ALL ? D : a.rot, half = rot / 2;
    const int part = lane % LPR, mine = lane / LPR;
    // A lane's dimensions, four from ca and four from cb: both members of its pairs
    // (as halves: ca and the same place of the second half), so that none comes from
    // another lane, unless halves end inside four.
    const bool odd = !ALL && !a.interleaved && half % 4 != 0, split = !a.interleaved && !odd;
    int ca = 8 * part, cb = ca + 4;
    if (split && ca < rot) {
        ca = 4 * part;
        cb = half + ca;
    }

    // sines and cosines, by the lanes; then this lane's four pairs'
    float sn[4], cs[4];
    unsigned turns = 0;  // which of them turn
    if (rot) {
        for (int i = lane; i < half; i += 32) {
            float s, c;
            sincos_turns(__ldg(a.steps + i) * (unsigned long long)pos, &s, &c);
            s_sin[warp][i] = s * a.mscale;
            s_cos[warp][i] = c * a.mscale;
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int i = split ? ca + e : 4 * part + e;  // the pair, if there is one
            const bool on = ALL || (split ? ca < half : i < half);
            turns |= (unsigned)on << e;
            sn[e] = on ? s_sin[warp][i] : 0.f;
            cs[e] = on ? s_cos[warp][i] : 1.f;
        }
    }
    float *const row = s_row[warp] + mine * D;

    // Rows h0 .. h1 - 1 of src, to dst (type f16) and, where pool is set, a token's
    // slot of it.
    auto rows = [&](const SeqRowsArgs &src, const SeqRowsArgs &dst, char *pool, const float *gain,
                    bool turn) {
        const long long sstep = src.sh * RPW * ES;
        const char *from = static_cast<const char *>(src.p) +
                           (t * src.st + (h0 + mine) * src.sh + ca) * ES;
        const int de = dst.f16 ? 2 : 4, pe = a.f16 ? 2 : 4;
        const long long dstep = dst.sh * RPW * de, pstep = (long long)a.page * D * RPW * pe;
        char *to = static_cast<char *>(dst.p) + (t * dst.st + (h0 + mine) * dst.sh + ca) * de;
        const int fb = (cb - ca) * ES, db = (cb - ca) * de, pb = (cb - ca) * pe;
        const bool put = dst.p != nullptr, store = pool != nullptr;
        char *in = pool + (store ? ((long long)(h0 + mine) * a.page * D + ca) * pe : 0);
        float g[8];
        if (gain) {
            const float4 g0 = __ldg(reinterpret_cast<const float4 *>(gain + ca));
            const float4 g1 = __ldg(reinterpret_cast<const float4 *>(gain + cb));
            g[0] = g0.x, g[1] = g0.y, g[2] = g0.z, g[3] = g0.w;
            g[4] = g1.x, g[5] = g1.y, g[6] = g1.z, g[7] = g1.w;
        }
#pragma unroll 1
        for (int h = h0 + mine; h - mine < h1; h += ROWS * RPW) {
            uint4 x[ROWS][2];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                if (h + i * RPW < h1) {
                    Raw4<SRC16>::load(from, x[i][0]);
                    Raw4<SRC16>::load(from + fb, x[i][1]);
                }
                from += sstep;
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                float y[8];  // (rows behind the last: whatever is there, stored nowhere)
                Raw4<SRC16>::get(x[i][0], y);
                Raw4<SRC16>::get(x[i][1], y + 4);
                if (gain) {
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
                    for (int e = 0; e < 8; ++e) {
                        y[e] -= mean;
                        sq = fmaf(y[e], y[e], sq);
                    }
#pragma unroll
                    for (int o = 1; o < LPR; o <<= 1)
                        sq += __shfl_xor_sync(0xffffffffu, sq, o);
                    const float f = 1.f / sqrtf(sq * (1.f / D) + a.eps);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] *= f * g[e];
                }
                if (turn && !odd) {
                    // (a choice of the result: a value that does not turn may be infinite
                    // or NaN, and a product with a sine of zero would spread it)
                    auto rotate = [&](float &p, float &q, int e) {
                        const float r = fmaf(p, cs[e], -q * sn[e]);
                        const float u = fmaf(q, cs[e], p * sn[e]);
                        const bool on = ALL || ((turns >> e) & 1);
                        p = on ? r : p;
                        q = on ? u : q;
                    };
                    if (a.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            rotate(y[2 * e], y[2 * e + 1], e);
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            rotate(y[e], y[4 + e], e);
                    }
                } else if (turn) {
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        row[ca + e] = y[e];
                    __syncwarp();
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int c = ca + e, k = c < half ? c : c - half;
                        if (c < rot)
                            y[e] = fmaf(y[e], s_cos[warp][k],
                                        c < half ? -row[c + half] * s_sin[warp][k]
                                                 : row[k] * s_sin[warp][k]);
                    }
                }
                if (h + i * RPW < h1) {
                    if (put) {
                        st4(to, dst.f16, y);
                        st4(to + db, dst.f16, y + 4);
                    }
                    if (store) {
                        st4(in, a.f16, y);
                        st4(in + pb, a.f16, y + 4);
                    }
                }
                to += dstep;
                in += pstep;
            }
        }
    };
    if (is_q) {
        rows(a.q, a.q_out, nullptr, a.q_gain, rot > 0);
        return;
    }
    const int slot = a.pk ? __ldg(a.slots + t) : -1;
    if (slot >= a.n_pages * a.page) {
        if (lane == 0)
            set_status(a.status, DV_ERR_DEVICE_INDEX);
    }
    const bool on = slot >= 0 && slot < a.n_pages * a.page;
    const long long at = on ? ((long long)(slot / a.page) * a.Hkv * a.page + slot % a.page) * D : 0;
    const int pe = a.f16 ? 2 : 4;
    if (a.k_out.p || on)
        rows(a.k, a.k_out, on ? static_cast<char *>(a.pk) + at * pe : nullptr, a.k_gain, rot > 0);
    if (a.v.p && on)
        rows(a.v, SeqRowsArgs{}, static_cast<char *>(a.pv) + at * pe, nullptr, false);
}

template <bool SRC16, int D>
cudaError_t launch_rope_d(const SeqRopeArgs &a, cudaStream_t st)
{
    constexpr int RPW = 32 / (D / 8), NW = kRopeThreads / 32;
    // Runs of 32 rows, shorter ones where that leaves fewer than 152 x 32 warps (an SM
    // holds 20 at a time); the fewest rows are one of every lane group.
    int per = 32 / RPW * RPW, q_runs, runs;
    for (;; per -= RPW) {
        q_runs = (a.H + per - 1) / per;
        runs = q_runs + (a.Hkv + per - 1) / per;
        if (per == RPW || (long long)a.T * runs >= 152 * 32)
            break;
    }
    const long long ctas = ((long long)a.T * runs + NW - 1) / NW;
    if (ctas > INT_MAX)
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kRopeThreads);
    cfg.stream = st;
    return a.rot == D ? cudaLaunchKernelEx(&cfg, k_qk_rope<SRC16, D, true>, a, runs, q_runs, per)
                      : cudaLaunchKernelEx(&cfg, k_qk_rope<SRC16, D, false>, a, runs, q_runs, per);
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
