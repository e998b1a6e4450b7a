// dv_seq_rope.cu -- per-head norms of queries and keys, rotation by position,
// and the store of keys and values in a paged pool, in one pass (sm_103a).
//
// A warp takes one token and a run of its rows (queries, keys, values): it forms
// the token's sines and cosines from 64-bit fixed-point angles, and then a lane
// holds the same 8 dimensions of every row that it meets, with their angles in
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

template <bool F16>
DV_DEV void ld8(const char *p, float (&x)[8])
{
    if constexpr (F16) {
        Elem<__half>::unpack(__ldcs(reinterpret_cast<const uint4 *>(p)), x);
    } else {
        const float4 *q = reinterpret_cast<const float4 *>(p);
        const float4 a = __ldcs(q), b = __ldcs(q + 1);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
        x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}
DV_DEV void st8(char *p, bool f16, const float (&x)[8])
{
    if (f16) {
        __half2 h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            h[e] = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
        *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(h);
    } else {
        float4 *q = reinterpret_cast<float4 *>(p);
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

// D / 8 lanes a row; ROWS rows of a lane group on their way at once.  A token's
// work is cut into runs of `per` rows: query heads (the first q_runs), then KV
// heads (their keys, then their values).
template <bool SRC16, int D>
__global__ void __launch_bounds__(kRopeThreads, 6)
    k_qk_rope(const SeqRopeArgs a, int runs, int q_runs, int per)
{
    constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = SRC16 ? 6 : 4, NW = kRopeThreads / 32;
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
    const int part = lane % LPR, c0 = part * 8, mine = lane / LPR, half = a.rot / 2;

    // sines and cosines, by the lanes; then this lane's: element e turns with sine
    // sn[e] (its sign for the pair's first or second), cosine cs[e]
    float sn[8], cs[8];
    if (a.rot) {
        for (int i = lane; i < half; i += 32) {
            float s, c;
            sincos_turns(__ldg(a.steps + i) * (unsigned long long)pos, &s, &c);
            s_sin[warp][i] = s * a.mscale;
            s_cos[warp][i] = c * a.mscale;
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = c0 + e;
            const bool turns = c < a.rot;
            const int i = !turns ? 0 : a.interleaved ? c >> 1 : c < half ? c : c - half;
            const bool first = a.interleaved ? !(c & 1) : c < half;
            sn[e] = turns ? (first ? -s_sin[warp][i] : s_sin[warp][i]) : 0.f;
            cs[e] = turns ? s_cos[warp][i] : 1.f;
        }
    }
    // where the other of a pair lies: the same element of another lane, or, for
    // halves that end inside a lane's elements, through shared memory
    const bool by_lane = half % 8 == 0;
    const int other = a.interleaved || c0 >= a.rot ? lane
                      : c0 < half ? lane + half / 8 : lane - half / 8;
    float *const row = s_row[warp] + mine * D;

    // Rows h0 .. h1 - 1 of src, to dst (type f16) and, where pool is set, a token's
    // slot of it.
    auto rows = [&](const SeqRowsArgs &src, const SeqRowsArgs &dst, char *pool, const float *gain,
                    bool turn) {
        const long long sstep = src.sh * RPW * ES;
        const char *from = static_cast<const char *>(src.p) +
                           (t * src.st + (h0 + mine) * src.sh + c0) * ES;
        const int de = dst.f16 ? 2 : 4, pe = a.f16 ? 2 : 4;
        const long long dstep = dst.sh * RPW * de, pstep = (long long)a.page * D * RPW * pe;
        char *to = static_cast<char *>(dst.p) + (t * dst.st + (h0 + mine) * dst.sh + c0) * de;
        const bool put = dst.p != nullptr, store = pool != nullptr;
        char *in = pool + (store ? ((long long)(h0 + mine) * a.page * D + c0) * pe : 0);
        float g[8];
        if (gain) {
            const float4 g0 = __ldg(reinterpret_cast<const float4 *>(gain + c0));
            const float4 g1 = __ldg(reinterpret_cast<const float4 *>(gain + c0) + 1);
            g[0] = g0.x, g[1] = g0.y, g[2] = g0.z, g[3] = g0.w;
            g[4] = g1.x, g[5] = g1.y, g[6] = g1.z, g[7] = g1.w;
        }
#pragma unroll 1
        for (int h = h0 + mine; h - mine < h1; h += ROWS * RPW) {
            float x[ROWS][8];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                if (h + i * RPW < h1)
                    ld8<SRC16>(from, x[i]);
                else
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[i][e] = 0.f;
                from += sstep;
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                float(&y)[8] = x[i];
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
                if (turn) {
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
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            row[c0 + e] = y[e];
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int c = c0 + e;
                            z[e] = c >= a.rot ? 0.f : row[c < half ? c + half : c - half];
                        }
                    }
                    if (c0 < a.rot) {  // (others keep what they have, whatever z is)
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (c0 + e < a.rot)
                                y[e] = fmaf(y[e], cs[e], z[e] * sn[e]);
                    }
                }
                if (h + i * RPW < h1) {
                    if (put)
                        st8(to, dst.f16, y);
                    if (store)
                        st8(in, a.f16, y);
                }
                to += dstep;
                in += pstep;
            }
        }
    };
    if (is_q) {
        rows(a.q, a.q_out, nullptr, a.q_gain, a.rot > 0);
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
        rows(a.k, a.k_out, on ? static_cast<char *>(a.pk) + at * pe : nullptr, a.k_gain, a.rot > 0);
    if (a.v.p && on)
        rows(a.v, SeqRowsArgs{}, static_cast<char *>(a.pv) + at * pe, nullptr, false);
}

template <bool SRC16, int D>
cudaError_t launch_rope_d(const SeqRopeArgs &a, cudaStream_t st)
{
    constexpr int RPW = 32 / (D / 8), NW = kRopeThreads / 32;
    // Runs of 32 rows, shorter ones where that leaves fewer than 32 warps an SM; the
    // fewest rows are one of every lane group.
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
    return cudaLaunchKernelEx(&cfg, k_qk_rope<SRC16, D>, a, runs, q_runs, per);
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
