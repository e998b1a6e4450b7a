// dv_kv_attn.cu -- attention over a KV cache for drafted trees and selected
// blocks on CUDA cores: every storage type and head size (sm_103a).
//
// o_r = sum_p softmax_p(scale q_r . k_p) v_p over the positions that row r
// sees, with the running max and sum of an online softmax in binary32.  A
// group of D esize / 16 lanes covers one cached row with 16-byte loads and
// serves four query rows with it; the groups of a warp, then the four warps
// (16 positions of a 64-position tile each) are merged when a unit ends
// (dv_kv_sched.cuh).  It serves binary32 caches and head sizes the
// tensor-core kernel does not tile.
//
// Four passes' rows (two of 8 bits: registers) are loaded together and their
// dot products reduced side by side: one token of 8 x 96 heads over 2049
// binary32 positions of 128 values takes 279 us, 0.85 of the bytes' rate (a
// pass at a time 1068).  More query rows are bound by the arithmetic and the
// shuffles of the CUDA cores: 64 tokens of one batch row 1174 us.
#include "dv_kv_sched.cuh"

namespace dv {
namespace {

constexpr int kGenThreads = 128;
constexpr int kGenWarps = kGenThreads / 32;
constexpr int RM = kKvGenRows;

// 16 bytes of a row as numbers.  (8-bit codes one by one: by pairs of binary16, as
// Store does it, one token of 8 x 32 heads over 2049 rows of 256 takes 244 us
// instead of 204.)
template <int DT>
DV_DEV void unpack(const uint4 &v, float (&f)[Store<DT>::EPC])
{
    if constexpr (DT == DV_I8) {
        const unsigned u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 16; ++i)
            f[i] = (float)(int8_t)(u[i / 4] >> (8 * (i % 4)));
    } else {
        Store<DT>::unpack(v, f);
    }
}

DV_DEV float safe(float m) { return m == -INFINITY ? 0.f : m; }

template <int DT, bool BLOCK>
__global__ void __launch_bounds__(kGenThreads) k_kv_attn(const KvAttnArgs a)
{
    using T = typename Store<DT>::T;
    constexpr int EPC = Store<DT>::EPC;
    __shared__ SchedSmem sm;
    __shared__ __align__(16) float qs[RM][256];
    __shared__ __align__(16) float wo[kGenWarps][RM][256];
    __shared__ float wm[kGenWarps][RM], wl[kGenWarps][RM], um[RM], ul[RM];
    __shared__ float wgt[kMergePieces][RM];
    __shared__ __align__(16) float so[RM * 256];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.c.D, lpk = D / EPC, dc = lane % lpk, ks = lane / lpk, kpw = 32 / lpk;
    const T *K = static_cast<const T *>(a.c.k);
    const T *V = static_cast<const T *>(a.c.v);
    const int G = a.H / a.c.Hkv;
    const Run run = sched_init<BLOCK>(a, RM, sm);
    Finish<BLOCK, RM, kGenThreads> fin;

    for (long long w = run.lo; w < run.hi;) {
        const Unit x = sched_unit<BLOCK>(a, RM, sm, run, w);
        const long long wend = min(run.hi, x.w1);
        const int t0 = tile_of(x, tile_place(x, w)), t1 = tile_of(x, wend);
        w = wend;
        if (x.h < 0)
            continue;
        for (int i = threadIdx.x; i < RM * D; i += kGenThreads) {
            const int r = i / D, d = i - r * D;
            qs[r][d] = r < x.nrows ? ld_row(a.q, q_at<BLOCK>(a, x, r) + d) * a.scale : 0.f;
        }
        unsigned long long bits[RM];
#pragma unroll
        for (int r = 0; r < RM; ++r)
            bits[r] = !BLOCK && r < x.nrows ? seen_bits(a, x, row_token(a, x.row0 + r)) : 0ull;
        __syncthreads();
        const size_t base =
            ((size_t)x.b * a.c.Hkv + (BLOCK ? x.h / G : x.h)) * (size_t)a.c.cap;
        float m[RM], l[RM], o[RM][EPC];
#pragma unroll
        for (int r = 0; r < RM; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int e = 0; e < EPC; ++e)
                o[r][e] = 0.f;
        }
        for (int t = t0; t < t1; ++t) {
            constexpr int PW = kKvTile / kGenWarps;  // positions of a warp's share
            constexpr int U = EPC == 16 ? 2 : 4;  // passes whose rows are on their way together
            for (int s = 0; s < PW; s += U * kpw) {
                int p[U];
                uint4 kv[U], vv[U];
                float ksc[U], vsc[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = s + u * kpw + ks;
                    const int at = t * kKvTile + warp * PW + i;
                    p[u] = -1;
                    if (i < PW) {
                        if (BLOCK)
                            p[u] = block_pos(a, x, at);
                        else
                            p[u] = at < x.len + x.ntok ? at : -1;
                    }
                    kv[u] = vv[u] = make_uint4(0u, 0u, 0u, 0u);
                    ksc[u] = vsc[u] = 1.f;
                    if (p[u] >= 0) {
                        kv[u] = __ldcg(reinterpret_cast<const uint4 *>(K + (base + p[u]) * D) + dc);
                        vv[u] = __ldcg(reinterpret_cast<const uint4 *>(V + (base + p[u]) * D) + dc);
                        if (DT == DV_I8) {
                            ksc[u] = __ldcg(a.c.ks + base + p[u]);
                            vsc[u] = __ldcg(a.c.vs + base + p[u]);
                        }
                    }
                }
#pragma unroll
                for (int r = 0; r < RM; ++r) {
                    if (r >= x.nrows)
                        break;
                    float dot[U];
                    const float4 *qp = reinterpret_cast<const float4 *>(&qs[r][dc * EPC]);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float kf[EPC];
                        unpack<DT>(kv[u], kf);
                        dot[u] = 0.f;
#pragma unroll
                        for (int e = 0; e < EPC; e += 4) {
                            const float4 q = qp[e / 4];
                            dot[u] = fmaf(q.x, kf[e], dot[u]);
                            dot[u] = fmaf(q.y, kf[e + 1], dot[u]);
                            dot[u] = fmaf(q.z, kf[e + 2], dot[u]);
                            dot[u] = fmaf(q.w, kf[e + 3], dot[u]);
                        }
                    }
                    for (int off = lpk / 2; off > 0; off >>= 1)
#pragma unroll
                        for (int u = 0; u < U; ++u)
                            dot[u] += __shfl_xor_sync(0xffffffffu, dot[u], off);
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int j = p[u] - x.len;
                        if (p[u] >= 0 && (j < 0 || ((bits[r] >> j) & 1))) {
                            float vf[EPC];
                            unpack<DT>(vv[u], vf);
                            const float y = dot[u] * ksc[u];
                            const float mn = fmaxf(m[r], y), ms = safe(mn);
                            const float sc = exp2f(m[r] - ms);
                            const float pe = exp2f(y - ms);
                            l[r] = fmaf(l[r], sc, pe);
                            const float pv = pe * vsc[u];
#pragma unroll
                            for (int e = 0; e < EPC; ++e)
                                o[r][e] = fmaf(o[r][e], sc, pv * vf[e]);
                            m[r] = mn;
                        }
                    }
                }
            }
        }
        // the key groups of the warp, then the warps
#pragma unroll
        for (int r = 0; r < RM; ++r) {
            for (int off = lpk; off < 32; off <<= 1) {
                const float m2 = __shfl_xor_sync(0xffffffffu, m[r], off);
                const float l2 = __shfl_xor_sync(0xffffffffu, l[r], off);
                const float mn = fmaxf(m[r], m2), ms = safe(mn);
                const float s1 = exp2f(m[r] - ms), s2 = exp2f(m2 - ms);
                l[r] = l[r] * s1 + l2 * s2;
#pragma unroll
                for (int e = 0; e < EPC; ++e)
                    o[r][e] = o[r][e] * s1 + __shfl_xor_sync(0xffffffffu, o[r][e], off) * s2;
                m[r] = mn;
            }
            if (ks == 0) {
#pragma unroll
                for (int e = 0; e < EPC; ++e)
                    wo[warp][r][dc * EPC + e] = o[r][e];
            }
            if (lane == 0) {
                wm[warp][r] = m[r];
                wl[warp][r] = l[r];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < RM * D; i += kGenThreads) {
            const int r = i / D, d = i - r * D;
            float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
            for (int v = 0; v < kGenWarps; ++v)
                M = fmaxf(M, wm[v][r]);
            const float ms = safe(M);
#pragma unroll
            for (int v = 0; v < kGenWarps; ++v) {
                const float s = exp2f(wm[v][r] - ms);
                L += wl[v][r] * s;
                O += wo[v][r][d] * s;
            }
            so[i] = O;
            if (d == 0) {
                um[r] = M;
                ul[r] = L;
            }
        }
        __syncthreads();
        fin.part(a, run, x, [&](int r, int d) { return so[r * D + d]; }, um, ul);
    }
    fin.end(a, run, sm, um, ul, wgt);
}

template <int DT>
cudaError_t launch_gen(const KvAttnArgs &a, int grid, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kGenThreads);
    cfg.stream = st;
    return a.idx ? cudaLaunchKernelEx(&cfg, k_kv_attn<DT, true>, a)
                 : cudaLaunchKernelEx(&cfg, k_kv_attn<DT, false>, a);
}

}  // namespace

std::atomic<int> g_tree_variant{0};

// Tensor cores serve binary16 and 8-bit rows of 64 and 128 values: units of 8
// query rows on mma.sync, of 64 on tcgen05 (rows: the largest unit's).
KvPlan kv_plan(int dtype, int D, int rows)
{
    KvPlan p;
    p.mma = dtype != DV_F32 && (D == 64 || D == 128);
    p.rows = !p.mma ? kKvGenRows : rows <= 8 ? 8 : 64;
    return p;
}

// Whether units of 8 rows, which read the cache once for every 8, are the
// faster ones for more than 8 rows.  Measured (us, units of 8 / of 64): 768
// heads of 2112 positions of 128 values, 8 bits: 16 rows 169 / 173, 24 rows
// 244 / 177, 40 rows 395 / 185; binary16: 12 rows 256 / 147; 120 heads of 17
// tiles at most, 8 bits: 12 rows 24 / 38, 40 rows 37 / 47; binary16: 26 / 35,
// 42 / 45.  So a tile of 64 positions takes the units of 8 about 3.6 (8-bit)
// or 5.0 ns a pass over it and the units of 64 7.4 or 4.9 ns, and these take
// about 15 us longer to start and to end.  The lengths are known on the device only:
// the capacity stands for them.  What a unit costs beside its tiles is not in the
// rule: 1024 heads of 2 tiles, binary16, 12 rows: 51 / 77, and it takes the 77.
static bool kv_small_units(const KvAttnArgs &a)
{
    if (const int v = g_tree_variant.load())
        return v == 1;
    const int rows = a.T * (a.H / a.c.Hkv), passes = (rows + 7) / 8;
    const double tiles = (double)a.B * (a.u_h ? a.max_u_h : a.c.Hkv) * ((a.c.cap + 63) / 64);
    const bool i8 = a.c.dtype == DV_I8;
    return tiles * (passes * (i8 ? 3.6 : 5.0) - (i8 ? 7.4 : 4.9)) <= 15000;
}

cudaError_t launch_kv_attn(const KvAttnArgs &a, const KvPlan &p, int nsm, cudaStream_t st)
{
    if (p.mma)
        return p.rows == 8 || kv_small_units(a) ? launch_kv_mma(a, nsm, st)
                                                : launch_kv_tc(a, nsm, st);
    const int grid = nsm * 4 < kKvMaxCtas ? nsm * 4 : kKvMaxCtas;
    if (a.c.dtype == DV_I8)
        return launch_gen<DV_I8>(a, grid, st);
    if (a.c.dtype == DV_F16)
        return launch_gen<DV_F16>(a, grid, st);
    return launch_gen<DV_F32>(a, grid, st);
}

}  // namespace dv
