// dv_seq_attn.cu -- causal attention of packed sequences on CUDA cores
// (sm_103a): binary32 rows, and binary16 rows of other sizes than the tensor
// cores' 64 and 128.
//
// A unit of 32 query rows meets tiles of 64 positions.  Eight threads share a
// row: each forms the scores of every eighth position (products over D from
// shared memory, one 16-byte read for four to sixteen multiply-adds) and sums an
// eighth of the output's dimensions.  One pass, with the running maximum and sum
// of the softmax in registers.  Bound by shared-memory reads and arithmetic.
#include "dv_seq_sched.cuh"

namespace dv {
namespace {

constexpr int RM = kSeqGenRows, TP = kSeqGenTile;
using Sched = SeqSched<TP, false, 1, 4>;

template <typename T>
DV_DEV void ld4(const T *p, float (&x)[4])
{
    if constexpr (sizeof(T) == 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&v.x));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&v.y));
        x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
    }
}
template <typename T>
DV_DEV void st_one(T *p, float x) { *p = Elem<T>::from_float(x); }

template <typename T, int D>
struct GenSmem {
    static constexpr int LD = D + 4, LP = TP + 4;
    static constexpr size_t BYTES = ((size_t)(RM + 2 * TP) * LD + RM * LP) * 4;
};

template <typename T, int D>
__global__ void __launch_bounds__(256) k_seq_attn(const SeqAttnArgs a)
{
    using S = GenSmem<T, D>;
    constexpr int LD = S::LD, LP = S::LP, OC = D / 8;  // output values a thread
    extern __shared__ __align__(16) float smem[];
    __shared__ SeqSmem ss;
    __shared__ int s_last;
    float *const sq = smem, *const sk = sq + RM * LD, *const sv = sk + TP * LD, *const sp = sv + TP * LD;
    const int tid = threadIdx.x, r = tid >> 3, j8 = tid & 7;
    const SeqRun run = Sched::init(a, ss);
    Sched::Walk walk;
    Sched::Piece x;
    walk.start(a, run);
    while (walk.next(a, run, x)) {
        const int nrows = x.ntok * a.group, ctx = x.pos + x.ntok;
        __syncthreads();
        for (int i = tid; i < RM * (D / 4); i += 256) {
            const int row = i / (D / 4), c = i % (D / 4) * 4;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (row < nrows)
                ld4(static_cast<const T *>(a.q.p) + (long long)(x.tok + row / a.group) * a.q.st +
                        (x.h0 + row % a.group) * a.q.sh + c,
                    v);
            *reinterpret_cast<float4 *>(sq + row * LD + c) = make_float4(v[0], v[1], v[2], v[3]);
        }
        // positions up to lim; nothing for rows of no token
        const int lim = r < nrows ? x.pos + r / a.group : -1;
        float m = -INFINITY, l = 0.f, o[OC];
#pragma unroll
        for (int e = 0; e < OC; ++e)
            o[e] = 0.f;
        for (int k = x.k0; k < x.k1; ++k) {
            const int p0 = k * TP;
            __syncthreads();
            for (int i = tid; i < TP * (D / 4); i += 256) {
                const int row = i / (D / 4), c = i % (D / 4) * 4, p = p0 + row;
                float kk[4] = {0.f, 0.f, 0.f, 0.f}, vv[4] = {0.f, 0.f, 0.f, 0.f};
                if (p < ctx) {
                    if (a.pk) {
                        const int pg = __ldg(a.tables + (long long)x.b * a.width + p / a.page);
                        if ((unsigned)pg < (unsigned)a.n_pages) {
                            const long long at =
                                (((long long)pg * a.Hkv + x.hkv) * a.page + p % a.page) * D + c;
                            ld4(static_cast<const T *>(a.pk) + at, kk);
                            ld4(static_cast<const T *>(a.pv) + at, vv);
                        } else {
                            set_status(a.status, DV_ERR_DEVICE_INDEX);
                        }
                    } else {
                        const long long t = x.tok - x.pos + p;  // (the request's first row + p)
                        ld4(static_cast<const T *>(a.k.p) + t * a.k.st + x.hkv * a.k.sh + c, kk);
                        ld4(static_cast<const T *>(a.v.p) + t * a.v.st + x.hkv * a.v.sh + c, vv);
                    }
                }
                *reinterpret_cast<float4 *>(sk + row * LD + c) =
                    make_float4(kk[0], kk[1], kk[2], kk[3]);
                *reinterpret_cast<float4 *>(sv + row * LD + c) =
                    make_float4(vv[0], vv[1], vv[2], vv[3]);
            }
            __syncthreads();
            if (lim < p0)  // (the same for a row's eight threads)
                continue;
            float s[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s[e] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                const float4 q = *reinterpret_cast<const float4 *>(sq + r * LD + c);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float4 kk =
                        *reinterpret_cast<const float4 *>(sk + (j8 + 8 * e) * LD + c);
                    s[e] = fmaf(q.x, kk.x, s[e]);
                    s[e] = fmaf(q.y, kk.y, s[e]);
                    s[e] = fmaf(q.z, kk.z, s[e]);
                    s[e] = fmaf(q.w, kk.w, s[e]);
                }
            }
            const unsigned octet = 0xffu << (tid & 24);
            float top = -INFINITY;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[e] = p0 + j8 + 8 * e <= lim ? s[e] * a.scale : -INFINITY;
                top = fmaxf(top, s[e]);
            }
#pragma unroll
            for (int w = 1; w < 8; w <<= 1)
                top = fmaxf(top, __shfl_xor_sync(octet, top, w));
            const float mn = fmaxf(m, top), ms = mn == -INFINITY ? 0.f : mn;
            const float f = exp2f(m - ms);
            m = mn;
            l *= f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float p = exp2f(s[e] - ms);
                l += p;
                sp[r * LP + j8 + 8 * e] = p;
            }
            __syncwarp(octet);
#pragma unroll
            for (int e = 0; e < OC; ++e)
                o[e] *= f;
            // (an unseen value row may hold anything)
            const int seen = min(TP, lim - p0 + 1);
            int i = 0;
            for (; i + 4 <= seen; i += 4) {
                const float4 p4 = *reinterpret_cast<const float4 *>(sp + r * LP + i);
                const float w4[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < OC; ++e)
                        o[e] = fmaf(w4[u], sv[(i + u) * LD + j8 * OC + e], o[e]);
            }
            for (; i < seen; ++i)
#pragma unroll
                for (int e = 0; e < OC; ++e)
                    o[e] = fmaf(sp[r * LP + i], sv[i * LD + j8 * OC + e], o[e]);
            __syncwarp(octet);
        }
#pragma unroll
        for (int w = 1; w < 8; w <<= 1)
            l += __shfl_xor_sync(0xffffffffu, l, w);
        T *const out = static_cast<T *>(a.out) +
                       ((long long)(x.tok + (r < nrows ? r / a.group : 0)) * a.H + x.h0 +
                        (r < nrows ? r % a.group : 0)) * D + j8 * OC;
        if (x.c0 == x.c1) {
            const float f = l == 0.f ? 0.f : 1.f / l;
            if (r < nrows)
#pragma unroll
                for (int e = 0; e < OC; ++e)
                    st_one(out + e, o[e] * f);
            continue;
        }
        // a piece of a unit that other runs share; the last to leave one merges
        constexpr size_t REC = (size_t)RM * (D + 2);
        float *rec = a.rec + Sched::slot(run.c, x.c0) * REC;
        if (r < nrows) {
#pragma unroll
            for (int e = 0; e < OC; ++e)
                __stcg(rec + r * D + j8 * OC + e, o[e]);
            if (j8 == 0) {
                __stcg(rec + RM * D + r, m);
                __stcg(rec + RM * (D + 1) + r, l);
            }
        }
        __threadfence();
        __syncthreads();
        if (tid == 0) {
            s_last = atomicAdd(a.cnt + x.c0, 1) == x.c1 - x.c0;
            if (s_last)
                a.cnt[x.c0] = 0;
            __threadfence();
        }
        __syncthreads();
        if (s_last && r < nrows) {
            float M = -INFINITY, L = 0.f;
            for (int c = x.c0; c <= x.c1; ++c)
                M = fmaxf(M, ld_cg(a.rec + Sched::slot(c, x.c0) * REC + RM * D + r));
            const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int e = 0; e < OC; ++e)
                o[e] = 0.f;
            for (int c = x.c0; c <= x.c1; ++c) {
                const float *p = a.rec + Sched::slot(c, x.c0) * REC;
                const float f = exp2f(ld_cg(p + RM * D + r) - ms);
                L = fmaf(ld_cg(p + RM * (D + 1) + r), f, L);
#pragma unroll
                for (int e = 0; e < OC; ++e)
                    o[e] = fmaf(ld_cg(p + r * D + j8 * OC + e), f, o[e]);
            }
            const float f = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
            for (int e = 0; e < OC; ++e)
                st_one(out + e, o[e] * f);
        }
    }
}

template <typename T, int D>
cudaError_t launch_gen(SeqAttnArgs a, int nsm, cudaStream_t st)
{
    seq_group(a, RM);
    auto kern = k_seq_attn<T, D>;
    constexpr size_t smem = GenSmem<T, D>::BYTES;
    static DeviceOnce once;
    cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess)
        return e;
    // (the runs and their order of sums follow the device alone)
    constexpr int per_sm = smem > 110 * 1024 ? 1 : smem > 70 * 1024 ? 2 : 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nsm * per_sm < kSeqMaxCtas ? nsm * per_sm : kSeqMaxCtas);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename T>
cudaError_t launch_type(const SeqAttnArgs &a, int nsm, cudaStream_t st)
{
    constexpr bool HALF = sizeof(T) == 2;  // (64 and 128 of them are the tensor cores')
    switch (a.D) {
    case 8: return launch_gen<T, 8>(a, nsm, st);
    case 16: return launch_gen<T, 16>(a, nsm, st);
    case 32: return launch_gen<T, 32>(a, nsm, st);
    case HALF ? 256 : 64: return launch_gen<T, HALF ? 256 : 64>(a, nsm, st);
    case 128:
        if constexpr (!HALF)
            return launch_gen<T, 128>(a, nsm, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_seq_attn(const SeqAttnArgs &a, int nsm, cudaStream_t st)
{
    return a.f16 ? launch_type<__half>(a, nsm, st) : launch_type<float>(a, nsm, st);
}

size_t seq_attn_record_bytes(int D)
{
    return 2 * (size_t)kSeqMaxCtas * kSeqGenRows * (D + 2) * 4;
}

}  // namespace dv
