// dv_kv_topk.cu -- the blocks of cached positions that a query attends to,
// chosen by a cheap score (sm_103a).
//
// The query is quantised as a row (codes qc); block j's quantised mean key
// has codes mc_j and scale m_j.  Its score is float(sum_d qc_d mc_jd) m_j:
// the sum is a whole number below 2^24, so the score is one rounded product
// and does not depend on any order of summation (the query's own scale is
// positive and common to all blocks).  The first n_first and last n_last
// blocks are always taken; of the others the best scores, ties to the lower
// block.
//
// One CTA per (row, query head): the means of a head (D bytes a block, 1/64
// of the 8-bit keys at blocks of 64) are read once with 16-byte loads and
// multiplied four codes at a time (dp4a); the scores stay in shared memory
// as order-preserving keys, and four 8-bit digits of a radix selection find
// the k-th.  32 rows of up to 8000 positions in blocks of 32, 64 heads: 25 us,
// 512 blocks in one CTA 12 us, both bound by the passes' barriers (one warp a
// row without any took 32 and 45 us for the former).
#include "dv_kv.cuh"

namespace dv {
namespace {

constexpr int kTopkThreads = 256;

__global__ void __launch_bounds__(kTopkThreads) k_kv_topk(const KvTopkArgs a)
{
    extern __shared__ unsigned keys[];
    __shared__ float red[33];
    __shared__ __align__(16) int8_t qc[256];
    __shared__ int hist[256];
    __shared__ int scan[33];
    __shared__ int s_digit, s_need;
    const KvCacheArgs &c = a.c;
    const int D = c.D, n = c.block, tid = threadIdx.x;
    const int b = blockIdx.x / a.H, h = blockIdx.x % a.H;
    int32_t *out = a.idx + (size_t)blockIdx.x * a.k;
    const int len = __ldg(a.lens + b);
    if (len < 0 || len > c.cap) {
        if (tid == 0)
            set_status(a.status, DV_ERR_DEVICE_INDEX);
        return;
    }
    const int nb = (int)(((long long)len + n - 1) / n);
    if (nb <= a.k) {  // every block
        for (int i = tid; i < a.k; i += kTopkThreads)
            out[i] = i < nb ? i : -1;
        return;
    }
    // the query's codes
    const float x = tid < D ? ld_row(a.q, b * a.q.sb + h * a.q.sh + tid) : 0.f;
    const float s = quant_scale(block_amax(fabsf(x), red));
    if (tid < D) {
        float v[4] = {x, 0.f, 0.f, 0.f};
        qc[tid] = s == s ? (int8_t)quant4(v, s, quant_inv(s)) : (int8_t)0;
    }
    __syncthreads();
    // scores of the blocks that are not taken anyway (complete ones: the
    // last block, the only one that may not be, is among the n_last)
    const int m = nb - a.n_first - a.n_last, want = a.k - a.n_first - a.n_last;
    const int cpr = D / 16, per = kTopkThreads / cpr;  // 16-byte chunks of a row; rows per step
    const size_t row0 = ((size_t)b * c.Hkv + h / (a.H / c.Hkv)) * (size_t)(c.cap / n) + a.n_first;
    const int part = tid % cpr;
    const int4 q4 = reinterpret_cast<const int4 *>(qc)[part];
    constexpr int UN = 8;  // rows in flight per lane group
    for (int j0 = tid / cpr; j0 < m + tid / cpr; j0 += UN * per) {
        int4 v[UN];
        float ms[UN];
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int j = j0 + i * per;
            v[i] = j < m ? __ldg(reinterpret_cast<const int4 *>(c.mean + (row0 + j) * D) + part)
                         : make_int4(0, 0, 0, 0);
            ms[i] = j < m ? __ldg(c.mean_scale + row0 + j) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < UN; ++i) {
            const int j = j0 + i * per;
            int dot = __dp4a(v[i].x, q4.x,
                             __dp4a(v[i].y, q4.y, __dp4a(v[i].z, q4.z, __dp4a(v[i].w, q4.w, 0))));
            for (int o = cpr / 2; o > 0; o >>= 1)
                dot += __shfl_xor_sync(0xffffffffu, dot, o);
            if (j < m && part == 0)
                keys[j] = score_key(ms[i] == INFINITY ? INFINITY : (float)dot * ms[i]);
        }
    }
    __syncthreads();
    // the want-th largest key, digit by digit
    unsigned prefix = 0;
    int need = want;  // still to take among the keys that share the prefix
    if (want > 0)
        for (int shift = 24; shift >= 0; shift -= 8) {
            hist[tid] = 0;
            __syncthreads();
            const unsigned above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int j = tid; j < m; j += kTopkThreads)
                if ((keys[j] & above) == prefix)
                    atomicAdd(&hist[(keys[j] >> shift) & 255], 1);
            __syncthreads();
            // thread t holds digit 255 - t: a prefix sum counts from the top
            const int cnt = hist[255 - tid];
            int total;
            const int before = block_excl_scan(cnt, scan, &total);
            if (before < need && need <= before + cnt) {
                s_digit = 255 - tid;
                s_need = need - before;
            }
            __syncthreads();
            prefix |= (unsigned)s_digit << shift;
            need = s_need;
            __syncthreads();
        }
    // ascending: every key above the k-th, and the first `need` equal to it
    for (int i = tid; i < a.n_first; i += kTopkThreads)
        out[i] = i;
    for (int i = tid; i < a.n_last; i += kTopkThreads)
        out[a.k - a.n_last + i] = nb - a.n_last + i;
    if (want > 0) {
        const int len_t = (m + kTopkThreads - 1) / kTopkThreads;
        const int j0 = min(m, tid * len_t), j1 = min(m, j0 + len_t);
        int over = 0, same = 0, total;
        for (int j = j0; j < j1; ++j) {
            over += keys[j] > prefix;
            same += keys[j] == prefix;
        }
        int same_before = block_excl_scan(same, scan, &total);
        const int over_before = block_excl_scan(over, scan, &total);
        int at = a.n_first + over_before + min(same_before, need);
        for (int j = j0; j < j1; ++j) {
            const bool eq = keys[j] == prefix;
            if (keys[j] > prefix || (eq && same_before < need))
                out[at++] = a.n_first + j;
            same_before += eq;
        }
    }
}

}  // namespace

cudaError_t launch_kv_topk(const KvTopkArgs &a, cudaStream_t st)
{
    static DeviceOnce once;
    cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(k_kv_topk, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    kKvMaxBlocks * 4);
    });
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.B * a.H);
    cfg.blockDim = dim3(kTopkThreads);
    cfg.dynamicSmemBytes = (size_t)(a.c.cap / a.c.block + 1) * 4;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, k_kv_topk, a);
}

}  // namespace dv
