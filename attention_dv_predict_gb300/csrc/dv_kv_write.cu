// dv_kv_write.cu -- writing a KV cache (quantising it, and keeping the mean
// key of every complete block), reading it back, and moving the rows of an
// accepted draft together (sm_103a).
#include "dv_kv.cuh"

namespace dv {
namespace {

constexpr int kWriteThreads = 256;

// Count of new tokens of row b, 0 and a recorded fault where its position or
// count is out of range.
DV_DEV int row_tokens(const int32_t *lens, const int32_t *n_tok, int b, int T, int cap,
                      int *status, int *len)
{
    const int l = __ldg(lens + b), n = n_tok ? __ldg(n_tok + b) : T;
    *len = l;
    if (l < 0 || n < 0 || n > T || l > cap - n) {
        if (threadIdx.x == 0)
            set_status(status, DV_ERR_DEVICE_INDEX);
        return 0;
    }
    return n;
}

// One warp writes one cached row from one given row.
DV_DEV void write_row(const KvCacheArgs &c, const KvRowsArgs &src, long long at, void *dst,
                      float *scale, size_t row, int lane)
{
    float4 x[2];
    float mx = 0.f;
    const int D = c.D;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int d = (lane + 32 * i) * 4;
        x[i] = d < D ? ld_row4(src, at + d) : make_float4(0.f, 0.f, 0.f, 0.f);
        mx = amax2(mx, amax2(amax2(x[i].x, x[i].y), amax2(x[i].z, x[i].w)));
    }
    if (c.dtype == DV_I8) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mx = amax2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float s = quant_scale(mx);
        const bool fine = s == s;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int d = (lane + 32 * i) * 4;
            if (d < D)
                *reinterpret_cast<unsigned *>(static_cast<int8_t *>(dst) + row * D + d) =
                    fine ? pack_codes(quant_code(x[i].x, s), quant_code(x[i].y, s),
                                      quant_code(x[i].z, s), quant_code(x[i].w, s))
                         : 0u;
        }
        if (lane == 0)
            scale[row] = s;
        return;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int d = (lane + 32 * i) * 4;
        if (d >= D)
            continue;
        if (c.dtype == DV_F32) {
            *reinterpret_cast<float4 *>(static_cast<float *>(dst) + row * D + d) = x[i];
        } else {
            __half2 h[2] = {__floats2half2_rn(x[i].x, x[i].y), __floats2half2_rn(x[i].z, x[i].w)};
            *reinterpret_cast<uint2 *>(static_cast<__half *>(dst) + row * D + d) =
                *reinterpret_cast<uint2 *>(h);
        }
    }
}

// One CTA owns the positions of one aligned tile (a block, where means are
// kept) of one (row, KV head): it writes the new tokens that fall into it
// and, when the tile's last position is among them, the block's mean.
__global__ void __launch_bounds__(kWriteThreads) k_kv_append(const KvAppendArgs a)
{
    __shared__ MeanSmem sm;
    const KvCacheArgs &c = a.c;
    const int BH = a.B * c.Hkv, bhi = blockIdx.x % BH;  // neighbouring heads together:
    const int b = bhi / c.Hkv, h = bhi % c.Hkv;         // their given rows lie side by side
    int len;
    const int n = row_tokens(a.lens, a.n_tok, b, a.T, c.cap, a.status, &len);
    if (n == 0)
        return;
    const int tile = len / a.tile + blockIdx.x / BH;
    const int lo = max(len, tile * a.tile), hi = min(len + n, (tile + 1) * a.tile);
    if (lo >= hi)
        return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t bh = (size_t)b * c.Hkv + h;
    for (int u = warp; u < 2 * (hi - lo); u += kWriteThreads / 32) {
        const int p = lo + (u >> 1);
        const KvRowsArgs &src = (u & 1) ? a.v : a.k;
        const long long at = b * src.sb + (long long)(p - len) * src.st + h * src.sh;
        write_row(c, src, at, (u & 1) ? c.v : c.k, (u & 1) ? c.vs : c.ks,
                  bh * (size_t)c.cap + p, lane);
    }
    if (c.block && hi == (tile + 1) * a.tile) {
        __syncthreads();
        block_mean(c, bh, tile, sm);
    }
}

// Four values per thread.
__global__ void __launch_bounds__(kWriteThreads) k_kv_read(const KvReadArgs a)
{
    const KvCacheArgs &c = a.c;
    const int lpr = c.D / 4, rows = kWriteThreads / lpr;
    const int BH = a.B * c.Hkv, bhi = blockIdx.x % BH;
    const int b = bhi / c.Hkv, h = bhi % c.Hkv;
    const int s0 = __ldg(a.start + b);
    if (s0 < 0 || s0 > c.cap - a.T) {
        if (threadIdx.x == 0)
            set_status(a.status, DV_ERR_DEVICE_INDEX);
        return;
    }
    const size_t bh = (size_t)b * c.Hkv + h;
    const int t = blockIdx.x / BH * rows + threadIdx.x / lpr, d = (threadIdx.x % lpr) * 4;
    if (t >= a.T)
        return;
    const size_t row = bh * (size_t)c.cap + s0 + t;
    const size_t o = (bh * (size_t)a.T + t) * c.D + d;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float4 x = ld_cached4(i ? c.v : c.k, c.dtype, row * c.D + d);
        if (c.dtype == DV_I8) {
            const float s = (i ? c.vs : c.ks)[row];
            x = make_float4(x.x * s, x.y * s, x.z * s, x.w * s);
        }
        void *dst = i ? a.v_out : a.k_out;
        if (a.f16) {
            __half2 hh[2] = {__floats2half2_rn(x.x, x.y), __floats2half2_rn(x.z, x.w)};
            *reinterpret_cast<uint2 *>(static_cast<__half *>(dst) + o) =
                *reinterpret_cast<uint2 *>(hh);
        } else {
            *reinterpret_cast<float4 *>(static_cast<float *>(dst) + o) = x;
        }
    }
}

// One CTA per (row, KV head) and side (0 keys, 1 values): row len + path[i]
// moves to len + i.  path ascends, so path[i] >= i and a chunk of rows, read
// whole before it is written, never overwrites a row that a later chunk
// reads.
__global__ void __launch_bounds__(kWriteThreads) k_kv_keep(const KvKeepArgs a)
{
    __shared__ MeanSmem sm;
    __shared__ int path[DV_TREE_MAX_TOKENS];
    __shared__ int bad;
    const KvCacheArgs &c = a.c;
    const int b = blockIdx.x / c.Hkv, h = blockIdx.x % c.Hkv, side = blockIdx.y;
    const int len = __ldg(a.lens + b), n = __ldg(a.n_keep + b);
    if (threadIdx.x == 0)
        bad = len < 0 || n < 0 || n > a.T || len > c.cap - n;
    __syncthreads();
    if (!bad && (int)threadIdx.x < n) {
        const int p = __ldg(a.path + (size_t)b * a.T + threadIdx.x);
        const int before = threadIdx.x ? __ldg(a.path + (size_t)b * a.T + threadIdx.x - 1) : -1;
        path[threadIdx.x] = p;
        if (p <= before || p >= a.T || p >= c.cap - len)
            bad = 1;  // (every writer stores the same value)
    }
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0)
            set_status(a.status, DV_ERR_DEVICE_INDEX);
        return;
    }
    const size_t bh = (size_t)b * c.Hkv + h, p0 = bh * (size_t)c.cap + len;
    const int es = c.dtype == DV_I8 ? 1 : (c.dtype == DV_F16 ? 2 : 4);
    const int cpr = c.D * es / 16, rows = kWriteThreads / cpr;
    uint4 *buf = static_cast<uint4 *>(side ? c.v : c.k);
    for (int i0 = 0; i0 < n; i0 += rows) {
        const int i = i0 + threadIdx.x / cpr, d = threadIdx.x % cpr;
        const bool move = i < n && (int)threadIdx.x < rows * cpr && path[i] != i;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (move)
            x = __ldcg(buf + (p0 + path[i]) * cpr + d);
        __syncthreads();
        if (move)
            buf[(p0 + i) * cpr + d] = x;
        __syncthreads();
    }
    if (c.dtype == DV_I8) {  // one scale per thread (n <= 64)
        float *s = side ? c.vs : c.ks;
        const bool move = (int)threadIdx.x < n && path[threadIdx.x] != (int)threadIdx.x;
        const float x = move ? __ldcg(s + p0 + path[threadIdx.x]) : 0.f;
        __syncthreads();
        if (move)
            s[p0 + threadIdx.x] = x;
    }
    if (c.block && side == 0)
        for (int j = len / c.block; (j + 1) * c.block <= len + n; ++j) {
            __syncthreads();
            block_mean(c, bh, j, sm);
        }
}

template <class K, class A>
cudaError_t launch(K kern, dim3 grid, const A &a, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kWriteThreads);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t st)
{
    // the aligned tiles that T positions at any offset can touch
    const int tiles = (a.T + a.tile - 2) / a.tile + 1;
    return launch(k_kv_append, dim3(tiles * a.B * a.c.Hkv), a, st);
}

cudaError_t launch_kv_read(const KvReadArgs &a, cudaStream_t st)
{
    const int rows = kWriteThreads / (a.c.D / 4);
    return launch(k_kv_read, dim3((a.T + rows - 1) / rows * a.B * a.c.Hkv), a, st);
}

cudaError_t launch_kv_keep(const KvKeepArgs &a, cudaStream_t st)
{
    return launch(k_kv_keep, dim3(a.B * a.c.Hkv, 2), a, st);
}

}  // namespace dv
