// dv_kv_write.cu -- writing a KV cache (quantising it, and keeping the mean
// key of every complete block), reading it back, and moving the rows of an
// accepted draft together (sm_103a).
#include "dv_kv.cuh"

namespace dv {
namespace {

constexpr int kWriteThreads = 256;  // (dv_kv_append: 128 for up to 64 rows)
constexpr int kReadRows = 2;  // rows a thread of dv_kv_read has in flight

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

// VEC values of a given row (F16: binary16 ones), as binary32.
template <int VEC, bool F16>
DV_DEV void ld_rows(const void *p, float (&x)[VEC])
{
    if (F16 && VEC >= 8) {
#pragma unroll
        for (int i = 0; i < VEC; i += 8) {
            const uint4 u = __ldg(reinterpret_cast<const uint4 *>(static_cast<const __half *>(p) + i));
            const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                x[i + 2 * k] = f.x;
                x[i + 2 * k + 1] = f.y;
            }
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
        float4 v;
        if (F16) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(static_cast<const __half *>(p) + i));
            const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&u.x));
            const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&u.y));
            v = make_float4(a.x, a.y, b.x, b.y);
        } else {
            v = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
        }
        x[i] = v.x;
        x[i + 1] = v.y;
        x[i + 2] = v.z;
        x[i + 3] = v.w;
    }
}

// VEC values of a row into the cache at p; a row is spread over lpr lanes
// (all of them call it, `on` or not).  Returns the row's scale (DV_I8).
template <int VEC, int DT>
DV_DEV float write_row(const float (&x)[VEC], typename Store<DT>::T *p, int lpr, bool on)
{
    if constexpr (DT == DV_I8) {
        float mx = amax_of(x);
        for (int k = lpr / 2; k > 0; k >>= 1)
            mx = amax2(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        const float s = quant_scale(mx);
        const float inv = quant_inv(s);
        unsigned w[VEC / 4];
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            w[i] = quant4(x + 4 * i, s, inv);  // (NaN where the row is not finite)
            w[i] = s == s ? w[i] : 0u;
        }
        if (on) {
            if constexpr (VEC == 16)
                *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            else
                *reinterpret_cast<unsigned *>(p) = w[0];
        }
        return s;
    } else if constexpr (DT == DV_F16) {
        unsigned w[VEC / 2];
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) {
            const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const unsigned *>(&h);
        }
        if (on) {
            if constexpr (VEC == 16) {
                reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
            } else {
                *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
            }
        }
    } else if (on) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
            *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
    return 0.f;
}

// One side (0 keys, 1 values) of the `rows` new rows of a tile: the given rows
// from token t0 of (b, h) on go to the cache rows from row0 on, by the threads
// from `first` on.  A row is spread over D / VEC lanes, and a lane group has
// UR rows in flight.
template <int VEC, int DT, bool F16, int UR, int NTHR>
DV_DEV void write_side(const KvAppendArgs &a, int side, int first, int b, int h, int t0, int rows,
                       size_t row0, float (&x)[UR][VEC])
{
    using T = typename Store<DT>::T;
    const KvCacheArgs &c = a.c;
    const int lpr = c.D / VEC, part = threadIdx.x % lpr;
    const int groups = (NTHR - first) / lpr, group = (threadIdx.x - first) / lpr;
    const KvRowsArgs &src = side ? a.v : a.k;
    const size_t es = F16 ? 2 : 4;
    const char *from = static_cast<const char *>(src.p) +
                       es * (b * src.sb + t0 * src.st + h * src.sh + part * VEC);
    const long long step = es * src.st;
    T *to = static_cast<T *>(side ? c.v : c.k) + row0 * c.D + part * VEC;
    float *scale = (side ? c.vs : c.ks) + row0;
    for (int u0 = group; u0 < rows + group; u0 += UR * groups) {
#pragma unroll
        for (int i = 0; i < UR; ++i) {
            const int u = u0 + i * groups;
            // (past the last row: that row once more, not written)
            ld_rows<VEC, F16>(from + min(u, rows - 1) * step, x[i]);
        }
#pragma unroll
        for (int i = 0; i < UR; ++i) {
            const int u = u0 + i * groups;
            const float s = write_row<VEC, DT>(x[i], to + (size_t)u * c.D, lpr, u < rows);
            if (DT == DV_I8 && u < rows && part == 0)
                scale[u] = s;
        }
    }
}

// One CTA owns the positions of one aligned tile of one (row, KV head): it
// writes the new tokens that fall into it and the means of the blocks that
// they complete.  A prompt of 8 x 96 heads x 2048 binary32 rows into 8 bits with
// blocks of 64: 367 us, 5.5 TB/s of the bytes it reads and writes (298 us at the
// copy rate); the rest is the means' second read of the codes.
template <int VEC, int DT, bool F16, int NTHR>
__global__ void __launch_bounds__(NTHR, 1024 / NTHR) k_kv_append(const KvAppendArgs a)
{
    constexpr int UR = VEC == 16 ? 2 : 4;
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
    const int rows = hi - lo;
    const size_t bh = (size_t)b * c.Hkv + h, row0 = bh * (size_t)c.cap + lo;
    float x[UR][VEC];
    write_side<VEC, DT, F16, UR, NTHR>(a, 0, 0, b, h, lo - len, rows, row0, x);
    // blocks whose last position is among the new ones: up to half of the warps
    // take their means from the cache while the others write the values
    const int j0 = c.block ? lo / c.block : 0, means = c.block ? hi / c.block - j0 : 0;
    const int takers = min(means, NTHR / 64);
    if (means > 0) {
        __syncthreads();
        const int warp = threadIdx.x >> 5;
        if (warp < takers) {
            for (int j = warp; j < means; j += takers)
                warp_mean<DT>(c, bh, j0 + j);
            return;
        }
    }
    write_side<VEC, DT, F16, UR, NTHR>(a, 1, 32 * takers, b, h, lo - len, rows, row0, x);
}

// VEC cached values as numbers, without their scale.
template <int VEC, int DT>
DV_DEV void ld_values(const typename Store<DT>::T *p, float (&f)[VEC])
{
    if constexpr (DT == DV_I8) {
        static_assert(VEC == 8, "half a 16-byte chunk");
        const uint2 u = __ldcs(reinterpret_cast<const uint2 *>(p));
        float g[16];
        Store<DV_I8>::unpack(make_uint4(u.x, u.y, 0x80808080u, 0x80808080u), g);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            f[i] = g[i];
    } else {
        ld_rows<VEC, DT == DV_F16>(p, f);
    }
}

// VEC values per thread of UR rows, keys and values.  That prompt back as
// binary16: 242 us, 5.0 TB/s (180 us at the copy rate), waiting for its loads;
// 4 and 8 rows in flight a thread took 335 and 529 us.
template <int VEC, int DT, bool F16>
__global__ void __launch_bounds__(kWriteThreads) k_kv_read(const KvReadArgs a)
{
    constexpr int UR = kReadRows;
    using T = typename Store<DT>::T;
    const KvCacheArgs &c = a.c;
    const int lpr = c.D / VEC, rows = kWriteThreads / lpr;
    const int BH = a.B * c.Hkv, bhi = blockIdx.x % BH;
    const int b = bhi / c.Hkv, h = bhi % c.Hkv;
    const int s0 = __ldg(a.start + b);
    if (s0 < 0 || s0 > c.cap - a.T) {
        if (threadIdx.x == 0)
            set_status(a.status, DV_ERR_DEVICE_INDEX);
        return;
    }
    const size_t bh = (size_t)b * c.Hkv + h;
    const int t0 = blockIdx.x / BH * (UR * rows) + threadIdx.x / lpr;
    const int d = (threadIdx.x % lpr) * VEC;
    float x[UR][2][VEC], s[UR][2];
#pragma unroll
    for (int i = 0; i < UR; ++i) {
        if (t0 + i * rows >= a.T)
            break;
        const size_t row = bh * (size_t)c.cap + s0 + t0 + i * rows;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            ld_values<VEC, DT>(static_cast<const T *>(k ? c.v : c.k) + row * c.D + d, x[i][k]);
            s[i][k] = DT == DV_I8 ? __ldg((k ? c.vs : c.ks) + row) : 1.f;
        }
    }
#pragma unroll
    for (int i = 0; i < UR; ++i) {
        if (t0 + i * rows >= a.T)
            break;
        const size_t o = (bh * (size_t)a.T + t0 + i * rows) * c.D + d;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            void *dst = k ? a.v_out : a.k_out;
            if (DT == DV_I8) {
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    x[i][k][e] *= s[i][k];
            }
            if (F16) {
                unsigned u[VEC / 2];
#pragma unroll
                for (int e = 0; e < VEC / 2; ++e) {
                    const __half2 hh = __floats2half2_rn(x[i][k][2 * e], x[i][k][2 * e + 1]);
                    u[e] = *reinterpret_cast<const unsigned *>(&hh);
                }
                __half *q = static_cast<__half *>(dst) + o;
                if constexpr (VEC >= 8) {
#pragma unroll
                    for (int e = 0; e < VEC / 8; ++e)
                        __stcs(reinterpret_cast<uint4 *>(q) + e,
                               make_uint4(u[4 * e], u[4 * e + 1], u[4 * e + 2], u[4 * e + 3]));
                } else {
                    __stcs(reinterpret_cast<uint2 *>(q), make_uint2(u[0], u[1]));
                }
            } else {
#pragma unroll
                for (int e = 0; e < VEC; e += 4)
                    __stcs(reinterpret_cast<float4 *>(static_cast<float *>(dst) + o + e),
                           make_float4(x[i][k][e], x[i][k][e + 1], x[i][k][e + 2],
                                       x[i][k][e + 3]));
            }
        }
    }
}

// One CTA per (row, KV head) and side (0 keys, 1 values): row len + path[i]
// moves to len + i.  path ascends, so path[i] >= i and a chunk of rows, read
// whole before it is written, never overwrites a row that a later chunk
// reads.
__global__ void __launch_bounds__(kWriteThreads) k_kv_keep(const KvKeepArgs a)
{
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
    if (c.block && side == 0) {  // the blocks that the kept span completes, a warp each
        __syncthreads();
        for (int j = len / c.block + (int)(threadIdx.x >> 5); (j + 1) * c.block <= len + n;
             j += kWriteThreads / 32) {
            if (c.dtype == DV_I8)
                warp_mean<DV_I8>(c, bh, j);
            else if (c.dtype == DV_F16)
                warp_mean<DV_F16>(c, bh, j);
            else
                warp_mean<DV_F32>(c, bh, j);
        }
    }
}

template <class K, class A>
cudaError_t launch(K kern, dim3 grid, const A &a, cudaStream_t st, int threads = kWriteThreads)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int VEC, int DT>
cudaError_t append_src(const KvAppendArgs &a, dim3 grid, cudaStream_t st)
{
    // a CTA's rows: more CTAs of fewer threads where they are few
    const int rows = a.T < a.tile ? a.T : a.tile;
    if (rows <= 64)
        return a.k.f16 ? launch(k_kv_append<VEC, DT, true, 128>, grid, a, st, 128)
                       : launch(k_kv_append<VEC, DT, false, 128>, grid, a, st, 128);
    return a.k.f16 ? launch(k_kv_append<VEC, DT, true, 256>, grid, a, st, 256)
                   : launch(k_kv_append<VEC, DT, false, 256>, grid, a, st, 256);
}

// (rows of fewer than 16 values are binary32 or binary16 ones)
template <int VEC>
cudaError_t append_dt(const KvAppendArgs &a, dim3 grid, cudaStream_t st)
{
    if (a.c.dtype == DV_F32)
        return append_src<VEC, DV_F32>(a, grid, st);
    if (a.c.dtype == DV_F16 || VEC < 16)
        return append_src<VEC, DV_F16>(a, grid, st);
    return append_src<VEC, VEC < 16 ? DV_F16 : DV_I8>(a, grid, st);
}

template <int VEC, int DT>
cudaError_t read_out(const KvReadArgs &a, dim3 grid, cudaStream_t st)
{
    return a.f16 ? launch(k_kv_read<VEC, DT, true>, grid, a, st)
                 : launch(k_kv_read<VEC, DT, false>, grid, a, st);
}

template <int VEC>
cudaError_t read_dt(const KvReadArgs &a, dim3 grid, cudaStream_t st)
{
    if (a.c.dtype == DV_F32)
        return read_out<VEC, DV_F32>(a, grid, st);
    if (a.c.dtype == DV_F16 || VEC < 8)
        return read_out<VEC, DV_F16>(a, grid, st);
    return read_out<VEC, VEC < 8 ? DV_F16 : DV_I8>(a, grid, st);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t st)
{
    // the aligned tiles that T positions at any offset can touch
    const int tiles = (a.T + a.tile - 2) / a.tile + 1;
    const dim3 grid(tiles * a.B * a.c.Hkv);
    return a.c.D >= 16 ? append_dt<16>(a, grid, st) : append_dt<4>(a, grid, st);
}

cudaError_t launch_kv_read(const KvReadArgs &a, cudaStream_t st)
{
    const int vec = a.c.D >= 8 ? 8 : 4, rows = kReadRows * (kWriteThreads / (a.c.D / vec));
    const dim3 grid((a.T + rows - 1) / rows * a.B * a.c.Hkv);
    return vec == 8 ? read_dt<8>(a, grid, st) : read_dt<4>(a, grid, st);
}

cudaError_t launch_kv_keep(const KvKeepArgs &a, cudaStream_t st)
{
    return launch(k_kv_keep, dim3(a.B * a.c.Hkv, 2), a, st);
}

}  // namespace dv
