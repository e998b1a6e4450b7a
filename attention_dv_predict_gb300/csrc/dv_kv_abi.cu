// dv_kv_abi.cu -- C entry points of the KV-cache operators: argument checks
// and workspace layout.  See include/dv.h.
#include <climits>
#include <cmath>
#include <cstring>
#include <mutex>

#include <cudaTypedefs.h>

#include "dv_kv.h"

using namespace dv;

namespace {

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int esize(int dtype) { return dtype == DV_I8 ? 1 : (dtype == DV_F16 ? 2 : 4); }
bool aligned(const void *p, size_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
dv_status cuda_status(cudaError_t e) { return cuda_failed(e) ? DV_ERR_CUDA : DV_OK; }

dv_status check_desc(const dv_kv_desc *D)
{
    if (!D)
        return DV_ERR_INVALID_ARG;
    if (D->n_heads <= 0 || D->n_kv_heads <= 0 || D->n_heads % D->n_kv_heads || D->head_dim <= 0 ||
        D->kv_cap <= 0)
        return DV_ERR_INVALID_ARG;
    if (D->dtype != DV_F32 && D->dtype != DV_F16 && D->dtype != DV_I8)
        return DV_ERR_INVALID_ARG;
    if (D->block < 0 || (D->block > 0 && D->kv_cap < D->block))
        return DV_ERR_INVALID_ARG;
    const int d = D->head_dim, hb = d * esize(D->dtype);
    if ((d & (d - 1)) || d > 256 || hb < 16 || hb > 512 || D->n_heads > 256)
        return DV_ERR_UNSUPPORTED;
    if (D->block > 0 && ((D->block != 16 && D->block != 32 && D->block != 64 && D->block != 128) ||
                         D->kv_cap / D->block >= kKvMaxBlocks || d < 16))
        return DV_ERR_UNSUPPORTED;
    if (D->kv_cap > (1 << 28))
        return DV_ERR_UNSUPPORTED;
    return DV_OK;
}

dv_status check_cache(const dv_kv_desc &D, const dv_kv_cache *c, int batch, KvCacheArgs *a)
{
    if (!c || !aligned(c->k, 16) || !aligned(c->v, 16) || batch < 1 || batch > DV_KV_MAX_BATCH)
        return DV_ERR_INVALID_ARG;
    if (D.dtype == DV_I8 && (!aligned(c->k_scale, 4) || !aligned(c->v_scale, 4)))
        return DV_ERR_INVALID_ARG;
    if (D.block && (!aligned(c->k_mean, 16) || !aligned(c->k_mean_scale, 4)))
        return DV_ERR_INVALID_ARG;
    a->k = c->k;
    a->v = c->v;
    a->ks = D.dtype == DV_I8 ? c->k_scale : nullptr;
    a->vs = D.dtype == DV_I8 ? c->v_scale : nullptr;
    a->mean = D.block ? c->k_mean : nullptr;
    a->mean_scale = D.block ? c->k_mean_scale : nullptr;
    a->Hkv = D.n_kv_heads;
    a->D = D.head_dim;
    a->cap = D.kv_cap;
    a->dtype = D.dtype;
    a->block = D.block;
    return DV_OK;
}

// Rows of D values: 16-byte aligned at every (b, t, h).
dv_status check_rows(const dv_kv_rows *r, KvRowsArgs *a)
{
    if (!r || !aligned(r->p, 16) || (r->dtype != DV_F32 && r->dtype != DV_F16))
        return DV_ERR_INVALID_ARG;
    const int64_t s[] = {r->stride_b, r->stride_t, r->stride_h};
    for (int64_t v : s)
        if (v < 0 || v % (16 / esize(r->dtype)))
            return DV_ERR_INVALID_ARG;
    a->p = r->p;
    a->f16 = r->dtype == DV_F16;
    a->sb = r->stride_b;
    a->st = r->stride_t;
    a->sh = r->stride_h;
    return DV_OK;
}

// Workspace: the status word's line, a counter per attention CTA, and two
// records of pieces per CTA (dv_kv_sched.cuh).  Only the records' size
// depends on the call, so one workspace serves any mix of calls that fit it.
size_t kv_ws_bytes(const dv_kv_desc &D, int tokens)
{
    const int G = D.n_heads / D.n_kv_heads;
    int rows = kv_plan(D.dtype, D.head_dim, 1).rows;
    for (int r : {tokens * G, G})
        if (kv_plan(D.dtype, D.head_dim, r).rows > rows)
            rows = kv_plan(D.dtype, D.head_dim, r).rows;
    return align_up(kKvRecOff + 2 * (size_t)kKvMaxCtas * rows * (D.head_dim + 2) * 4, 256);
}

dv_status check_ws(const dv_kv_desc &D, int tokens, void *ws, size_t ws_bytes)
{
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < kv_ws_bytes(D, tokens))
        return DV_ERR_WORKSPACE;
    return DV_OK;
}

dv_status attn_launch(const KvAttnArgs &a, const KvPlan &p, void *stream)
{
    int dev = 0, nsm = 0;
    if (cuda_failed(cudaGetDevice(&dev)) ||
        cuda_failed(cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))
        return DV_ERR_CUDA;
    return cuda_status(launch_kv_attn(a, p, nsm, static_cast<cudaStream_t>(stream)));
}

template <typename P>
P *at(void *ws, size_t off) { return reinterpret_cast<P *>(static_cast<char *>(ws) + off); }

// The softmax scale in units of log2, as the kernels take it.
float scale2(float scale) { return scale * 1.4426950408889634f; }

// Work items of a 1-D grid fit its limit.
bool grid_ok(long long n) { return n > 0 && n <= INT_MAX; }

}  // namespace

namespace dv {

// The driver's encoder is resolved through the runtime, so the library does
// not link the driver library itself.
cudaError_t kv_maps(const KvCacheArgs &c, int B, int rows, KvMaps *m)
{
    static std::once_flag once;
    static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    });
    if (!encode)
        return cudaErrorNotSupported;
    const cuuint64_t rb = (cuuint64_t)c.D * esize(c.dtype);
    const cuuint64_t dims[3] = {rb, (cuuint64_t)c.cap, (cuuint64_t)B * c.Hkv};
    const cuuint64_t strides[2] = {rb, rb * c.cap};
    const cuuint32_t box[3] = {(cuuint32_t)(rb < 128 ? rb : 128), (cuuint32_t)rows, 1};
    const cuuint32_t steps[3] = {1, 1, 1};
    const CUtensorMapSwizzle swz = rb < 128 ? CU_TENSOR_MAP_SWIZZLE_64B
                                            : CU_TENSOR_MAP_SWIZZLE_128B;
    for (int i = 0; i < 2; ++i)
        if (encode(i ? &m->v : &m->k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, i ? c.v : c.k, dims,
                   strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    return cudaSuccess;
}

}  // namespace dv

extern "C" {

dv_status dv_set_tree_kernel(int variant)
{
    if (variant < 0 || variant > 2)
        return DV_ERR_INVALID_ARG;
    g_tree_variant.store(variant);
    return DV_OK;
}

size_t dv_kv_workspace_size(const dv_kv_desc *desc, int batch, int tokens)
{
    if (check_desc(desc) != DV_OK || batch < 1 || batch > DV_KV_MAX_BATCH || tokens < 1 ||
        tokens > desc->kv_cap)
        return 0;
    return kv_ws_bytes(*desc, tokens > DV_TREE_MAX_TOKENS ? DV_TREE_MAX_TOKENS : tokens);
}

int dv_kv_append(const dv_kv_desc *desc, const dv_kv_cache *cache, const dv_kv_rows *k,
                 const dv_kv_rows *v, int batch, int tokens, const int32_t *lens,
                 const int32_t *n_tok, void *ws, size_t ws_bytes, void *stream)
{
    dv_status s = check_desc(desc);
    if (s)
        return s;
    KvAppendArgs a;
    std::memset(&a, 0, sizeof(a));
    if ((s = check_cache(*desc, cache, batch, &a.c)) || (s = check_rows(k, &a.k)) ||
        (s = check_rows(v, &a.v)))
        return s;
    if (a.k.f16 != a.v.f16)
        return DV_ERR_INVALID_ARG;
    if (tokens < 1 || tokens > desc->kv_cap || !aligned(lens, 4) || (n_tok && !aligned(n_tok, 4)))
        return DV_ERR_INVALID_ARG;
    if ((s = check_ws(*desc, 1, ws, ws_bytes)))
        return s;
    a.tile = kKvWriteTile;
    if (!grid_ok((long long)batch * desc->n_kv_heads * ((tokens - 2) / a.tile + 2)))
        return DV_ERR_UNSUPPORTED;
    a.lens = lens;
    a.n_tok = n_tok;
    a.B = batch;
    a.T = tokens;
    a.status = at<int>(ws, 0);
    return cuda_status(launch_kv_append(a, static_cast<cudaStream_t>(stream)));
}

int dv_kv_read(const dv_kv_desc *desc, const dv_kv_cache *cache, int batch, int tokens,
               const int32_t *start, int out_dtype, void *k_out, void *v_out, void *ws,
               size_t ws_bytes, void *stream)
{
    dv_status s = check_desc(desc);
    if (s)
        return s;
    KvReadArgs a;
    std::memset(&a, 0, sizeof(a));
    if ((s = check_cache(*desc, cache, batch, &a.c)))
        return s;
    if (tokens < 1 || tokens > desc->kv_cap || !aligned(start, 4) || !aligned(k_out, 16) ||
        !aligned(v_out, 16) || (out_dtype != DV_F32 && out_dtype != DV_F16))
        return DV_ERR_INVALID_ARG;
    if ((s = check_ws(*desc, 1, ws, ws_bytes)))
        return s;
    if (!grid_ok((long long)batch * desc->n_kv_heads * tokens))
        return DV_ERR_UNSUPPORTED;
    a.start = start;
    a.B = batch;
    a.T = tokens;
    a.f16 = out_dtype == DV_F16;
    a.k_out = k_out;
    a.v_out = v_out;
    a.status = at<int>(ws, 0);
    return cuda_status(launch_kv_read(a, static_cast<cudaStream_t>(stream)));
}

int dv_kv_keep(const dv_kv_desc *desc, const dv_kv_cache *cache, int batch, int tokens,
               const int32_t *lens, const int32_t *path, const int32_t *n_keep, void *ws,
               size_t ws_bytes, void *stream)
{
    dv_status s = check_desc(desc);
    if (s)
        return s;
    KvKeepArgs a;
    std::memset(&a, 0, sizeof(a));
    if ((s = check_cache(*desc, cache, batch, &a.c)))
        return s;
    if (tokens < 1 || tokens > DV_TREE_MAX_TOKENS || tokens > desc->kv_cap || !aligned(lens, 4) ||
        !aligned(path, 4) || !aligned(n_keep, 4))
        return DV_ERR_INVALID_ARG;
    if ((s = check_ws(*desc, 1, ws, ws_bytes)))
        return s;
    a.lens = lens;
    a.path = path;
    a.n_keep = n_keep;
    a.B = batch;
    a.T = tokens;
    a.status = at<int>(ws, 0);
    return cuda_status(launch_kv_keep(a, static_cast<cudaStream_t>(stream)));
}

int dv_tree_attn(const dv_kv_desc *desc, const dv_kv_cache *cache, const dv_kv_rows *q, int batch,
                 int tokens, const int32_t *lens, const int32_t *n_tok, const uint64_t *mask,
                 float scale, const int32_t *u_h, const int32_t *n_u_h, int max_u_h, float *out,
                 void *ws, size_t ws_bytes, void *stream)
{
    dv_status s = check_desc(desc);
    if (s)
        return s;
    KvAttnArgs a;
    std::memset(&a, 0, sizeof(a));
    if ((s = check_cache(*desc, cache, batch, &a.c)) || (s = check_rows(q, &a.q)))
        return s;
    if (tokens < 1 || tokens > DV_TREE_MAX_TOKENS || tokens > desc->kv_cap || !aligned(lens, 4) ||
        (n_tok && !aligned(n_tok, 4)) || (mask && !aligned(mask, 8)) || !std::isfinite(scale2(scale)) ||
        !aligned(out, 16))
        return DV_ERR_INVALID_ARG;
    if (u_h ? !aligned(u_h, 4) || !aligned(n_u_h, 4) || max_u_h < 1 || max_u_h > desc->n_kv_heads
            : n_u_h || max_u_h)
        return DV_ERR_INVALID_ARG;
    if ((s = check_ws(*desc, tokens, ws, ws_bytes)))
        return s;
    a.lens = lens;
    a.n_tok = n_tok;
    a.mask = reinterpret_cast<const unsigned long long *>(mask);
    a.u_h = u_h;
    a.n_u_h = n_u_h;
    a.max_u_h = max_u_h;
    a.B = batch;
    a.H = desc->n_heads;
    a.T = tokens;
    a.r_group = (float)desc->n_kv_heads / (float)desc->n_heads;
    a.scale = scale2(scale);
    a.out = out;
    a.rec = at<float>(ws, kKvRecOff);
    a.cnt = at<int>(ws, kKvCntOff);
    a.status = at<int>(ws, 0);
    const int G = desc->n_heads / desc->n_kv_heads;
    return attn_launch(a, kv_plan(desc->dtype, desc->head_dim, tokens * G), stream);
}

int dv_block_topk(const dv_kv_desc *desc, const dv_kv_cache *cache, const dv_kv_rows *q, int batch,
                  const int32_t *lens, int k_blocks, int n_first, int n_last, int32_t *idx,
                  void *ws, size_t ws_bytes, void *stream)
{
    dv_status s = check_desc(desc);
    if (s)
        return s;
    KvTopkArgs a;
    std::memset(&a, 0, sizeof(a));
    if ((s = check_cache(*desc, cache, batch, &a.c)) || (s = check_rows(q, &a.q)))
        return s;
    if (!desc->block || k_blocks < 1 || k_blocks > kKvMaxBlocks || n_first < 0 || n_last < 1 ||
        n_first > k_blocks || n_last > k_blocks - n_first || !aligned(lens, 4) || !aligned(idx, 4))
        return DV_ERR_INVALID_ARG;
    if ((s = check_ws(*desc, 1, ws, ws_bytes)))
        return s;
    a.lens = lens;
    a.B = batch;
    a.H = desc->n_heads;
    a.k = k_blocks;
    a.n_first = n_first;
    a.n_last = n_last;
    a.idx = idx;
    a.status = at<int>(ws, 0);
    return cuda_status(launch_kv_topk(a, static_cast<cudaStream_t>(stream)));
}

int dv_block_attn(const dv_kv_desc *desc, const dv_kv_cache *cache, const dv_kv_rows *q, int batch,
                  const int32_t *lens, const int32_t *idx, int k_blocks, float scale, float *out,
                  void *ws, size_t ws_bytes, void *stream)
{
    dv_status s = check_desc(desc);
    if (s)
        return s;
    KvAttnArgs a;
    std::memset(&a, 0, sizeof(a));
    if ((s = check_cache(*desc, cache, batch, &a.c)) || (s = check_rows(q, &a.q)))
        return s;
    if (!desc->block || k_blocks < 1 || k_blocks > kKvMaxBlocks || !aligned(lens, 4) ||
        !aligned(idx, 4) || !std::isfinite(scale2(scale)) || !aligned(out, 16))
        return DV_ERR_INVALID_ARG;
    if ((s = check_ws(*desc, 1, ws, ws_bytes)))
        return s;
    a.lens = lens;
    a.idx = idx;
    a.k = k_blocks;
    while ((1 << a.blog) < desc->block)
        ++a.blog;
    a.B = batch;
    a.H = desc->n_heads;
    a.T = 1;
    a.r_group = (float)desc->n_kv_heads / (float)desc->n_heads;
    a.scale = scale2(scale);
    a.out = out;
    a.rec = at<float>(ws, kKvRecOff);
    a.cnt = at<int>(ws, kKvCntOff);
    a.status = at<int>(ws, 0);
    return attn_launch(a, kv_plan(desc->dtype, desc->head_dim, 1), stream);
}

}  // extern "C"
