// dv_seq_abi.cu -- C entry points of the operators over packed sequences and
// paged caches: argument checks and workspace layout.  See include/dv.h.
#include <cfloat>
#include <climits>
#include <cmath>
#include <cstring>

#include "dv_seq.h"

using namespace dv;

namespace {

int esize(int dtype) { return dtype == DV_F16 ? 2 : 4; }
bool aligned(const void *p, size_t a) { return p && (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
dv_status cuda_status(cudaError_t e) { return cuda_failed(e) ? DV_ERR_CUDA : DV_OK; }

constexpr int kMaxTokens = 1 << 28;

dv_status check_desc(const dv_seq_desc *D)
{
    if (!D || D->n_heads <= 0 || D->n_kv_heads <= 0 || D->n_heads % D->n_kv_heads ||
        D->head_dim <= 0 || D->page < 0 || D->n_pages < 0 || !D->page != !D->n_pages)
        return DV_ERR_INVALID_ARG;
    if (D->dtype != DV_F32 && D->dtype != DV_F16)
        return DV_ERR_INVALID_ARG;
    const int d = D->head_dim;
    if ((d & (d - 1)) || d < 8 || d > 256 || d * esize(D->dtype) > 512 || D->n_heads > 256)
        return DV_ERR_UNSUPPORTED;
    if (D->page && D->page != 16 && D->page != 32 && D->page != 64 && D->page != 128)
        return DV_ERR_UNSUPPORTED;
    // (page numbers times heads are a 32-bit coordinate of the copies)
    if ((long long)D->n_pages * D->page > 1 << 30 ||
        (long long)D->n_pages * D->n_kv_heads > INT_MAX)
        return DV_ERR_UNSUPPORTED;
    return DV_OK;
}

// Binary16 rows of 64 and 128 values run on tensor cores.
bool on_tc(int f16, int D) { return f16 && (D == 64 || D == 128); }

size_t seq_ws_bytes(const dv_seq_desc &D)
{
    const size_t rec = on_tc(D.dtype == DV_F16, D.head_dim) ? seq_tc_record_bytes(D.head_dim)
                                                            : seq_attn_record_bytes(D.head_dim);
    return (kSeqRecOff + rec + 255) / 256 * 256;
}

dv_status check_ws(const dv_seq_desc &D, void *ws, size_t ws_bytes)
{
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < seq_ws_bytes(D))
        return DV_ERR_WORKSPACE;
    return DV_OK;
}

// Rows (t, h) of D values, 16-byte aligned.  own: rows that differ must not
// overlap (their strides are at least D).
dv_status check_rows(const dv_kv_rows *r, int D, int tokens, int heads, bool own, SeqRowsArgs *a)
{
    if (!r || !aligned(r->p, 16) || (r->dtype != DV_F32 && r->dtype != DV_F16))
        return DV_ERR_INVALID_ARG;
    const int64_t s[] = {r->stride_t, r->stride_h};
    for (int i = 0; i < 2; ++i) {
        if (s[i] < 0 || s[i] % (16 / esize(r->dtype)) || s[i] >= (int64_t)1 << 38)
            return DV_ERR_INVALID_ARG;
        if (own && (i ? heads : tokens) > 1 && s[i] < D)
            return DV_ERR_INVALID_ARG;
    }
    a->p = const_cast<void *>(r->p);
    a->f16 = r->dtype == DV_F16;
    a->st = r->stride_t;
    a->sh = r->stride_h;
    return DV_OK;
}

dv_status check_pool(const dv_seq_desc &D, const dv_page_pool *p)
{
    if (!D.page || !p || !aligned(p->k, 16) || !aligned(p->v, 16))
        return DV_ERR_INVALID_ARG;
    return DV_OK;
}

template <typename P>
P *at(void *ws, size_t off) { return reinterpret_cast<P *>(static_cast<char *>(ws) + off); }

dv_status check_batch(int batch) { return batch < 1 || batch > DV_SEQ_MAX_BATCH ? DV_ERR_INVALID_ARG : DV_OK; }

// Positions that a row of the block tables can hold.
bool table_ok(const dv_seq_desc &D, int max_pages)
{
    return max_pages >= 1 && (long long)max_pages * D.page <= 1 << 30;
}

// What both attention calls check and set.
dv_status attn_args(const dv_seq_desc *desc, int batch, int tokens, int max_tok,
                    const dv_kv_rows *q, const int32_t *cu, float scale, void *out, void *ws,
                    size_t ws_bytes, SeqAttnArgs *a)
{
    dv_status s = check_desc(desc);
    if (s)
        return s;
    std::memset(a, 0, sizeof(*a));
    if ((s = check_batch(batch)))
        return s;
    if (tokens < 1 || tokens > kMaxTokens || max_tok < 1 || !aligned(cu, 4) || !aligned(out, 16))
        return DV_ERR_INVALID_ARG;
    const float scale2 = scale * 1.4426950408889634f;
    if (!(scale2 >= FLT_MIN && scale2 <= FLT_MAX))
        return DV_ERR_INVALID_ARG;
    if ((s = check_rows(q, desc->head_dim, tokens, desc->n_heads, true, &a->q)))
        return s;
    if (a->q.f16 != (desc->dtype == DV_F16))
        return DV_ERR_INVALID_ARG;
    if ((s = check_ws(*desc, ws, ws_bytes)))
        return s;
    a->cu = cu;
    a->B = batch;
    a->T = tokens;
    a->max_tok = max_tok < tokens ? max_tok : tokens;
    a->H = desc->n_heads;
    a->Hkv = desc->n_kv_heads;
    a->D = desc->head_dim;
    a->f16 = a->q.f16;
    a->scale = scale2;
    a->out = out;
    a->rec = at<float>(ws, kSeqRecOff);
    a->cnt = at<int>(ws, kSeqCntOff);
    a->status = at<int>(ws, 0);
    return DV_OK;
}

dv_status attn_launch(SeqAttnArgs &a, void *stream)
{
    int dev = 0, nsm = 0;
    if (cuda_failed(cudaGetDevice(&dev)) ||
        cuda_failed(cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev)))
        return DV_ERR_CUDA;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return cuda_status(on_tc(a.f16, a.D) ? launch_seq_tc(a, nsm, st) : launch_seq_attn(a, nsm, st));
}

}  // namespace

namespace dv {

// A unit's rows are `group` query heads of a KV head times 2^tlog tokens.  The
// more heads, the fewer times the cache is read (each group reads it); but the
// rows that a power of two of tokens leaves empty cost as much as full ones.  So:
// all heads of the KV head where a request's tokens fit one unit anyway, else
// the most heads that fill three quarters of the rows.
void seq_group(SeqAttnArgs &a, int rows)
{
    const int G = a.H / a.Hkv;
    auto log_tokens = [rows](int g) {
        int t = 0;
        while ((2 << t) * g <= rows)
            ++t;
        return t;
    };
    a.group = 1;
    for (int g = G < rows ? G : rows; g > 1; --g) {
        const int fit = g << log_tokens(g);
        if (G % g == 0 && (4 * fit >= 3 * rows || (long long)a.max_tok * g <= fit)) {
            a.group = g;
            break;
        }
    }
    a.tlog = log_tokens(a.group);
    a.sub = G / a.group;
}

}  // namespace dv

extern "C" {

size_t dv_seq_workspace_size(const dv_seq_desc *desc)
{
    return check_desc(desc) == DV_OK ? seq_ws_bytes(*desc) : 0;
}

int dv_page_release(const dv_seq_desc *desc, int batch, const int32_t *lens, const int32_t *done,
                    int max_pages, const int32_t *tables, int32_t *free_pages,
                    const int32_t *n_free, int32_t *n_free_out, void *ws, size_t ws_bytes,
                    void *stream)
{
    dv_status s = check_desc(desc);
    if (s || (s = check_batch(batch)))
        return s;
    if (!desc->page || !table_ok(*desc, max_pages) || !aligned(lens, 4) || !aligned(done, 4) ||
        !aligned(tables, 4) || !aligned(free_pages, 4) || !aligned(n_free, 4) ||
        !aligned(n_free_out, 4))
        return DV_ERR_INVALID_ARG;
    if ((s = check_ws(*desc, ws, ws_bytes)))
        return s;
    SeqReleaseArgs a;
    std::memset(&a, 0, sizeof(a));
    a.lens = lens;
    a.done = done;
    a.tables = tables;
    a.n_free = n_free;
    a.free_pages = free_pages;
    a.n_free_out = n_free_out;
    a.B = batch;
    a.width = max_pages;
    a.page = desc->page;
    a.n_pages = desc->n_pages;
    a.status = at<int>(ws, 0);
    return cuda_status(launch_page_release(a, static_cast<cudaStream_t>(stream)));
}

int dv_page_take(const dv_seq_desc *desc, int batch, const int32_t *lens, const int32_t *n_tok,
                 int max_pages, int32_t *tables, const int32_t *free_pages, const int32_t *n_free,
                 int32_t *n_free_out, int32_t *cu, int32_t *pos, int32_t *slots, int max_tokens,
                 void *ws, size_t ws_bytes, void *stream)
{
    dv_status s = check_desc(desc);
    if (s || (s = check_batch(batch)))
        return s;
    if (!desc->page || !table_ok(*desc, max_pages) || max_tokens < 1 || max_tokens > kMaxTokens ||
        !aligned(lens, 4) || !aligned(n_tok, 4) || !aligned(tables, 4) || !aligned(free_pages, 4) ||
        !aligned(n_free, 4) || !aligned(n_free_out, 4) || !aligned(cu, 4) || !aligned(pos, 4) ||
        !aligned(slots, 4))
        return DV_ERR_INVALID_ARG;
    if ((s = check_ws(*desc, ws, ws_bytes)))
        return s;
    SeqTakeArgs a;
    std::memset(&a, 0, sizeof(a));
    a.lens = lens;
    a.n_tok = n_tok;
    a.free_pages = free_pages;
    a.n_free = n_free;
    a.tables = tables;
    a.n_free_out = n_free_out;
    a.cu = cu;
    a.pos = pos;
    a.slots = slots;
    a.B = batch;
    a.width = max_pages;
    a.page = desc->page;
    a.n_pages = desc->n_pages;
    a.T = max_tokens;
    a.cnt = at<int>(ws, kSeqPageCnt);
    a.status = at<int>(ws, 0);
    return cuda_status(launch_page_take(a, static_cast<cudaStream_t>(stream)));
}

int dv_qk_rope(const dv_seq_desc *desc, const dv_rope *rope, int tokens, const int32_t *pos,
               const dv_kv_rows *q, const dv_kv_rows *k, const dv_kv_rows *v,
               const dv_kv_rows *q_out, const dv_kv_rows *k_out, const dv_page_pool *pool,
               const int32_t *slots, void *ws, size_t ws_bytes, void *stream)
{
    dv_status s = check_desc(desc);
    if (s)
        return s;
    SeqRopeArgs a;
    std::memset(&a, 0, sizeof(a));
    const int D = desc->head_dim, H = desc->n_heads, Hkv = desc->n_kv_heads;
    if (tokens < 1 || tokens > kMaxTokens || !aligned(pos, 4) || !rope)
        return DV_ERR_INVALID_ARG;
    if ((s = check_rows(q, D, tokens, H, false, &a.q)) ||
        (s = check_rows(k, D, tokens, Hkv, false, &a.k)) ||
        (v && (s = check_rows(v, D, tokens, Hkv, false, &a.v))) ||
        (s = check_rows(q_out, D, tokens, H, true, &a.q_out)) ||
        (k_out && (s = check_rows(k_out, D, tokens, Hkv, true, &a.k_out))))
        return s;
    if (a.k.f16 != a.q.f16 || (v && (a.v.f16 != a.q.f16 || !pool)) || (!k_out && !pool) ||
        !pool != !slots || (slots && !aligned(slots, 4)))
        return DV_ERR_INVALID_ARG;
    if (pool && (s = check_pool(*desc, pool)))
        return s;
    if (rope->rot_dim < 0 || rope->rot_dim % 2 || rope->rot_dim > D ||
        (rope->rot_dim && (!aligned(rope->steps, 8) || !std::isfinite(rope->mscale))) ||
        (rope->interleaved != 0 && rope->interleaved != 1))
        return DV_ERR_INVALID_ARG;
    if (rope->q_gain || rope->k_gain) {
        if ((rope->q_gain && !aligned(rope->q_gain, 16)) ||
            (rope->k_gain && !aligned(rope->k_gain, 16)) ||
            (rope->norm != DV_LAYERNORM && rope->norm != DV_RMSNORM) || !(rope->eps > 0) ||
            !std::isfinite(rope->eps))
            return DV_ERR_INVALID_ARG;
    }
    if ((s = check_ws(*desc, ws, ws_bytes)))
        return s;
    a.pk = pool ? pool->k : nullptr;
    a.pv = pool ? pool->v : nullptr;
    a.pos = pos;
    a.slots = slots;
    a.steps = reinterpret_cast<const unsigned long long *>(rope->steps);
    a.q_gain = rope->q_gain;
    a.k_gain = rope->k_gain;
    a.T = tokens;
    a.H = H;
    a.Hkv = Hkv;
    a.D = D;
    a.f16 = desc->dtype == DV_F16;
    a.page = desc->page;
    a.n_pages = desc->n_pages;
    a.rot = rope->rot_dim;
    a.interleaved = rope->interleaved;
    a.layer = rope->norm == DV_LAYERNORM;
    a.mscale = rope->mscale;
    a.eps = rope->eps;
    a.status = at<int>(ws, 0);
    return cuda_status(launch_qk_rope(a, static_cast<cudaStream_t>(stream)));
}

int dv_prompt_attn(const dv_seq_desc *desc, int batch, int tokens, int max_tok,
                   const dv_kv_rows *q, const dv_kv_rows *k, const dv_kv_rows *v,
                   const int32_t *cu, float scale, void *out, void *ws, size_t ws_bytes,
                   void *stream)
{
    SeqAttnArgs a;
    dv_status s = attn_args(desc, batch, tokens, max_tok, q, cu, scale, out, ws, ws_bytes, &a);
    if (s)
        return s;
    if ((s = check_rows(k, a.D, tokens, a.Hkv, true, &a.k)) ||
        (s = check_rows(v, a.D, tokens, a.Hkv, true, &a.v)))
        return s;
    if (a.k.f16 != a.f16 || a.v.f16 != a.f16)
        return DV_ERR_INVALID_ARG;
    return attn_launch(a, stream);
}

int dv_paged_attn(const dv_seq_desc *desc, const dv_page_pool *pool, int batch, int tokens,
                  int max_tok, const dv_kv_rows *q, const int32_t *cu, const int32_t *lens,
                  const int32_t *tables, int max_pages, float scale, void *out, void *ws,
                  size_t ws_bytes, void *stream)
{
    SeqAttnArgs a;
    dv_status s = attn_args(desc, batch, tokens, max_tok, q, cu, scale, out, ws, ws_bytes, &a);
    if (s || (s = check_pool(*desc, pool)))
        return s;
    if (!table_ok(*desc, max_pages) || !aligned(lens, 4) || !aligned(tables, 4))
        return DV_ERR_INVALID_ARG;
    a.pk = pool->k;
    a.pv = pool->v;
    a.lens = lens;
    a.tables = tables;
    a.page = desc->page;
    a.n_pages = desc->n_pages;
    a.width = max_pages;
    return attn_launch(a, stream);
}

}  // extern "C"
