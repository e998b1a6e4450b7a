// dv_kv.h -- argument blocks and launchers of the KV-cache operators
// (append / read / keep, attention over drafted trees and selected blocks,
// block selection), shared by dv_kv_abi.cu and the kernel translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "dv.h"
#include "dv_internal.h"

namespace dv {

constexpr int kKvTile = 64;        // cached positions per attention tile
constexpr int kKvWriteTile = 256;  // positions per CTA of dv_kv_append: a multiple of every block
constexpr int kKvMaxCtas = 608;    // attention CTAs (four per SM of 152); sizes the records
constexpr int kKvGenRows = 4;      // query rows per unit of the CUDA-core attention kernel
constexpr int kKvMaxBlocks = 16384;  // selectable blocks per row (scores in shared memory)

constexpr size_t kKvCntOff = 256;  // workspace: counters after the status word's line,
constexpr size_t kKvRecOff = (kKvCntOff + kKvMaxCtas * 4 + 255) / 256 * 256;  // then records

// One cache as the kernels see it.
struct KvCacheArgs {
    void *k, *v;
    float *ks, *vs;        // DV_I8: one scale per row of D values
    int8_t *mean;          // block means, [B][Hkv][cap / block][D]
    float *mean_scale;
    int Hkv, D, cap, dtype, block;
};

// Rows of D contiguous values at p + b sb + t st + h sh (elements).
struct KvRowsArgs {
    const void *p;
    int f16;
    long long sb, st, sh;
};

struct KvAppendArgs {
    KvCacheArgs c;
    KvRowsArgs k, v;
    const int32_t *lens, *n_tok;
    int B, T;
    int tile;              // positions per CTA (kKvWriteTile)
    int *status;
};

struct KvReadArgs {
    KvCacheArgs c;
    const int32_t *start;
    int B, T, f16;
    void *k_out, *v_out;
    int *status;
};

struct KvKeepArgs {
    KvCacheArgs c;
    const int32_t *lens, *path, *n_keep;
    int B, T;
    int *status;
};

struct KvTopkArgs {
    KvCacheArgs c;
    KvRowsArgs q;
    const int32_t *lens;
    int B, H, k, n_first, n_last;
    int32_t *idx;
    int *status;
};

struct KvAttnArgs {
    KvCacheArgs c;
    KvRowsArgs q;
    const int32_t *lens, *n_tok;
    const unsigned long long *mask;
    const int32_t *u_h, *n_u_h;
    int max_u_h;
    const int32_t *idx;    // block mode: [B][H][k]
    int k;
    int blog;              // log2(block)
    int B, H, T;
    float r_group;         // 1 / (query heads per KV head)
    float scale;           // softmax scale x log2(e)
    float *out;            // [B][T][H][D]
    // workspace
    float *rec;            // [2 x CTAs][rows][D + 2] pieces of units shared by CTAs
    int *cnt;              // per unit: pieces written (zero at rest)
    int *status;
};

// Attention variant of a shape: rows per unit (kKvGenRows: CUDA-core kernel).
struct KvPlan {
    int rows;    // query rows per unit
    bool mma;    // tensor-core kernel
};
KvPlan kv_plan(int dtype, int D, int rows);

// Units of dv_tree_attn where both kinds serve: 0 by rule, 1 of 8 rows, 2 of 64.
extern std::atomic<int> g_tree_variant;

cudaError_t launch_kv_append(const KvAppendArgs &a, cudaStream_t st);
cudaError_t launch_kv_read(const KvReadArgs &a, cudaStream_t st);
cudaError_t launch_kv_keep(const KvKeepArgs &a, cudaStream_t st);
cudaError_t launch_kv_topk(const KvTopkArgs &a, cudaStream_t st);
// Tensor maps of a cache's keys and values for boxes of `rows` positions of
// one (row, head), at most 128 bytes of a row wide (dv_kv_abi.cu): the box's
// rows are swizzled over their own width.
struct KvMaps {
    CUtensorMap k, v;
};
cudaError_t kv_maps(const KvCacheArgs &c, int B, int rows, KvMaps *m);
cudaError_t launch_kv_mma(const KvAttnArgs &a, int nsm, cudaStream_t st);
cudaError_t launch_kv_tc(const KvAttnArgs &a, int nsm, cudaStream_t st);
cudaError_t launch_kv_attn(const KvAttnArgs &a, const KvPlan &p, int nsm, cudaStream_t st);

}  // namespace dv
