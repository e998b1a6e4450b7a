// dv_seq.h -- argument blocks and launchers of the operators over packed
// sequences and paged caches, shared by dv_seq_abi.cu and the kernel
// translation units.
#pragma once

#include "dv_kv.h"

namespace dv {

constexpr int kSeqMaxCtas = 608;   // attention CTAs on CUDA cores (four per SM of 152)
constexpr int kSeqTcCtas = 152;    // tensor-core attention CTAs (one per SM)
constexpr int kSeqGenRows = 32;    // the CUDA-core kernel's query rows a unit
constexpr int kSeqGenTile = 64;    // and cached positions a tile

// Workspace: the status word's line, counters (zero at rest), then records of
// attention units that several CTAs share.
constexpr size_t kSeqPageCnt = 256;
constexpr size_t kSeqCntOff = 512;
constexpr size_t kSeqRecOff = (kSeqCntOff + kSeqMaxCtas * 4 + 255) / 256 * 256;

// Rows of D contiguous values at p + t st + h sh (elements).
struct SeqRowsArgs {
    void *p;
    int f16;
    long long st, sh;
};

struct SeqReleaseArgs {
    const int32_t *lens, *done, *tables, *n_free;
    int32_t *free_pages, *n_free_out;
    int B, width, page, n_pages;
    int *status;
};

struct SeqTakeArgs {
    const int32_t *lens, *n_tok, *free_pages, *n_free;
    int32_t *tables, *n_free_out, *cu, *pos, *slots;
    int B, width, page, n_pages, T;
    int *cnt;       // CTAs done (zero at rest)
    int *status;
};

struct SeqRopeArgs {
    SeqRowsArgs q, k, v, q_out, k_out;  // p NULL: none
    void *pk, *pv;                      // pool, NULL: none
    const int32_t *pos, *slots;
    const unsigned long long *steps;
    const float *q_gain, *k_gain;
    int T, H, Hkv, D, f16;              // f16: the pool's type
    int page, n_pages;
    int rot, interleaved, layer;        // layer: mean taken off
    float mscale, eps;
    int *status;
};

struct SeqAttnArgs {
    SeqRowsArgs q, k, v;     // k, v: packed rows (prompt) or p NULL
    const void *pk, *pv;     // pool, NULL: packed rows
    const int32_t *cu, *lens, *tables;
    int B, T, max_tok, H, Hkv, D, f16;
    int page, n_pages, width;
    // query heads of a KV head fill a unit's rows in groups of `group` (which
    // divides their number), `tq` tokens (a power of two) to 2^tlog x group rows
    int group, tlog;
    int sub;                 // groups of a KV head's query heads
    float scale;             // softmax scale x log2(e)
    void *out;               // [T][H][D]
    float *rec;
    int *cnt;
    int *status;
};

// Sets group, tlog and sub for units of `rows` query rows (dv_seq_abi.cu).
void seq_group(SeqAttnArgs &a, int rows);

cudaError_t launch_page_release(const SeqReleaseArgs &a, cudaStream_t st);
cudaError_t launch_page_take(const SeqTakeArgs &a, cudaStream_t st);
cudaError_t launch_qk_rope(const SeqRopeArgs &a, cudaStream_t st);
cudaError_t launch_seq_attn(const SeqAttnArgs &a, int nsm, cudaStream_t st);
size_t seq_attn_record_bytes(int D);
cudaError_t launch_seq_tc(const SeqAttnArgs &a, int nsm, cudaStream_t st);
size_t seq_tc_record_bytes(int D);

}  // namespace dv
