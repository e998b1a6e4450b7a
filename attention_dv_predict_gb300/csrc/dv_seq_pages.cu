// dv_seq_pages.cu -- pages of a pool given back and taken; block tables,
// positions and slots of packed tokens from the requests' lengths (sm_103a).
//
// Taking needs two prefix sums over the requests, of their tokens and of their
// new pages.  A CTA forms both by itself (a request a thread: one round trip
// for the lengths) and then writes its own 1024 tokens and its share of the
// table entries, so one launch does it all: a token's page is in the table
// already or is that place of the stack which the prefix sum gives, whoever
// writes the table entry.  Latency bounds it, not bytes.
#include "dv_common.cuh"
#include "dv_seq.h"

namespace dv {
namespace {

constexpr int kPageThreads = 1024;
constexpr int kPageTokens = 1024;  // tokens per CTA
static_assert(DV_SEQ_MAX_BATCH <= kPageThreads, "a request a thread");

DV_DEV int pages_of(long long n, int page) { return (int)((n + page - 1) / page); }

// Exclusive prefix sum over the block of long long.
DV_DEV long long scan64(long long v, long long *scratch, long long *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, inc, o);
        inc += lane >= o ? t : 0;
    }
    if (lane == 31)
        scratch[warp] = inc;
    __syncthreads();
    long long s = lane < nw ? scratch[lane] : 0, t = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, t, o);
        t += lane >= o ? u : 0;
    }
    *total = __shfl_sync(0xffffffffu, t, 31);
    const long long before = __shfl_sync(0xffffffffu, t - s, warp);
    __syncthreads();
    return before + inc - v;
}

__global__ void __launch_bounds__(kPageThreads) k_page_take(const SeqTakeArgs a)
{
    __shared__ long long scratch[32];
    __shared__ int s_cu[DV_SEQ_MAX_BATCH + 1], s_len[DV_SEQ_MAX_BATCH], s_have[DV_SEQ_MAX_BATCH];
    __shared__ int s_need[DV_SEQ_MAX_BATCH];  // new pages; -1: not served
    __shared__ int s_top[DV_SEQ_MAX_BATCH];   // stack place of the first of them
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool report = blockIdx.x == 0;
    // (a request a thread: DV_SEQ_MAX_BATCH is the block's size)
    int len = 0, n = 0, have = 0, need = 0;
    const int n_free = __ldcg(a.n_free);
    int top = n_free;
    if (top < 0 || top > a.n_pages) {  // no page is taken
        top = 0;
        if (report && tid == 0)
            set_status(a.status, DV_ERR_DEVICE_INDEX);
    }
    if (tid < a.B) {
        len = __ldg(a.lens + tid);
        n = __ldg(a.n_tok + tid);
        if (len < 0 || n < 0 || (long long)len + n > (long long)a.width * a.page) {
            len = n = 0;
            if (report)
                set_status(a.status, DV_ERR_DEVICE_INDEX);
        }
        have = pages_of(len, a.page);
        need = pages_of((long long)len + n, a.page) - have;
    }
    long long tokens, pages;
    const long long t0 = scan64(n, scratch, &tokens);
    const long long p0 = scan64(need, scratch, &pages);
    if (tid < a.B) {
        const bool fits = need == 0 || p0 + need <= top;
        s_cu[tid + 1] = (int)min(t0 + n, (long long)a.T);
        s_len[tid] = len;
        s_have[tid] = have;
        s_need[tid] = fits ? need : -1;
        s_top[tid] = fits ? top - 1 - (int)p0 : 0;
        if (report) {
            a.cu[tid + 1] = s_cu[tid + 1];
            if (!fits)
                set_status(a.status, DV_ERR_PAGES);
            else if (t0 + n > a.T)
                set_status(a.status, DV_ERR_DEVICE_INDEX);
        }
    }
    if (tid == 0) {
        s_cu[0] = 0;
        if (report)
            a.cu[0] = 0;
    }
    // served requests that take pages are a prefix of those that need some
    long long taken = 0;
    scan64(tid < a.B && p0 + need <= top ? need : 0, scratch, &taken);

    // table entries: a warp a request
    for (int b = blockIdx.x * (kPageThreads / 32) + warp; b < a.B;
         b += gridDim.x * (kPageThreads / 32))
        for (int j = lane; j < s_need[b]; j += 32)
            a.tables[(size_t)b * a.width + s_have[b] + j] = __ldg(a.free_pages + s_top[b] - j);

    // tokens
    const long long t = (long long)blockIdx.x * kPageTokens + tid;
    if (t < a.T) {
        int pos = -1, slot = -1;
        if (t < s_cu[a.B]) {
            int b = 0;
            for (int step = DV_SEQ_MAX_BATCH / 2; step > 0; step >>= 1)  // largest b with cu[b] <= t
                if (b + step < a.B && s_cu[b + step] <= t)
                    b += step;
            pos = s_len[b] + (int)t - s_cu[b];
            const int j = pos / a.page, k = j - s_have[b];
            if (k < 0 || s_need[b] >= 0) {
                const int pg = k < 0 ? __ldg(a.tables + (size_t)b * a.width + j)
                                     : __ldg(a.free_pages + s_top[b] - k);
                if (s_need[b] < 0)
                    ;  // not served, its first page's rest either
                else if (pg < 0 || pg >= a.n_pages)
                    set_status(a.status, DV_ERR_DEVICE_INDEX);
                else
                    slot = pg * a.page + pos % a.page;
            }
        }
        a.pos[t] = pos;
        a.slots[t] = slot;
    }

    // n_free_out may be n_free: written when every CTA has read it
    __syncthreads();
    if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(a.cnt, 1) == (int)gridDim.x - 1;
        if (s_last) {
            *a.cnt = 0;
            *a.n_free_out = n_free - (int)taken;
        }
    }
}

// One CTA (few requests finish in a step): a warp a request checks its page
// numbers, a prefix sum places them, and the warps copy them.
__global__ void __launch_bounds__(kPageThreads) k_page_release(const SeqReleaseArgs a)
{
    __shared__ long long scratch[32];
    __shared__ int s_held[DV_SEQ_MAX_BATCH], s_at[DV_SEQ_MAX_BATCH];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_free = *a.n_free;
    int top = n_free;
    bool bad = top < 0 || top > a.n_pages;
    if (tid < a.B) {
        int held = 0;
        if (a.done[tid]) {
            const int len = a.lens[tid];
            if (len < 0 || len > (long long)a.width * a.page)
                bad = true;
            else
                held = pages_of(len, a.page);
        }
        s_held[tid] = held;
    }
    if (top < 0 || top > a.n_pages)
        top = a.n_pages;  // (no room: every request is skipped)
    __syncthreads();
    for (int b = warp; b < a.B; b += kPageThreads / 32) {
        const int held = s_held[b];
        bool off = false;
#pragma unroll 4
        for (int j = lane; j < held; j += 32)
            off |= (unsigned)__ldg(a.tables + (size_t)b * a.width + j) >= (unsigned)a.n_pages;
        off = __any_sync(0xffffffffu, off);
        __syncwarp();
        if (off) {
            bad = true;
            if (lane == 0)
                s_held[b] = 0;
        }
    }
    __syncthreads();
    const int held = tid < a.B ? s_held[tid] : 0;
    long long all;
    const long long at = scan64(held, scratch, &all);
    // those that fit are a prefix of the requests that give pages back
    const bool fits = top + at + held <= a.n_pages;
    bad |= held > 0 && !fits;
    long long pushed;
    scan64(fits ? held : 0, scratch, &pushed);
    if (tid < a.B) {
        s_at[tid] = top + (int)at;
        if (!fits)
            s_held[tid] = 0;
    }
    __syncthreads();
    for (int b = warp; b < a.B; b += kPageThreads / 32)
#pragma unroll 4
        for (int j = lane; j < s_held[b]; j += 32)
            a.free_pages[s_at[b] + j] = __ldg(a.tables + (size_t)b * a.width + j);
    if (bad)
        set_status(a.status, DV_ERR_DEVICE_INDEX);
    // (the count was read before the barriers above)
    if (tid == 0)
        *a.n_free_out = n_free + (int)pushed;
}

}  // namespace

cudaError_t launch_page_release(const SeqReleaseArgs &a, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPageThreads);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, k_page_release, a);
}

cudaError_t launch_page_take(const SeqTakeArgs &a, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.T + kPageTokens - 1) / kPageTokens);
    cfg.blockDim = dim3(kPageThreads);
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, k_page_take, a);
}

}  // namespace dv
