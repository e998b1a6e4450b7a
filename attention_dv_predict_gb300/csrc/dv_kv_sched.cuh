// dv_kv_sched.cuh -- how the KV attention kernels share their work (sm_103a).
//
// A unit is up to `rows` query rows (token-major: row = token G + group
// member) of one (batch row, KV head) -- of one (batch row, query head) in
// block mode -- and its work is the tiles of 64 cached positions it sees.
// Lengths differ from row to row and are known on the device only, so the
// tiles of all units are laid end to end and the grid's C CTAs take equal
// runs of them: CTA c the tiles [W c / C, W (c + 1) / C).  A unit inside one
// run is finished by its CTA; a unit cut by a run's end leaves a piece (max
// m, sum l, weighted values o, per row) in a record, and the last of its CTAs
// to arrive merges the pieces in the order of the positions, so the result
// does not depend on who was last.  At most one cut unit starts in a CTA's
// run, so a counter per CTA is enough, and a CTA has at most two pieces: one
// that began before its run (or at its start), one that goes on after it.
// No CTA waits for another.
#pragma once

#include "dv_kv.cuh"

namespace dv {
namespace {

struct SchedSmem {
    long long pref[DV_KV_MAX_BATCH + 1];  // tiles before batch row b
    int tiles[DV_KV_MAX_BATCH];           // tiles of one unit of the row
    int mb[DV_KV_MAX_BATCH];              // units per head
    int last;
};

// The unit that a tile belongs to.
struct Unit {
    int b, h;         // batch row; KV head (block mode: query head); h < 0: none such
    int row0, nrows;  // first query row and count
    int len, ntok;    // cached prefix, drafted tokens (block mode: 0)
    int ent;          // block mode: entries of the index list
    long long w0, w1; // its tiles
};

struct Run {
    long long W, lo, hi;
    int C, c, nsel;
};

// Fills sm (every thread of the CTA calls it) and returns this CTA's run.
template <bool BLOCK>
DV_DEV Run sched_init(const KvAttnArgs &a, int rows, SchedSmem &sm)
{
    const int G = a.H / a.c.Hkv;
    int nsel = a.H;
    if (!BLOCK)
        nsel = a.u_h ? min(max(__ldg(a.n_u_h), 0), a.max_u_h) : a.c.Hkv;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const int len = __ldg(a.lens + b);
        int tiles = 0, mb = 0;
        if (BLOCK) {
            if (len >= 0 && len <= a.c.cap) {
                const long long e = min(a.k, (len + a.c.block - 1) / a.c.block);
                tiles = max(1, (int)((e * a.c.block + kKvTile - 1) / kKvTile));
                mb = 1;
            } else if (blockIdx.x == 0) {
                set_status(a.status, DV_ERR_DEVICE_INDEX);
            }
        } else {
            const int n = a.n_tok ? __ldg(a.n_tok + b) : a.T;
            if (len >= 0 && n >= 0 && n <= a.T && len <= a.c.cap - n) {
                if (n > 0) {
                    tiles = (len + n + kKvTile - 1) / kKvTile;
                    mb = (n * G + rows - 1) / rows;
                }
            } else if (blockIdx.x == 0) {
                set_status(a.status, DV_ERR_DEVICE_INDEX);
            }
        }
        sm.tiles[b] = tiles;
        sm.mb[b] = mb;
        sm.pref[b + 1] = (long long)tiles * mb * nsel;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        long long base = 0;
        if (threadIdx.x == 0)
            sm.pref[0] = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int b = b0 + threadIdx.x;
            long long v = b < a.B ? sm.pref[b + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, v, o);
                if ((int)threadIdx.x >= o)
                    v += t;
            }
            if (b < a.B)
                sm.pref[b + 1] = base + v;
            base += __shfl_sync(0xffffffffu, v, 31);
        }
    }
    __syncthreads();
    Run r;
    r.W = sm.pref[a.B];
    r.C = (int)min((long long)gridDim.x, r.W);
    r.c = blockIdx.x;
    r.nsel = nsel;
    r.lo = r.c < r.C ? r.W * r.c / r.C : 0;
    r.hi = r.c < r.C ? r.W * (r.c + 1) / r.C : 0;
    return r;
}

// The unit of tile w (0 <= w < W).
template <bool BLOCK>
DV_DEV Unit sched_unit(const KvAttnArgs &a, int rows, const SchedSmem &sm, const Run &r,
                       long long w)
{
    int b = 0;
    for (int step = 128; step > 0; step >>= 1)  // largest b with pref[b] <= w
        if (b + step < a.B && sm.pref[b + step] <= w)
            b += step;
    const int tiles = sm.tiles[b], mb = sm.mb[b];
    const int u = (int)((w - sm.pref[b]) / tiles);
    const int j = u / mb, m = u - j * mb;
    Unit x;
    x.b = b;
    x.w0 = sm.pref[b] + (long long)u * tiles;
    x.w1 = x.w0 + tiles;
    x.len = __ldg(a.lens + b);
    if (BLOCK) {
        x.h = j;
        x.row0 = 0;
        x.nrows = 1;
        x.ntok = 0;
        x.ent = min(a.k, (x.len + a.c.block - 1) / a.c.block);
    } else {
        const int G = a.H / a.c.Hkv;
        x.h = a.u_h ? __ldg(a.u_h + j) : j;
        if (x.h < 0 || x.h >= a.c.Hkv) {
            if (threadIdx.x == 0)
                set_status(a.status, DV_ERR_DEVICE_INDEX);
            x.h = -1;
        }
        x.ntok = a.n_tok ? __ldg(a.n_tok + b) : a.T;
        x.row0 = m * rows;
        x.nrows = min(rows, x.ntok * G - x.row0);
        x.ent = 0;
    }
    return x;
}

// Offset of a unit's query row among the given ones, and of its result.
template <bool BLOCK>
DV_DEV long long q_at(const KvAttnArgs &a, const Unit &x, int r)
{
    if (BLOCK)
        return x.b * a.q.sb + x.h * a.q.sh;
    const int G = a.H / a.c.Hkv, t = (x.row0 + r) / G, g = (x.row0 + r) - t * G;
    return x.b * a.q.sb + t * a.q.st + (long long)(x.h * G + g) * a.q.sh;
}
template <bool BLOCK>
DV_DEV size_t out_at(const KvAttnArgs &a, const Unit &x, int r)
{
    if (BLOCK)
        return ((size_t)x.b * a.H + x.h) * a.c.D;
    const int G = a.H / a.c.Hkv, t = (x.row0 + r) / G, g = (x.row0 + r) - t * G;
    return (((size_t)x.b * a.T + t) * a.H + x.h * G + g) * a.c.D;
}

// Drafted tokens that token t of row b sees, as bits below the row's count.
DV_DEV unsigned long long seen_bits(const KvAttnArgs &a, const Unit &x, int t)
{
    const unsigned long long all = x.ntok >= 64 ? ~0ull : (1ull << x.ntok) - 1;
    const unsigned long long m =
        a.mask ? __ldg(a.mask + (size_t)x.b * a.T + t) : (t >= 63 ? ~0ull : (2ull << t) - 1);
    return m & all;
}

// Cached position of place i of a unit's tile sequence in block mode, -1
// where there is none.
DV_DEV int block_pos(const KvAttnArgs &a, const Unit &x, int i)
{
    const int lg = a.blog, e = i >> lg;
    if (e >= x.ent)
        return -1;
    const int j = __ldg(a.idx + ((size_t)x.b * a.H + x.h) * a.k + e);
    if (j < 0 || j > (x.len - 1) >> lg) {
        if (j != -1)
            set_status(a.status, DV_ERR_DEVICE_INDEX);
        return -1;
    }
    const int p = (j << lg) + (i & (a.c.block - 1));
    return p < x.len ? p : -1;
}

DV_DEV float row_result(float o, float l) { return l == 0.f ? 0.f : o / l; }

constexpr int kMergePieces = 16;  // pieces whose weights are in shared memory at a time

// A run's part of a unit is done: so[RM * D] (in the kernel's own order: at(row,
// d) is the place of a value), u_m, u_l [RM] hold it merged over the CTA,
// visible to every thread (m in units of log2).  Writes the result, or a
// piece, and merges the pieces if it is the last.  Every thread of the CTA
// (NTHR of them) calls it; the buffers may be reused after it returns.
template <bool BLOCK, int RM, int NTHR, class F, class R>
DV_DEV void finish_unit(const KvAttnArgs &a, const Run &r, const Unit &x, SchedSmem &sm,
                        float *so, float *u_m, float *u_l, float (*wgt)[RM], F at, R rowof)
{
    const int D = a.c.D, n4 = RM * D / 4;
    if (!(r.lo <= x.w0 && x.w1 <= r.hi)) {
        const size_t rsz = (size_t)RM * (D + 2);
        float *rec = a.rec + (2 * (size_t)r.c + (x.w0 > r.lo)) * rsz;
        for (int i = threadIdx.x; i < n4; i += NTHR)
            __stcg(reinterpret_cast<float4 *>(rec) + i, reinterpret_cast<const float4 *>(so)[i]);
        for (int i = threadIdx.x; i < RM; i += NTHR) {
            __stcg(rec + RM * D + i, u_m[i]);
            __stcg(rec + RM * D + RM + i, u_l[i]);
        }
        __threadfence();
        __syncthreads();
        const int c0 = (int)(((x.w0 + 1) * r.C - 1) / r.W), c1 = (int)((x.w1 * r.C - 1) / r.W);
        if (threadIdx.x == 0)
            sm.last = atomicAdd(a.cnt + c0, 1) == c1 - c0;
        __syncthreads();
        if (!sm.last)
            return;
        __threadfence();
        // record of piece c (the unit's first CTA has it after its run's start, or at it)
        auto piece = [&](int c) {
            const bool late = c == c0 && x.w0 > r.W * c / r.C;
            return a.rec + (2 * (size_t)c + late) * rsz;
        };
        const int lane = threadIdx.x & 31;
        for (int row = threadIdx.x >> 5; row < RM; row += NTHR / 32) {
            float M = -INFINITY, L = 0.f;
            for (int c = c0 + lane; c <= c1; c += 32)
                M = fmaxf(M, __ldcg(piece(c) + RM * D + row));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
            const float ms = M == -INFINITY ? 0.f : M;
            for (int c = c0 + lane; c <= c1; c += 32) {
                const float *p = piece(c) + RM * D;
                L = fmaf(__ldcg(p + RM + row), exp2f(__ldcg(p + row) - ms), L);
            }
            L = warp_sum(L);
            if (lane == 0) {
                u_m[row] = ms;
                u_l[row] = L;
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < n4; i += NTHR)
            reinterpret_cast<float4 *>(so)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int cb = c0; cb <= c1; cb += kMergePieces) {
            const int nc = min(kMergePieces, c1 - cb + 1);
            for (int i = threadIdx.x; i < nc * RM; i += NTHR) {
                const int k = i / RM, row = i - k * RM;
                wgt[k][row] = exp2f(__ldcg(piece(cb + k) + RM * D + row) - u_m[row]);
            }
            __syncthreads();
            for (int i = threadIdx.x; i < n4; i += NTHR) {
                float4 acc = reinterpret_cast<float4 *>(so)[i];
                const int row = rowof(4 * i);
#pragma unroll 8
                for (int k = 0; k < nc; ++k) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(piece(cb + k)) + i);
                    const float wt = wgt[k][row];
                    // (a piece without a seen position has zeros, whatever else is NaN)
                    acc.x = fmaf(v.x, wt, acc.x);
                    acc.y = fmaf(v.y, wt, acc.y);
                    acc.z = fmaf(v.z, wt, acc.z);
                    acc.w = fmaf(v.w, wt, acc.w);
                }
                reinterpret_cast<float4 *>(so)[i] = acc;
            }
            __syncthreads();
        }
        if (threadIdx.x == 0)
            a.cnt[c0] = 0;  // ready for the next call
    }
    const int lg = __ffs(D) - 1;
    for (int i = threadIdx.x; i < x.nrows * D; i += NTHR) {
        const int row = i >> lg, d = i & (D - 1);
        a.out[out_at<BLOCK>(a, x, row) + d] = row_result(so[at(row, d)], u_l[row]);
    }
    __syncthreads();
}

}  // namespace
}  // namespace dv
