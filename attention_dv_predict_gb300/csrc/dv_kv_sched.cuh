// dv_kv_sched.cuh -- how the KV attention kernels share their work (sm_103a).
//
// A unit is up to `rows` query rows (token-major: row = token G + group
// member) of one (batch row, KV head) -- of one (batch row, query head) in
// block mode -- and its work is the tiles of 64 cached positions it sees.
// Lengths differ from row to row and are known on the device only, so the
// tiles of all units are laid end to end, each unit's behind kUnitCost empty
// places for what a unit costs beside its tiles, and the grid's C CTAs take
// equal runs: CTA c the places [W c / C, W (c + 1) / C), an end among a
// unit's empty places counting as the unit's start.  (Without them a ragged
// batch's short rows all fell to a few CTAs: 32 rows of 1 to 8000 positions,
// 48 blocks of 32 for each of 64 heads, 420 us against 188.)  A unit inside
// one run is finished by its CTA; a unit cut by a run's end leaves a piece
// (max m, sum l, weighted values o, per row) in a record, and the last of its
// CTAs to arrive merges the pieces in the order of the positions, so the
// result does not depend on who was last.  At most one cut unit starts in a
// CTA's run, so a counter per CTA is enough, and a CTA has at most two
// pieces: one that began before its run (or at its start), one that goes on
// after it.  No CTA waits for another.
#pragma once

#include "dv_kv.cuh"

namespace dv {
namespace {

constexpr int kUnitCost = 4;  // tiles that a unit's start and end take the time of

struct SchedSmem {
    long long pref[DV_KV_MAX_BATCH + 1];  // places before batch row b
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
    long long w0, w1; // its places, its tiles from w0 + kUnitCost on
};

struct Run {
    long long W, lo, hi;
    int C, c, nsel;
};

// a / b for 0 <= a, 0 < b: in 32 bits where that does (a 64-bit division is a
// subroutine of some 100 instructions, and a CTA starts with several).
DV_DEV long long quot(long long a, long long b)
{
    return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// The batch row of place w.
DV_DEV int sched_row(const KvAttnArgs &a, const SchedSmem &sm, long long w)
{
    int b = 0;
    for (int step = 128; step > 0; step >>= 1)  // largest b with pref[b] <= w
        if (b + step < a.B && sm.pref[b + step] <= w)
            b += step;
    return b;
}

// w, or the start of the unit whose empty places it is among.
DV_DEV long long sched_snap(const KvAttnArgs &a, const SchedSmem &sm, long long w)
{
    const int b = sched_row(a, sm, w), size = sm.tiles[b] + kUnitCost;
    if (w >= sm.pref[a.B])
        return w;
    const long long at = w - sm.pref[b];
    const int in = (int)(at - quot(at, size) * size);
    return in <= kUnitCost ? w - in : w;
}

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
        sm.pref[b + 1] = (long long)(tiles ? tiles + kUnitCost : 0) * mb * nsel;
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
    r.lo = r.c < r.C ? sched_snap(a, sm, quot(r.W * r.c, r.C)) : 0;
    r.hi = r.c < r.C ? sched_snap(a, sm, quot(r.W * (r.c + 1), r.C)) : 0;
    return r;
}

// The unit of place w (0 <= w < W).
template <bool BLOCK>
DV_DEV Unit sched_unit(const KvAttnArgs &a, int rows, const SchedSmem &sm, const Run &r,
                       long long w)
{
    const int b = sched_row(a, sm, w), size = sm.tiles[b] + kUnitCost, mb = sm.mb[b];
    const int u = (int)quot(w - sm.pref[b], size);
    const int j = u / mb, m = u - j * mb;
    Unit x;
    x.b = b;
    x.w0 = sm.pref[b] + (long long)u * size;
    x.w1 = x.w0 + size;
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
            if ((threadIdx.x & 31) == 0)
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

// Tile of place w of unit x; the first place from w on that has one.
DV_DEV int tile_of(const Unit &x, long long w) { return (int)(w - x.w0) - kUnitCost; }
DV_DEV long long tile_place(const Unit &x, long long w) { return max(w, x.w0 + kUnitCost); }

// Drafted token of query row n (n / group size; n < 2^14).
DV_DEV int row_token(const KvAttnArgs &a, int n) { return (int)((n + 0.5f) * a.r_group); }

// Offset of a unit's query row among the given ones, and of its result.
template <bool BLOCK>
DV_DEV long long q_at(const KvAttnArgs &a, const Unit &x, int r)
{
    if (BLOCK)
        return x.b * a.q.sb + x.h * a.q.sh;
    const int G = a.H / a.c.Hkv, t = row_token(a, x.row0 + r), g = (x.row0 + r) - t * G;
    return x.b * a.q.sb + t * a.q.st + (long long)(x.h * G + g) * a.q.sh;
}
template <bool BLOCK>
DV_DEV size_t out_at(const KvAttnArgs &a, const Unit &x, int r)
{
    if (BLOCK)
        return ((size_t)x.b * a.H + x.h) * a.c.D;
    const int G = a.H / a.c.Hkv, t = row_token(a, x.row0 + r), g = (x.row0 + r) - t * G;
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

// l 2^d, also where l is large and 2^d below binary32's range (the references of
// pieces whose value scales lie far apart).
DV_DEV float sum_shift(float l, float d)
{
    return l * exp2f(fmaxf(d, -120.f)) * exp2f(fminf(d + 120.f, 0.f));
}

// o / l by the reciprocal (one more rounding); 0 where nothing was seen.
DV_DEV float4 row_result(const float4 &o, float l)
{
    const float r = l == 0.f ? 0.f : __frcp_rn(l);
    return make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
}

constexpr int kMergePieces = 32;  // pieces whose weights are held in shared memory

struct CtaSync {
    DV_DEV static void sync() { __syncthreads(); }
};

// What becomes of a run's part of each unit.  NTHR threads (which meet in S)
// call it together.
template <bool BLOCK, int RM, int NTHR, class S = CtaSync>
struct Finish {
    long long w[2];  // first place of the units this CTA left a piece of
    int got[2], n = 0;

    // A part is done: val(row, d) and u_m, u_l [RM] give it merged over the
    // CTA, visible to every thread (m in units of log2).  Writes the result,
    // or a piece; whether the piece was the last of its unit is asked for
    // here and looked at in end(), a memory round trip later.
    template <class F>
    DV_DEV void part(const KvAttnArgs &a, const Run &r, const Unit &x, F val, const float *u_m,
                     const float *u_l)
    {
        const int D = a.c.D, lg = __ffs(D) - 1, items = x.nrows * D / 4;
        const bool all = whole(r, x);
        float *rec = record(a, r, x);
        for (int i = threadIdx.x; i < items; i += NTHR) {
            const int row = (4 * i) >> lg, d = (4 * i) & (D - 1);
            const float4 v =
                make_float4(val(row, d), val(row, d + 1), val(row, d + 2), val(row, d + 3));
            if (all)
                *reinterpret_cast<float4 *>(a.out + out_at<BLOCK>(a, x, row) + d) =
                    row_result(v, u_l[row]);
            else
                __stcg(reinterpret_cast<float4 *>(rec) + i, v);
        }
        if (!all)
            for (int i = threadIdx.x; i < x.nrows; i += NTHR) {
                __stcg(rec + RM * D + i, u_m[i]);
                __stcg(rec + RM * D + RM + i, u_l[i]);
            }
        done(a, r, x);
    }

    // The unit lies within the run; the record of this CTA's piece of it, [RM][D]
    // values, then m and l [RM] each.
    DV_DEV static bool whole(const Run &r, const Unit &x) { return r.lo <= x.w0 && x.w1 <= r.hi; }
    DV_DEV static float *record(const KvAttnArgs &a, const Run &r, const Unit &x)
    {
        return a.rec + (2 * (size_t)r.c + (x.w0 > r.lo)) * ((size_t)RM * (a.c.D + 2));
    }

    // The part's stores are made.
    DV_DEV void done(const KvAttnArgs &a, const Run &r, const Unit &x)
    {
        S::sync();
        if (!whole(r, x)) {
            // release of the CTA's stores above (ordered before it by the
            // barrier), acquire of the other pieces'
            if (threadIdx.x == 0) {
                int was;
                asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;"
                             : "=r"(was)
                             : "l"(a.cnt + first_cta(r, x))
                             : "memory");
                got[n & 1] = was;
            }
            w[n++ & 1] = x.w0;
        }
    }

    DV_DEV static int first_cta(const Run &r, const Unit &x)
    {
        return (int)quot((x.w0 + kUnitCost + 1) * r.C - 1, r.W);
    }

    // The run is over: merges the units whose last piece was this CTA's, in
    // the order of their positions.
    DV_DEV void end(const KvAttnArgs &a, const Run &r, SchedSmem &sm, float *u_m, float *u_l,
                    float (*wgt)[RM])
    {
        const int D = a.c.D, lg = __ffs(D) - 1, lane = threadIdx.x & 31;
        const size_t rsz = (size_t)RM * (D + 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (i >= n)
                break;
            const Unit x = sched_unit<BLOCK>(a, RM, sm, r, w[i]);
            const int c0 = first_cta(r, x), c1 = (int)quot(x.w1 * r.C - 1, r.W), np = c1 - c0 + 1;
            if (threadIdx.x == 0)
                sm.last = got[i] == np - 1;
            S::sync();
            const bool last = sm.last;
            S::sync();
            if (!last)
                continue;
            // records: the unit's first CTA has it after its run's start, or at it
            const float *rec0 = a.rec + (2 * (size_t)c0 + (x.w0 > quot(r.W * c0, r.C))) * rsz;
            auto piece = [&](int k) {
                return k == 0 ? rec0 : a.rec + 2 * (size_t)(c0 + k) * rsz;
            };
            for (int row = threadIdx.x >> 5; row < x.nrows; row += NTHR / 32) {
                float M = -INFINITY, L = 0.f, mine = -INFINITY;
                for (int k = lane; k < np; k += 32) {
                    const float *p = piece(k) + RM * D + row;
                    const float m = __ldcg(p), l = __ldcg(p + RM);
                    const float mn = fmaxf(M, m), ms = mn == -INFINITY ? 0.f : mn;
                    L = sum_shift(L, M - ms) + sum_shift(l, m - ms);
                    M = mn;
                    if (k < 32)
                        mine = m;
                }
                float top = M;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float ms = top == -INFINITY ? 0.f : top;
                L = warp_sum(sum_shift(L, M - ms));
                if (lane < kMergePieces)
                    wgt[lane][row] = exp2f(mine - ms);
                if (lane == 0) {
                    u_m[row] = ms;
                    u_l[row] = L;
                }
            }
            S::sync();
            for (int it = threadIdx.x; it < x.nrows * D / 4; it += NTHR) {
                const int row = (4 * it) >> lg, d = (4 * it) & (D - 1);
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int k = 0; k < np; ++k) {
                    const float *p = piece(k);
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(p) + it);
                    const float wt = k < kMergePieces
                                         ? wgt[k][row]
                                         : exp2f(__ldcg(p + RM * D + row) - u_m[row]);
                    acc.x = fmaf(v.x, wt, acc.x);
                    acc.y = fmaf(v.y, wt, acc.y);
                    acc.z = fmaf(v.z, wt, acc.z);
                    acc.w = fmaf(v.w, wt, acc.w);
                }
                *reinterpret_cast<float4 *>(a.out + out_at<BLOCK>(a, x, row) + d) =
                    row_result(acc, u_l[row]);
            }
            if (threadIdx.x == 0)
                a.cnt[c0] = 0;  // ready for the next call
            S::sync();
        }
    }
};

}  // namespace
}  // namespace dv
