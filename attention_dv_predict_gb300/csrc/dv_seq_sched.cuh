// dv_seq_sched.cuh -- how attention over packed sequences shares its work
// (sm_103a).
//
// A unit is a piece of one request's tokens with the query heads of one group
// of a KV head: ROWS rows (row = token x group + head), or with PAIR twice that
// where the request has that many left.  Its work is the tiles of TP cached
// positions that its last token sees.  Token counts and lengths are known on
// the device only, so the tiles of all units are laid end to end (request,
// head, tokens), each unit's behind COST empty places for what a unit
// costs beside its tiles and two places a tile for a pair, and C CTAs take
// equal runs of places, each the tiles that begin in its run.  A unit inside
// one run is finished by its CTA; of a unit cut by a run's end every CTA leaves
// a piece in a record, and the last to arrive merges them in the order of the
// positions, so the result does not depend on who was last.  At most one cut
// unit starts in a run, so a counter per CTA is enough, and a CTA has at most
// two pieces.  No CTA waits for another.
//
// The place of a unit's first tile is a closed form (tokens of a unit are a
// power of two): a CTA finds its run by a scan over the requests and a binary
// search, and then steps from unit to unit.  Every role of a CTA steps through
// the same units by itself.
#pragma once

#include "dv_common.cuh"
#include "dv_seq.h"

namespace dv {
namespace {

struct SeqSmem {
    long long part[33];
    long long base;
    int b;
};

struct SeqRun {
    long long W, lo, hi, base;  // all places; this run; the place of request b's first unit
    int C, c, b;                // runs, this run, the request of place lo
};

// One request: its first packed row, tokens and cached positions.  n = 0 for
// one that is out of range.
struct SeqRow {
    int t0, n, len;
};

DV_DEV SeqRow seq_row(const SeqAttnArgs &a, int b, bool report)
{
    SeqRow r;
    r.t0 = __ldg(a.cu + b);
    const int t1 = __ldg(a.cu + b + 1);
    r.len = a.lens ? __ldg(a.lens + b) : 0;
    const long long n = (long long)t1 - r.t0;
    bool ok = r.t0 >= 0 && n >= 0 && n <= a.max_tok && t1 <= a.T && r.len >= 0;
    if (a.pk)
        ok = ok && r.len + n <= (long long)a.width * a.page;
    if (!ok && report)
        set_status(a.status, DV_ERR_DEVICE_INDEX);
    r.n = ok ? (int)n : 0;
    return r;
}

// a / b for 0 <= a, 0 < b: in 32 bits where that does (a 64-bit division is a
// subroutine of some 100 instructions, and a CTA starts with several).
DV_DEV long long seq_quot(long long a, long long b)
{
    return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

template <int TP_, bool PAIR_, int COST_, int MIN_RUN_>
struct SeqSched {
    static constexpr int TP = TP_, COST = COST_, MIN_RUN = MIN_RUN_;
    static constexpr bool PAIR = PAIR_;
    static constexpr int TPLOG = 6;
    static_assert(TP == 1 << TPLOG && MIN_RUN >= 4, "a run holds a tile's start");

    DV_DEV static int tiles(int len, int e) { return (int)(((long long)len + e + TP - 1) >> TPLOG); }
    // Tiles of the first m whole units (2^u tokens each): the sum of
    // ceil((len + 2^u i) / TP) over i = 1 .. m.
    DV_DEV static long long sum_tiles(int len, int u, long long m)
    {
        if (u >= TPLOG)
            return m * ((len + TP - 1) >> TPLOG) + ((m * (m + 1) / 2) << (u - TPLOG));
        const int r = TPLOG - u;
        auto upto = [r](long long x) {  // the sum of ceil(y / 2^r) over y = 1 .. x
            const long long q = x >> r;
            return ((q * (q + 1) / 2) << r) + (x & ((1 << r) - 1)) * (q + 1);
        };
        const long long l = ((long long)len + (1 << u) - 1) >> u;
        return upto(l + m) - upto(l);
    }
    DV_DEV static int ulog(const SeqAttnArgs &a) { return a.tlog + PAIR; }
    DV_DEV static long long whole(const SeqAttnArgs &a, int len, long long m)
    {
        return m * COST + (sum_tiles(len, ulog(a), m) << PAIR);
    }
    // Places of a request's units of one group of heads.
    DV_DEV static long long places(const SeqAttnArgs &a, const SeqRow &r)
    {
        const int u = ulog(a), rem = r.n & ((1 << u) - 1);
        long long w = whole(a, r.len, r.n >> u);
        if (rem)
            w += COST + ((long long)tiles(r.len, r.n) << (PAIR && rem > 1 << a.tlog));
        return w;
    }

    // Every thread of the CTA calls it.  (At most 1024 threads, whole warps.)
    DV_DEV static SeqRun init(const SeqAttnArgs &a, SeqSmem &sm)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        const int hs = a.H / a.group;
        long long v = 0, before = 0;
        // the places before request b0 + threadIdx.x and their sum through the block
        auto scan = [&](int b0, bool report) {
            const int b = b0 + threadIdx.x;
            v = b < a.B ? places(a, seq_row(a, b, report)) * hs : 0;
            long long inc = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                inc += lane >= o ? t : 0;
            }
            __syncthreads();
            if (lane == 31)
                sm.part[warp] = inc;
            __syncthreads();
            long long all = 0;
            before = inc - v;
#pragma unroll 1
            for (int w = 0; w < nw; ++w) {
                before += w < warp ? sm.part[w] : 0;
                all += sm.part[w];
            }
            return all;
        };
        SeqRun r;
        r.W = 0;
        auto runs = [&]() {
            r.C = (int)min((long long)gridDim.x, max(1ll, r.W / MIN_RUN));
            r.c = blockIdx.x;
            r.lo = r.c < r.C ? seq_quot(r.W * r.c, r.C) : r.W;
            r.hi = r.c < r.C ? seq_quot(r.W * (r.c + 1), r.C) : r.W;
        };
        if (a.B <= 32) {  // every warp for itself: no barrier between them
            v = lane < a.B ? places(a, seq_row(a, lane, blockIdx.x == 0 && warp == 0)) * hs : 0;
            before = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, before, o);
                before += lane >= o ? t : 0;
            }
            r.W = __shfl_sync(0xffffffffu, before, 31);
            before -= v;
            runs();
            const unsigned in = __ballot_sync(0xffffffffu, before <= r.lo && r.lo < before + v);
            r.b = in ? __ffs(in) - 1 : 0;
            r.base = __shfl_sync(0xffffffffu, before, r.b);
            return r;
        }
        const int step = blockDim.x;
        for (int b0 = 0; b0 < a.B; b0 += step)
            r.W += scan(b0, blockIdx.x == 0);
        runs();
        long long base = 0;
        for (int b0 = 0; b0 < a.B; b0 += step) {
            const long long all = a.B <= step ? 0 : scan(b0, false);
            const long long at = base + before;
            if (at <= r.lo && r.lo < at + v) {
                sm.b = b0 + threadIdx.x;
                sm.base = at;
            }
            base += all;
        }
        __syncthreads();
        r.b = r.lo < r.hi ? sm.b : 0;
        r.base = r.lo < r.hi ? sm.base : 0;
        return r;
    }

    // What a role works through: the pieces of units in this run.
    struct Piece {
        int tok, ntok;  // first packed row and tokens of the unit
        int pos;        // position of its first token
        int h0, hkv;    // first query head, KV head
        int b;
        int nt, k0, k1; // the unit's tiles; this run's are k0 .. k1 - 1
        int c0, c1;     // runs that have tiles of it (c0 = c1: finished here)
        bool pair;      // more than 2^tlog tokens
    };

    // Where a role is: the request, its group of heads and unit that come next.
    struct Walk {
        SeqRow row;
        int b, hs, i;
        long long u0;  // the unit's place

        DV_DEV void start(const SeqAttnArgs &a, const SeqRun &r)
        {
            row = SeqRow{0, 0, 0};
            b = r.b;
            hs = i = 0;
            u0 = r.hi;
            if (r.lo >= r.hi)
                return;
            row = seq_row(a, b, false);
            const long long per = places(a, row), at = r.lo - r.base;
            hs = (int)seq_quot(at, per);
            const long long rest = at - hs * per;
            // the last whole unit, or the partial one behind them, that starts by `rest`
            int lo = 0, hi = units(a) - 1;
#pragma unroll 1
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (whole(a, row.len, mid) <= rest)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            i = lo;
            u0 = r.lo - (rest - whole(a, row.len, i));
        }
        DV_DEV int units(const SeqAttnArgs &a) const
        {
            return (row.n + (1 << ulog(a)) - 1) >> ulog(a);
        }
        // The next piece, false behind the last.
        DV_DEV bool next(const SeqAttnArgs &a, const SeqRun &r, Piece &p)
        {
#pragma unroll 1
            while (u0 < r.hi) {
                const int first = i << ulog(a);
                p.ntok = min(1 << ulog(a), row.n - first);
                p.tok = row.t0 + first;
                p.pos = row.len + first;
                p.nt = tiles(row.len, first + p.ntok);
                p.pair = PAIR && p.ntok > 1 << a.tlog;
                p.b = b;
                p.h0 = hs * a.group;
                p.hkv = a.sub == 1 ? hs : hs / a.sub;
                const int wt = p.pair;  // (log2 of a tile's places)
                const long long t0 = u0 + COST, end = t0 + ((long long)p.nt << wt);
                const bool head = t0 >= r.lo, tail = end <= r.hi;  // its first, last tile is here
                p.k0 = 0;
                p.k1 = p.nt;
                p.c0 = p.c1 = r.c;
                if (!head || !tail) {
                    p.k0 = (int)max(0ll, (r.lo - t0 + wt) >> wt);
                    p.k1 = (int)max(0ll, min((long long)p.nt, (r.hi - t0 + wt) >> wt));
                    if (p.k0 > 0)
                        p.c0 = run_of(r, t0);
                    if (p.k1 < p.nt)
                        p.c1 = run_of(r, t0 + ((long long)(p.nt - 1) << wt));
                }
                u0 = end;
                if (++i >= units(a)) {
                    i = 0;
                    if (++hs == a.H / a.group) {
                        hs = 0;
#pragma unroll 1
                        do {
                            if (++b < a.B)
                                row = seq_row(a, b, false);
                        } while (b < a.B && row.n == 0);
                        if (b >= a.B)
                            u0 = max(u0, r.hi);
                    }
                }
                if (p.k0 < p.k1)
                    return true;
            }
            return false;
        }
    };
    // The run that place w falls to: the last c with floor(W c / C) <= w.
    DV_DEV static int run_of(const SeqRun &r, long long w)
    {
        return (int)seq_quot((w + 1) * r.C - 1, r.W);
    }
    // Record of run c's piece of a unit that starts in run c0.
    DV_DEV static int slot(int c, int c0) { return 2 * c + (c == c0); }
};

}  // namespace
}  // namespace dv
