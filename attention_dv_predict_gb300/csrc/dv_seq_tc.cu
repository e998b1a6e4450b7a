// dv_seq_tc.cu -- causal attention of packed sequences on tcgen05 (sm_103a):
// binary16 rows of 64 or 128 values, packed or in pages.
//
// A unit's query rows fill one or two M = 128 tiles.  Two streams of softmax,
// four warps each with a row a thread, share the tensor cores.  A unit of two
// tiles (a pair: prompts, chunks) gives each stream its own rows and the same
// positions; a unit of one (decode, a chunk's end) gives both the same rows and
// every other tile of positions, and they are merged when it ends.  Scores lie
// in tensor memory, the weights (binary16) take their place as the A operand of
// the value product, and the outputs are summed there in binary32.
//
// A tile is 64 positions and a stream has two score buffers, so that the next
// tile's scores are there when a softmax warp gets to them and the products of
// both streams run back to back: a tile of 128 (whose scores fill tensor memory
// with one buffer a stream) left the tensor cores waiting for every softmax.
// Per pair tile the score products take 384 cycles each (bound by their reads
// of shared memory) and the value products 256.
//
// Warps of a CTA (one CTA per SM):
//   0-3, 4-7  softmax of stream 0, 1
//   8         copies of keys and values: a ring of tiles; of a paged cache a
//             lane a page, the page numbers a tile ahead
//   9, 10     the products of stream 0, 1 (one thread each issues them: an issue
//             takes as long as the product before runs, and a wait for a barrier
//             100 cycles even if it is over, so with one warp for both streams the
//             tensor cores idled half of the time)
//   11        copies of queries; takes NaN and infinities out of value rows that
//             some row of the unit does not see (only its last tiles hold any)
// Hand-overs are mbarriers; every wait has a limit (DV_ERR_TIMEOUT).
//
// A row's reference point m stands in for its running maximum: weights are
// 2^(s - m) with m a whole number 6 below the first tile's maximum, and m moves
// (for this row alone) when a weight would pass 2^15, near the end of binary16's
// range, so the outputs are rarely rescaled.
//
// A weight is one binary16 number (2^-11 of itself), rounded as the result is: both
// together leave 2.6e-4 to 3e-4 of the results against 64 bits, the result's own
// rounding alone 2.1e-4.  Two parts, as the operators with binary32 results have, would
// be a second value product, 256 cycles more beside the 640 of a stream's tile.
//
// A stream's buffers: with tiles c - 2, c - 1, c, ... of a stream's own, the scores
// of c take the place of the weights of c - 2, whose value product has been issued
// (an entry of the ring brings values two tiles of the run behind its keys, and a
// stream's c - 2 is at least that far behind its c).
#include <cudaTypedefs.h>

#include "dv_kv_tma.cuh"
#include "dv_seq_sched.cuh"

namespace dv {
namespace {

struct SeqMaps {
    CUtensorMap q, k, v, out;
};

// What a unit costs beside its tiles, and the shortest run, in places: swept over
// single tokens, short and long prompts and a mix of them (a unit of 6: the mix 476
// us, ragged prompts 374; of 12: 409 and 338; of 20: 416 and 346; with sums of rounded
// weights and outputs set aside, both later, 12 takes 415 and 359).
using TcSched = SeqSched<64, true, 12, 12>;

// PAGED: keys and values of a pool.  Their tiles are laid out by groups of 8 rows,
// a group's 64-dimension halves side by side, so that one copy brings a whole page
// (as two halves of 64 rows each, like packed rows', 64 rows of 8 x 8 heads over
// 4096 positions took 248 us in pages of 16, and 198 so).
// FEW: no unit has more than 32 rows (decode): none is a pair, and the room that
// queries and results do not need is two more stages of the ring (pages of 64: 182
// us with three, 172 with five).
template <int D_, bool PAGED_, bool FEW_>
struct SeqTcCfg {
    static constexpr bool PAGED = PAGED_, FEW = FEW_;
    static constexpr int D = D_, TP = 64, RM = 128;
    static constexpr int TILE = TP * D * 2, HALF = TP * 128;    // keys or values; 64 dimensions
    static constexpr int GROUP = PAGED ? D * 16 : 1024;         // bytes from 8 rows to the next 8
    static constexpr int KHALF = PAGED ? 1024 : HALF;           // and to their other half
    static constexpr int QTILE = RM * D * 2, QHALF = RM * 128;  // queries of 128 rows
    static constexpr int NST = D == 128 ? (FEW ? 5 : 3) : 8;    // ring stages
    static constexpr int THREADS = 384;
    static constexpr int XROWS = FEW ? 32 : RM;                 // rows that streams exchange
    static constexpr int OUT = XROWS * D * 2;                   // a stream's results
    static constexpr int OFF_KV = (FEW ? 1 : 2) * QTILE, OFF_OUT = OFF_KV + NST * 2 * TILE,
                         OFF_CTL = OFF_OUT + 2 * OUT;
    static constexpr int T_S = 0, T_O = 256, T_COLS = 512;  // tensor-memory columns
    static constexpr int REC = 2 * RM * D + 4 * RM;      // floats of a piece's record
    static constexpr int ACC = RM * D + RM;              // and of what a stream has set aside
    using Sched = TcSched;
};

// Control block behind the ring.
struct SeqCtl {
    SeqSmem sched;
    uint64_t full[8], empty[8], q_full[2];
    uint64_t s_full[2][2], p_full[2][2];  // scores and weights of a stream's buffers
    uint64_t o_full[2][2];                // the value product with a buffer's weights is done
    // A unit's score products are done: of a pair's streams each; of both.
    uint64_t q_free[2], q_both;
    // Edge tiles, by their number modulo 8.  (With no more ring stages than that a
    // slot is used again only after both streams have released its tile's values.)
    uint64_t v_req[8], v_ok[8];
    uint64_t end[2];
    float m[2][128], l[2][128];  // exchange of a unit of one tile
    unsigned bad[8][2];          // positions of an edge tile that were not finite
    int last[2];
    unsigned tmem;
    SeqRun run;
    int4 plan[2][4];             // a products' warp: pieces between their keys and values
};

DV_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
DV_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
DV_DEV void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle: 8-row groups sbo bytes
// apart; lbo: bytes between 64-element blocks of an MN-major operand.
DV_DEV uint64_t tc_desc(unsigned saddr, unsigned lbo, unsigned sbo)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(sbo >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16, f32 accumulate, M = 128, N columns; tb: B is MN-major.
__host__ __device__ constexpr uint32_t tc_idesc(int N, bool tb)
{
    return (1u << 4) | (tb ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}
DV_DEV void tc_mma_ss(unsigned d, uint64_t ad, uint64_t bd, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(ad), "l"(bd), "r"(idesc), "r"((int)acc)
        : "memory");
}
DV_DEV void tc_mma_ts(unsigned d, unsigned a, uint64_t bd, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bd), "r"(idesc), "r"((int)acc)
        : "memory");
}
DV_DEV void tc_commit(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
            smem_addr(bar))
        : "memory");
}
// 32 columns of a thread's lane of tensor memory.
DV_DEV void tm_ld(unsigned addr, float *v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, "
                 "%26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
                   "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]),
                   "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
                   "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]),
                   "=f"(v[30]), "=f"(v[31])
                 : "r"(addr));
}
// The loads into v have landed (v passes through, so that no use moves before it).
DV_DEV void tm_wait_ld(float *v)
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                   "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                   "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                   "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                   "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                   "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}
// 16 columns, landed.
DV_DEV void tm_ld16(unsigned addr, float *v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
                 "%14, %15}, [%16];"
                 "\n\ttcgen05.wait::ld.sync.aligned;"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]),
                   "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                 : "r"(addr)
                 : "memory");
}
DV_DEV void tm_st16(unsigned addr, const unsigned *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
                 "%15, %16};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]),
                 "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}
// 8 columns.
DV_DEV void tm_st8(unsigned addr, const unsigned *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                     addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
                 : "memory");
}
DV_DEV void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// From a page: its groups of 8 rows from `group` on, whole rows.
DV_DEV void tma_load_page(unsigned dst, const CUtensorMap *map, int group, int z, unsigned bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %2, %2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(0), "r"(group), "r"(z), "r"(bar)
        : "memory");
}
// A box of shared memory to (dimension, head, token) of the results.
DV_DEV void tma_store(const CUtensorMap *map, int x, int h, int tok, unsigned src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     map),
                 "r"(x), "r"(h), "r"(tok), "r"(src)
                 : "memory");
}

DV_DEV bool elect_one()
{
    unsigned p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(p));
    return p != 0;
}
DV_DEV float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// Sums of the weights as rounded, so that a row's weights add up to 1 whatever
// their rounding: a row of one position is that position's value.
DV_DEV void add_pair(float &a, float &b, unsigned pair)
{
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
        "add.rn.f32.f16 %0, x, %0;\n\tadd.rn.f32.f16 %1, y, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(pair));
}
template <int N>
DV_DEV void group_sync(int bar)
{
    asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(N) : "memory");
}

// Whether the phase with this parity is complete, without waiting.
DV_DEV bool seq_test(uint64_t *bar, unsigned parity)
{
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity & 1)
        : "memory");
    return ok;
}
// The same; may wait a little.
DV_DEV bool seq_try(unsigned bar, unsigned parity)
{
    unsigned ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity & 1)
        : "memory");
    return ok;
}
// True once the phase with this parity is complete; false after 2^21 polls of
// at most a microsecond each.
__device__ __noinline__ bool seq_wait_on(unsigned bar, unsigned parity)
{
#pragma unroll 1
    for (int it = 0; it < kKvSpin; ++it) {
        unsigned ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity & 1), "r"(1000)
            : "memory");
        if (ok)
            return true;
    }
    return false;
}
DV_DEV bool seq_wait(uint64_t *bar, unsigned parity)
{
    return seq_try(smem_addr(bar), parity) || seq_wait_on(smem_addr(bar), parity);
}

// A role's waits: after one has run out the others no longer wait (the
// results are lost, the status says so, every loop still ends).  What is over
// already costs a poll and a branch.
struct SeqWaiter {
    int *status;
    bool dead = false;
    DV_DEV void operator()(uint64_t *bar, unsigned parity)
    {
        if (!seq_try(smem_addr(bar), parity) && !dead && !seq_wait_on(smem_addr(bar), parity)) {
            dead = true;
            set_status(status, DV_ERR_TIMEOUT);
        }
    }
};

// A piece's tiles as both streams see them.  Entry e of the ring holds the keys
// of the run's tile e and the values of its tile e - 2, which are used together
// (two tiles' scores are computed ahead, of the next piece too): one wait for both.
template <class C>
struct Plan {
    int n, n0;       // tiles; of them, a pair's first 128 rows' own
    int edge;        // first tile (of the piece) that some row does not see whole
    bool pair;
    DV_DEV Plan(const SeqAttnArgs &a, const typename C::Sched::Piece &x)
    {
        pair = !C::FEW && x.pair;
        n = x.k1 - x.k0;
        n0 = pair ? min(max((x.pos + (1 << a.tlog) + C::TP - 1) / C::TP - x.k0, 0), n) : n;
        edge = min(max((x.pos + 1) / C::TP - x.k0, 0), n);
    }
    DV_DEV int of_stream(int w) const { return pair ? (w ? n : n0) : (n + 1 - w) >> 1; }
};

constexpr float kSeqShift = 6.f;   // the first tile's largest weight is 2^6 to 2^7
constexpr float kSeqLimit = 15.f;  // a weight above 2^15 moves the reference
// Tensor cores cut off what they add instead of rounding it: of the 16 products of a
// step and the sum before them each below 2^-25 of the largest of these, and the new sum
// below 2^-23 of itself (measured, with terms of chosen sizes).  A tile is four steps, so
// outputs could lose 5.25 x 2^-21 of the sum of their terms' sizes a tile.  After this
// many tiles a stream sets its outputs aside, where they are added in binary32: 1.6e-4 at
// most, a third of binary16's half step, and 3.5e-5 in the mean over 262144 positions of one
// sign (256 tiles: 6.4e-4, seen 2.4e-4 beside a term that outweighs the others; 9.5e-5).  It
// costs 4 % of two prompts of 16384 and 7 % of 2048 tokens after 30000, against 256 tiles;
// 48 tiles cost 3 % more, in decode too.
constexpr int kSeqFold = 64;

// Outputs of a row are added to those set aside (`first`: there are none) and start
// from zero again, or, `back`, return with them.  Whole warps.  Not inlined: between
// the tiles' loops its code took 3 % of long prompts' time without ever running.
template <class C>
__device__ __noinline__ void seq_fold(float *rec, int stream, int row, unsigned tO, float m,
                                      bool first, bool back)
{
    constexpr int RM = C::RM, D = C::D;
    float *const acc = rec + 2 * (size_t)kSeqTcCtas * C::REC + (size_t)stream * C::ACC;
    const float was = first ? -INFINITY : ld_cg(acc + RM * D + row);
    const float f = was == -INFINITY ? 0.f : pow2(was - m);
    tc_fence_after();
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
        float y[16];
        unsigned z[16];
        tm_ld16(tO + c, y);
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            float4 *const at = reinterpret_cast<float4 *>(acc) + (c + i) / 4 * RM + row;
            float4 o = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
            if (!first) {
                const float4 g = __ldcg(at);
                o = make_float4(fmaf(g.x, f, o.x), fmaf(g.y, f, o.y), fmaf(g.z, f, o.z),
                                fmaf(g.w, f, o.w));
            }
            if (!back)
                __stcg(at, o);
            z[i] = back ? __float_as_uint(o.x) : 0u;
            z[i + 1] = back ? __float_as_uint(o.y) : 0u;
            z[i + 2] = back ? __float_as_uint(o.z) : 0u;
            z[i + 3] = back ? __float_as_uint(o.w) : 0u;
        }
        tm_st16(tO + c, z);
    }
    if (!back)
        __stcg(acc + RM * D + row, m);
    tm_wait_st();
    tc_fence_before();
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    k_seq_tc(const SeqAttnArgs a, const __grid_constant__ SeqMaps maps, int q_tokens)
{
    constexpr int D = C::D, TP = C::TP, RM = C::RM, NST = C::NST;
    using Sched = typename C::Sched;
    extern __shared__ __align__(1024) unsigned char smem[];
    SeqCtl &ctl = *reinterpret_cast<SeqCtl *>(smem + C::OFF_CTL);
    const unsigned sbase = smem_addr(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (warp == 9) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&ctl.tmem)),
                     "r"(C::T_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (warp == 10 && lane < 3)
        asm volatile("prefetch.tensormap [%0];" ::"l"(lane == 0 ? &maps.q : lane == 1 ? &maps.k : &maps.v)
                     : "memory");
    if (tid == 0) {
        auto init = [](uint64_t &b, int n) { bar_init(smem_addr(&b), n); };
        for (int i = 0; i < NST; ++i) {
            init(ctl.full[i], 1);
            init(ctl.empty[i], 2);
        }
        for (int w = 0; w < 2; ++w) {
            for (int b = 0; b < 2; ++b) {
                init(ctl.s_full[w][b], 1);
                init(ctl.p_full[w][b], 4);
                init(ctl.o_full[w][b], 1);
            }
            init(ctl.q_full[w], 1);
            init(ctl.end[w], 1);
            init(ctl.q_free[w], 1);
        }
        init(ctl.q_both, 2);
        for (int i = 0; i < 8; ++i) {
            init(ctl.v_req[i], 1);
            init(ctl.v_ok[i], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    const SeqRun run0 = Sched::init(a, ctl.sched);  // (barriers)
    if (tid == 0)
        ctl.run = run0;
    __syncthreads();
    const SeqRun &run = ctl.run;
    tc_fence_after();
    const unsigned tmem = ctl.tmem;
    SeqWaiter wait{a.status};
    typename Sched::Piece x = {};

    if (warp == 8) {
        // ---- keys and values
        unsigned i = 0;  // ring entries so far
        // A lane a copy, of the keys or the values: a page's rows of the tile, or of
        // packed rows 64 dimensions (c).
        constexpr int NC = C::PAGED ? 1 : D / 64;
        const int rows = C::PAGED ? min(a.page, TP) : TP, np = TP / rows, piece = lane % np;
        const int c = lane / np % NC, kv = lane / np / NC;
        const CUtensorMap *const map = kv ? &maps.v : &maps.k;
        const unsigned lane_dst = kv * C::TILE + c * C::HALF + piece * (rows * D * 2);
        const int none = C::PAGED ? a.n_pages * a.Hkv : 0;
        // where this lane's page of tile t lies: the page and head in the pool, or
        // one behind the pool, which reads as zeros
        auto page_of = [&](int t) {
            const int p = t * TP + piece * rows;
            if (p >= x.pos + x.ntok)
                return none;
            const int pg = __ldg(a.tables + (long long)x.b * a.width + p / a.page);
            if ((unsigned)pg >= (unsigned)a.n_pages) {
                set_status(a.status, DV_ERR_DEVICE_INDEX);
                return none;
            }
            return pg * a.Hkv + x.hkv;
        };
        typename Sched::Walk walk;
        walk.start(a, run);
        int t = 0, zn = 0, row[3] = {}, z[3] = {};  // of the run's tiles e, e - 1, e - 2
        bool more = true;
        int behind = 0;  // tiles whose values are still to come
#pragma unroll 1
        for (;; ++i) {
            if (more && t >= x.k1) {
                more = walk.next(a, run, x);
                t = x.k0;
                if (more && C::PAGED)
                    zn = page_of(t);
            }
            const bool v = i >= 2 && behind > 0;
            if (!more && behind == 0)
                break;
            row[2] = row[1], row[1] = row[0];
            z[2] = z[1], z[1] = z[0];
            if (more) {
                row[0] = C::PAGED ? (t * TP & (a.page - 1)) >> 3 : x.tok - x.pos + t * TP;
                z[0] = C::PAGED ? zn : x.hkv;
                if (C::PAGED && t + 1 < x.k1)
                    zn = page_of(t + 1);
            }
            const unsigned st = i % NST, full = smem_addr(&ctl.full[st]);
            if (i >= NST)
                wait(&ctl.empty[st], i / NST - 1);
            if (!wait.dead) {
                if (lane == 0)
                    bar_expect(full, ((int)more + v) * C::TILE);
                __syncwarp();
                if (kv == 0 ? more : kv == 1 && v) {
                    const unsigned dst = sbase + C::OFF_KV + st * 2 * C::TILE + lane_dst;
                    const int r = kv ? row[2] : row[0], zz = kv ? z[2] : z[0];
                    if constexpr (C::PAGED)
                        tma_load_page(dst, map, r, zz, full);
                    else
                        tma_load(dst, map, 64 * c, r, zz, full);
                }
            }
            behind += (int)more - v;
            t += more;
        }
        // no copy may outlive the CTA
        for (unsigned k = i < NST ? 0 : i - NST; k < i && !wait.dead; ++k)
            seq_wait(&ctl.full[k % NST], (k / NST) & 1);
        if (wait.dead)
            for (int k = 0; k < NST; ++k) {  // (either phase: what was issued lands in time)
                seq_wait(&ctl.full[k], 0);
                seq_wait(&ctl.full[k], 1);
            }
    } else if (warp == 11) {
        // ---- queries, and value rows that some row does not see
        unsigned u = 0, pairs = 0, singles = 0, base = 0, edges = 0;
        const unsigned bytes = (unsigned)(a.group * q_tokens) * 128 * (D / 64);
        auto queries = [&](const typename Sched::Piece &q, int w) {
            if (lane == 0 && !wait.dead && (w == 0 || q.pair)) {
                const unsigned full = smem_addr(&ctl.q_full[w]);
                bar_expect(full, bytes);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load(sbase + w * C::QTILE + c * C::QHALF, &maps.q, 64 * c, q.h0,
                             q.tok + (w << a.tlog), full);
            }
            __syncwarp();
        };
        typename Sched::Walk walk;
        walk.start(a, run);
        typename Sched::Piece next = {};
        bool more = walk.next(a, run, x);
        if (more) {
            queries(x, 0);
            queries(x, 1);
        }
#pragma unroll 1
        for (; more; x = next) {
            const Plan<C> pl(a, x);
            more = walk.next(a, run, next);
            int loaded = 0;  // queries of the next piece on their way
            // (sent for as soon as the products with this piece's are done, between its
            // edge tiles too)
            auto ahead = [&](bool must) {
#pragma unroll 1
                while (loaded < 2) {
                    uint64_t *const bar = x.pair ? &ctl.q_free[loaded] : &ctl.q_both;
                    const unsigned phase = x.pair ? pairs : singles;
                    if (must)
                        wait(bar, phase);
                    else if (!__all_sync(0xffffffffu, seq_test(bar, phase)))
                        return;
                    if (more)
                        queries(next, loaded);
                    ++loaded;
                }
            };
#pragma unroll 1
            for (int t = pl.edge; t < pl.n; ++t, ++edges) {
                // (asked for when the tile's keys are there: what the ring's stage held
                // before its values has been waited for by then, so a parity tells the
                // phases apart)
                wait(&ctl.v_req[edges & 7], edges >> 3);
                ahead(false);
                const unsigned i = base + t + 2, st = i % NST;
                wait(&ctl.full[st], i / NST);
                unsigned *const bad = ctl.bad[edges & 7];
                if (lane < TP / 32)
                    bad[lane] = 0u;
                __syncwarp();
                // rows up to the first token's position are seen by all
                const int r0 = max(0, x.pos + 1 - (x.k0 + t) * TP);
                const unsigned at = sbase + C::OFF_KV + st * 2 * C::TILE + C::TILE;
#pragma unroll 1
                for (int c = 0; c < D / 64; ++c)
#pragma unroll 4
                    for (int j = r0 * 8 + lane; j < TP * 8; j += 32) {
                        const unsigned p = at + c * C::KHALF + (j >> 6) * C::GROUP + (j & 63) * 16;
                        const uint4 y = lds16(p);
                        // an exponent field of ones carries into its half's top bit
                        unsigned z = ((y.x & 0x7c007c00u) + 0x04000400u) |
                                     ((y.y & 0x7c007c00u) + 0x04000400u) |
                                     ((y.z & 0x7c007c00u) + 0x04000400u) |
                                     ((y.w & 0x7c007c00u) + 0x04000400u);
                        if (z & 0x80008000u) {
                            sts16(p, 0u, 0u, 0u, 0u);
                            atomicOr(bad + (j >> 8), 1u << ((j >> 3) & 31));
                        }
                    }
                fence_async_smem();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(smem_addr(&ctl.v_ok[edges & 7]));
            }
            ahead(true);
            base += pl.n;
            ++u;
            pairs += x.pair;
            singles += !x.pair;
        }
        if (u > 0)
            seq_wait(&ctl.q_full[0], (u - 1) & 1);
        if (pairs > 0)
            seq_wait(&ctl.q_full[1], (pairs - 1) & 1);
    } else if (warp == 9 || warp == 10) {
        // ---- products of stream w.  The warp runs its loop together, so that
        // descriptors stay in uniform registers, and one thread issues.  Both
        // warps follow the whole ring, entry by entry.
        constexpr uint32_t ID_S = tc_idesc(TP, false), ID_O = tc_idesc(D, true);
        constexpr unsigned STAGE = 2 * C::TILE >> 4;
        const int w = warp - 9;
        const uint64_t dk = tc_desc(sbase + C::OFF_KV, 16, C::GROUP),
                       dv = tc_desc(sbase + C::OFF_KV + C::TILE, C::KHALF, C::GROUP);
        const unsigned tS = tmem + C::T_S + w * 128, tO = tmem + C::T_O + w * 128;
        const bool one = elect_one();
        unsigned units = 0, pairs = 0, edges = 0;
        unsigned ns = 0, nv = 0;  // products so far
        unsigned rs = 0, rp = 0;  // the ring's next stage and its phase
        typename Sched::Walk walk;
        walk.start(a, run);
        auto entry = [&]() {  // the next ring entry is there
            wait(&ctl.full[rs], rp);
            const unsigned st = rs;
            if (++rs == NST) {
                rs = 0;
                rp ^= 1;
            }
            return st;
        };
        auto value_product = [&](unsigned st, bool acc) {
            const unsigned b = nv & 1;
            wait(&ctl.p_full[w][b], nv++ >> 1);
            tc_fence_after();
            const uint64_t v = dv + st * STAGE;
            if (one) {
#pragma unroll
                for (int kk = 0; kk < TP / 16; ++kk)
                    tc_mma_ts(tO, tS + b * 64 + kk * 8, v + kk * (2 * C::GROUP >> 4), ID_O, acc || kk > 0);
                tc_commit(&ctl.o_full[w][b]);
            }
        };
        uint64_t dq = 0;
        // (the buffer's weights have been read by then: the value product with them
        // was issued before)
        auto score_product = [&](unsigned st) {
            const unsigned b = ns++ & 1;
            const uint64_t k = dk + st * STAGE;
            if (one) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    tc_mma_ss(tS + b * 64, dq + (kk / 4) * (C::QHALF >> 4) + (kk % 4) * 2,
                              k + (kk / 4) * (C::KHALF >> 4) + (kk % 4) * 2, ID_S, kk > 0);
                tc_commit(&ctl.s_full[w][b]);
            }
        };
        // The piece whose keys come and the one whose values come, two tiles behind:
        // its tiles, those of them that are this stream's, the first with an edge and
        // whether it is a pair.  (Shuffled, so that they are known to be the same in
        // every lane: descriptors are then formed in uniform registers.)
        int4 kp = make_int4(0, 0, 0, 0), vp = kp;
        int tk = 0, tv = 0, behind = 0;
        unsigned vpieces = 0, vedges = 0;  // pieces and edges that the values have come to
        bool more = true;
        // whether a tile is this stream's
        auto uses = [&](const int4 &p, int t) { return p.w ? t < p.y : (t & 1) == w; };
#pragma unroll 1
        for (unsigned e = 0;; ++e) {
            if (more && tk == kp.x) {
                edges += kp.x - kp.z;
                more = walk.next(a, run, x);
                if (more) {
                    const Plan<C> pl(a, x);
                    kp = make_int4(__shfl_sync(0xffffffffu, pl.n, 0),
                                   __shfl_sync(0xffffffffu, pl.of_stream(w), 0),
                                   __shfl_sync(0xffffffffu, pl.edge, 0),
                                   __shfl_sync(0xffffffffu, (int)pl.pair, 0));
                    if (lane == 0)
                        ctl.plan[w][units & 3] = kp;
                    __syncwarp();
                    tk = 0;
                    dq = tc_desc(sbase + (kp.w ? w * C::QTILE : 0), 16, 1024);
                }
            }
            const bool k_on = more, v_on = e >= 2 && behind > 0;
            if (!k_on && behind == 0)
                break;
            if (v_on && tv == vp.x) {  // (its place is written again four pieces on)
                vedges += vp.x - vp.z;
                const int4 p = ctl.plan[w][vpieces++ & 3];
                vp = make_int4(__shfl_sync(0xffffffffu, p.x, 0), __shfl_sync(0xffffffffu, p.y, 0),
                               __shfl_sync(0xffffffffu, p.z, 0), __shfl_sync(0xffffffffu, p.w, 0));
                tv = 0;
            }
            // Most entries of a pair have both products and no edge: nothing else is
            // done there, as every instruction keeps the tensor cores waiting.
            if (k_on && vpieces == units && tk == tv + 2 && tv >= 1 && kp.w) {
                const int plain = min(kp.y - 1, kp.z), from = tk;
#pragma unroll 1
                for (; tk < plain; ++tk) {
                    const unsigned st = entry();
                    value_product(st, true);
                    score_product(st);
                    if (one)
                        tc_commit(&ctl.empty[st]);
                    __syncwarp();
                }
                tv += tk - from;
            }
            const unsigned st = entry();
            tc_fence_after();
            const bool values = v_on && uses(vp, tv), scores = k_on && uses(kp, tk);
            if (one && k_on && tk >= kp.z && (kp.w ? w == 1 : scores))
                bar_arrive(smem_addr(&ctl.v_req[(edges + tk - kp.z) & 7]));
            if (values) {
                if (tv >= vp.z) {
                    const unsigned k = vedges + tv - vp.z;
                    wait(&ctl.v_ok[k & 7], k >> 3);
                }
                value_product(st, tv > (vp.w ? 0 : 1));
            }
            if (k_on && tk == 0) {  // the piece's queries
                wait(&ctl.q_full[0], units++);
                if (kp.w && w)
                    wait(&ctl.q_full[1], pairs);
                pairs += kp.w;
                tc_fence_after();
                if (one && kp.y == 0)  // (no tile of them is this stream's)
                    bar_arrive(smem_addr(kp.w ? &ctl.q_free[w] : &ctl.q_both));
            }
            if (scores)
                score_product(st);
            if (one) {
                if (scores && (kp.w ? tk == kp.y - 1 : tk + 2 >= kp.x))  // its last
                    tc_commit(kp.w ? &ctl.q_free[w] : &ctl.q_both);
                if (scores || values)
                    tc_commit(&ctl.empty[st]);
                else
                    bar_arrive(smem_addr(&ctl.empty[st]));
            }
            __syncwarp();
            behind += (int)k_on - v_on;
            tk += k_on;
            tv += v_on;
        }
        // every product is done before tensor memory goes
        if (one)
            tc_commit(&ctl.end[w]);
        __syncwarp();
        seq_wait(&ctl.end[w], 0);
    } else {
        // ---- softmax of stream w: a thread a row
        const int w = warp >> 2, row = tid & 127, rtok = row / a.group, rhead = row % a.group;
        const unsigned lanes = (unsigned)(32 * (warp & 3)) << 16;
        const unsigned tS = tmem + lanes + C::T_S + w * 128, tO = tmem + lanes + C::T_O + w * 128;
        const float scale = a.scale;
        unsigned tiles = 0, edges = 0;
        typename Sched::Walk walk;
        walk.start(a, run);
        typename Sched::Piece next = {};
        bool more = walk.next(a, run, x);
#pragma unroll 1
        for (; more; x = next) {
            const Plan<C> pl(a, x);
            const int n = pl.of_stream(w);
            const int tok0 = pl.pair && w ? 1 << a.tlog : 0;  // this stream's first token
            const int ntok = pl.pair && !w ? 1 << a.tlog : x.ntok - tok0;
            const bool on = rtok < ntok;
            const bool busy = __any_sync(0xffffffffu, on);  // the warp has a row
            const int lim = x.pos + tok0 + rtok;
            float m = -INFINITY, l = 0.f;
            bool ready = false;  // the next scores are there already
            // One tile: `edged` if some row does not see all of it, or another stream's
            // row does not.
            auto tile = [&](int j, auto edged) {
                constexpr bool EDGE = decltype(edged)::value;
                const unsigned buf = tiles & 1, tP = tS + buf * 64;
                if (!ready)
                    wait(&ctl.s_full[w][buf], tiles >> 1);
                __syncwarp();
                if (busy) {
                    tc_fence_after();
                    const int t = EDGE ? (pl.pair ? j : 2 * j + w) : 0;
                    const int d = EDGE ? lim - (x.k0 + t) * TP : 0;  // the last seen column
                    float v[TP], tops[4];
                    tm_ld(tP, v);
                    tm_ld(tP + 32, v + 32);
                    tm_wait_ld(v);
                    tm_wait_ld(v + 32);
                    if (EDGE) {
#pragma unroll
                        for (int i = 0; i < TP; ++i)
                            v[i] = i <= d ? v[i] : -INFINITY;
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        tops[k] = fmaxf(v[2 * k], v[2 * k + 1]);
#pragma unroll
                    for (int i = 8; i < TP; i += 2)
                        tops[i / 2 % 4] = max3(tops[i / 2 % 4], v[i], v[i + 1]);
                    const float high = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * scale;
                    // From 2^24 on a score rounded (m) and the product in a multiply-add may
                    // be further apart than the weights' range: both are the former then.
                    const bool far = fabsf(high) >= 0x1p24f && high > -INFINITY;
                    const bool need = m == -INFINITY ? high > -INFINITY : high - m > kSeqLimit;
                    float sc = scale;
                    if (__any_sync(0xffffffffu, need || far)) {  // (a row's first tile, or rarely)
                        if (far) {
                            sc = 1.f;
#pragma unroll
                            for (int i = 0; i < TP; ++i)
                                v[i] *= scale;
                        }
                        const float mn = need ? floorf(high) - kSeqShift : m;
                        const float f = need ? pow2(m - mn) : 1.f;
                        m = mn;
                        l *= f;
                        if (j > 0) {
                            // (at rest once the product before is done; this one's is
                            // not issued yet, so a parity tells)
                            wait(&ctl.o_full[w][buf ^ 1], (tiles - 1) >> 1);
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                float y[16];
                                unsigned z[16];
                                tm_ld16(tO + c, y);
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    z[i] = __float_as_uint(y[i] * f);
                                tm_st16(tO + c, z);
                            }
                        }
                    }
                    const float ms = m == -INFINITY ? 0.f : m;
                    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < TP; c += 16) {
                        unsigned pr[8];
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            float p = v[c + i], q = v[c + i + 1];
                            fma2(p, q, sc, -ms);
                            p = ex2(p);
                            q = ex2(q);
                            pr[i / 2] = h2(p, q);
                            add_pair(sum[i & 2], sum[(i & 2) + 1], pr[i / 2]);
                        }
                        tm_st8(tP + c / 2, pr);
                    }
                    ready = seq_test(&ctl.s_full[w][buf ^ 1], (tiles + 1) >> 1);
                    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
                    if (EDGE && t >= pl.edge) {  // a row that sees what was taken out is not finite
                        const unsigned e = edges + t - pl.edge;
                        wait(&ctl.v_ok[e & 7], e >> 3);
                        const unsigned *bad = ctl.bad[e & 7];
#pragma unroll
                        for (int k = 0; k < TP / 32; ++k) {
                            const int s = d - 32 * k;
                            const unsigned seen = s < 0 ? 0u : s >= 31 ? ~0u : (2u << s) - 1;
                            if (bad[k] & seen)
                                l = __int_as_float(0x7fc00000);
                        }
                    }
                    tm_wait_st();
                    tc_fence_before();
                } else {
                    ready = false;
                }
                __syncwarp();
                if (lane == 0)
                    bar_arrive(smem_addr(&ctl.p_full[w][buf]));
                ++tiles;
            };
            // (at rest behind the product before, like a rescaling)
            auto fold = [&](bool first, bool back) {
                wait(&ctl.o_full[w][(tiles - 1) & 1], (tiles - 1) >> 1);
                __syncwarp();
                seq_fold<C>(a.rec, 2 * run.c + w, row, tO, m, first, back);
            };
            // (the first tile with an edge, of this stream's)
            const int plain = min(n, pl.pair ? pl.edge : (pl.edge + 1 - w) >> 1);
            int j = 0;
#pragma unroll 1
            while (j < n) {
                if (j > 0 && busy)
                    fold(j == kSeqFold, false);
                const int stop = min(n, j + kSeqFold), inner = min(plain, stop);
#pragma unroll 1
                for (; j < inner; ++j)
                    tile(j, std::false_type{});
#pragma unroll 1
                for (; j < stop; ++j)
                    tile(j, std::true_type{});
            }
            edges += pl.n - pl.edge;

            // ---- the piece's end; the next one is found while its last product runs
            more = walk.next(a, run, next);
            const bool whole = x.c0 == x.c1;
            const long long off = ((long long)(x.tok + tok0 + rtok) * a.H + x.h0 + rhead) * D;
            float *const rec = a.rec + (size_t)Sched::slot(run.c, x.c0) * C::REC;
            float *const rec_m = rec + 2 * RM * D + w * 2 * RM, *const rec_l = rec_m + RM;
            if (n > 0) {
                wait(&ctl.o_full[w][(tiles - 1) & 1], (tiles - 1) >> 1);
                tc_fence_after();
                if (n > kSeqFold && busy)
                    fold(false, true);
            }
            // Results go to shared memory, laid out as a copy to the output takes them: a
            // thread writing its own row took 7000 cycles a pair.
            const unsigned mine = sbase + C::OFF_OUT + w * C::OUT;
            if (row == 0)  // the copy before has read it
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            // four values of row r's piece, columns 4 c ..
            auto rec_at = [&](float *base, int r, int c) {
                return reinterpret_cast<float4 *>(base) + c * (2 * RM) + r;
            };
            const int r0 = pl.pair ? w * RM : 0;  // the record's rows of this stream
            if (pl.pair && whole) {
                group_sync<128>(2 + w);
                const float f = l == 0.f ? 0.f : __frcp_rn(l);
                if (busy) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 64) {
                        float y[64];
                        tm_ld(tO + c, y);
                        tm_ld(tO + c + 32, y + 32);
                        tm_wait_ld(y);
                        tm_wait_ld(y + 32);
#pragma unroll
                        for (int i = 0; i < 64; i += 8) {
#pragma unroll
                            for (int k = 0; k < 8; k += 2)
                                mul2(y[i + k], y[i + k + 1], f, f);
                            sts16(mine + (c >> 6) * C::QHALF + row * 128 + (((i >> 3) ^ (row & 7)) << 4),
                                  h2(y[i], y[i + 1]), h2(y[i + 2], y[i + 3]), h2(y[i + 4], y[i + 5]),
                                  h2(y[i + 6], y[i + 7]));
                        }
                    }
                    tc_fence_before();
                }
                if (ntok == 1 << a.tlog) {  // all of the tile's tokens: by a copy
                    fence_async_smem();
                    group_sync<128>(2 + w);
                    if (row == 0) {
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_store(&maps.out, 64 * c, x.h0, x.tok + tok0, mine + c * C::QHALF);
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                } else {  // a warp its rows, in whole lines
                    __syncwarp();
                    const unsigned rows_on = __ballot_sync(0xffffffffu, on);
#pragma unroll 1
                    for (int i = lane; i < 32 * (D / 8); i += 32) {
                        const int r = i / (D / 8), ch = i % (D / 8), at = row - lane + r;
                        const long long to = __shfl_sync(0xffffffffu, off, r);
                        const uint4 u = lds16(mine + (ch >> 3) * C::QHALF + at * 128 +
                                              (((ch ^ at) & 7) << 4));
                        if ((rows_on >> r) & 1)
                            *reinterpret_cast<uint4 *>(static_cast<__half *>(a.out) + to + 8 * ch) = u;
                    }
                }
            } else if (pl.pair) {
                if (busy && n > 0) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        float y[16];
                        tm_ld16(tO + c, y);
                        if (on) {
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                __stcg(rec_at(rec, r0 + row, (c + i) / 4),
                                       make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]));
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before();
            } else {
                // Stream w finishes columns w D / 2 .. of all rows; the other
                // stream's share of them comes through the results' place.
                constexpr int HC = D / 2;
                group_sync<256>(1);  // (both have left the unit before, too)
                ctl.m[w][row] = m;
                ctl.l[w][row] = l;
                float4 *const give = reinterpret_cast<float4 *>(smem + C::OFF_OUT + (w ^ 1) * C::OUT) + row;
                const float4 *const get = reinterpret_cast<float4 *>(smem + C::OFF_OUT + w * C::OUT) + row;
                if (busy && n > 0) {
#pragma unroll 1
                    for (int c = 0; c < HC; c += 16) {
                        float y[16];
                        tm_ld16(tO + (w ^ 1) * HC + c, y);
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            give[(c + i) / 4 * C::XROWS] = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
                    }
                }
                group_sync<256>(1);
                if (busy) {
                    const float mo = ctl.m[w ^ 1][row], M = fmaxf(m, mo);
                    const float ms = M == -INFINITY ? 0.f : M;
                    const float fw = pow2(m - ms), fo = pow2(mo - ms);
                    const bool other = pl.of_stream(w ^ 1) > 0;
                    l = l * fw + ctl.l[w ^ 1][row] * fo;
                    m = M;
                    const float f = l == 0.f ? 0.f : __frcp_rn(l);
#pragma unroll 1
                    for (int c = 0; c < HC; c += 16) {
                        float y[16];
                        if (n > 0)
                            tm_ld16(tO + w * HC + c, y);
#pragma unroll
                        for (int i = 0; i < 16; i += 4) {
                            float4 g = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (other)
                                g = get[(c + i) / 4 * C::XROWS];
                            y[i] = n > 0 ? fmaf(y[i], fw, g.x * fo) : g.x * fo;
                            y[i + 1] = n > 0 ? fmaf(y[i + 1], fw, g.y * fo) : g.y * fo;
                            y[i + 2] = n > 0 ? fmaf(y[i + 2], fw, g.z * fo) : g.z * fo;
                            y[i + 3] = n > 0 ? fmaf(y[i + 3], fw, g.w * fo) : g.w * fo;
                        }
                        if (on && whole) {
#pragma unroll
                            for (int i = 0; i < 16; i += 8)
                                *reinterpret_cast<uint4 *>(static_cast<__half *>(a.out) + off + w * HC +
                                                           c + i) =
                                    make_uint4(h2(y[i] * f, y[i + 1] * f),
                                               h2(y[i + 2] * f, y[i + 3] * f),
                                               h2(y[i + 4] * f, y[i + 5] * f),
                                               h2(y[i + 6] * f, y[i + 7] * f));
                        } else if (on) {
#pragma unroll
                            for (int i = 0; i < 16; i += 4)
                                __stcg(rec_at(rec, row, (w * HC + c + i) / 4),
                                       make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]));
                        }
                        __syncwarp();
                    }
                    tc_fence_before();
                }
            }
            if (whole)
                continue;
            if (on) {
                // (a stream without a tile of this piece has left no outputs)
                __stcg(rec_m + row, m);
                __stcg(rec_l + row, l);
            }
            __threadfence();
            group_sync<128>(2 + w);
            if (row == 0) {
                int *cnt = a.cnt + 2 * x.c0 + w;
                const int was = atomicAdd(cnt, 1);
                ctl.last[w] = was == x.c1 - x.c0;
                if (ctl.last[w])
                    *cnt = 0;
                __threadfence();
            }
            group_sync<128>(2 + w);
            if (!ctl.last[w])
                continue;
            // ---- merge: the rows (a power of two of them) x groups of columns over the
            // stream's threads, eight float4 of every piece on their way at once
            const int rows = min(ntok * a.group, RM), rlog = rows > 1 ? 32 - __clz(rows - 1) : 0;
            const int r = row & ((1 << rlog) - 1), cg = pl.pair ? D / 4 : D / 8;
            const int per = max(1, cg >> (7 - rlog)), c0 = (row >> rlog) * per;
            if (r < rows && c0 < cg) {
                auto rec_of = [&](int p) { return a.rec + (size_t)Sched::slot(p, x.c0) * C::REC; };
                const int at_m = 2 * RM * D + w * 2 * RM + r;
                float M = -INFINITY, L = 0.f;
#pragma unroll 4
                for (int p = x.c0; p <= x.c1; ++p)
                    M = fmaxf(M, ld_cg(rec_of(p) + at_m));
                const float ms = M == -INFINITY ? 0.f : M;
#pragma unroll 4
                for (int p = x.c0; p <= x.c1; ++p)
                    L = fmaf(ld_cg(rec_of(p) + at_m + RM), pow2(ld_cg(rec_of(p) + at_m) - ms), L);
                const float f = L == 0.f ? 0.f : __frcp_rn(L);
                __half *const to = static_cast<__half *>(a.out) +
                                   ((long long)(x.tok + tok0 + r / a.group) * a.H + x.h0 + r % a.group) * D;
                const int first = (pl.pair ? 0 : w * (D / 8)) + c0;
#pragma unroll 1
                for (int i0 = 0; i0 < per; i0 += 8) {
                    float4 o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                    for (int p = x.c0; p <= x.c1; ++p) {
                        const float mp = ld_cg(rec_of(p) + at_m), g = pow2(mp - ms);
                        if (mp == -INFINITY)  // (a stream without a tile of the piece left none)
                            continue;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (i < per) {
                                const float4 y = __ldcg(rec_at(rec_of(p), r0 + r, first + i0 + i));
                                o[i].x = fmaf(y.x, g, o[i].x);
                                o[i].y = fmaf(y.y, g, o[i].y);
                                o[i].z = fmaf(y.z, g, o[i].z);
                                o[i].w = fmaf(y.w, g, o[i].w);
                            }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (i < per)
                            *reinterpret_cast<uint2 *>(to + 4 * (first + i0 + i)) =
                                make_uint2(h2(o[i].x * f, o[i].y * f), h2(o[i].z * f, o[i].w * f));
                }
            }
        }
        if (row == 0)
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(C::T_COLS)
                     : "memory");
    }
}

// Tensor maps of binary16 rows, encoded by the driver's function (resolved
// through the runtime: the library does not link the driver library).
struct SeqMapEncoder {
    PFN_cuTensorMapEncodeTiled_v12000 encode;
    SeqMapEncoder()
    {
        static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
            void *f = nullptr;
            cudaDriverEntryPointQueryResult q;
            const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                             cudaEnableDefault, &q) == cudaSuccess &&
                            q == cudaDriverEntryPointSuccess;
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ok ? f : nullptr);
        }();
        encode = fn;
    }
    // N dimensions, the strides of all but the first in elements; swizzled rows of
    // 128 bytes.
    template <int N>
    cudaError_t operator()(CUtensorMap *m, const void *p, const unsigned (&dims)[N],
                           const long long (&strides)[N - 1], const unsigned (&box)[N]) const
    {
        if (!encode)
            return cudaErrorNotSupported;
        cuuint64_t d[N], s[N - 1];
        cuuint32_t b[N], one[N];
        for (int i = 0; i < N; ++i) {
            d[i] = dims[i];
            b[i] = box[i];
            one[i] = 1;
            if (i)
                s[i - 1] = (cuuint64_t)strides[i - 1] * 2;
        }
        return encode(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, N, const_cast<void *>(p), d, s, b, one,
                      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                      CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
                   ? cudaSuccess
                   : cudaErrorInvalidValue;
    }
};

template <class C>
cudaError_t launch_tc(const SeqAttnArgs &a, int nsm, cudaStream_t st)
{
    auto kern = k_seq_tc<C>;
    constexpr size_t smem = C::OFF_CTL + sizeof(SeqCtl);
    static_assert(smem <= 227 * 1024 && C::NST <= 8, "shared memory of a CTA; see SeqCtl");
    static DeviceOnce once;
    cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
    if (e != cudaSuccess)
        return e;
    int q_tokens = 1;  // of a copy: no more than a request can have
    while (q_tokens < a.max_tok && q_tokens < 1 << a.tlog)
        q_tokens *= 2;
    const SeqMapEncoder enc;
    SeqMaps maps;
    constexpr unsigned D = C::D;
    // queries (dimension, head, token), boxes of a unit's heads and tokens
    if ((e = enc.template operator()<3>(
             &maps.q, a.q.p, {D, (unsigned)a.H, (unsigned)a.T},
                 {a.H > 1 ? a.q.sh : D, a.T > 1 ? a.q.st : D},
                 {64, (unsigned)a.group, (unsigned)q_tokens})))
        return e;
    // results, a unit's 128 rows
    if ((e = enc.template operator()<3>(
             &maps.out, a.out, {D, (unsigned)a.H, (unsigned)a.T}, {D, (long long)D * a.H},
                 {64, (unsigned)a.group, 1u << a.tlog})))
        return e;
    for (int i = 0; i < 2; ++i) {
        CUtensorMap *m = i ? &maps.v : &maps.k;
        const SeqRowsArgs &r = i ? a.v : a.k;
        const unsigned groups = (unsigned)a.page / 8;
        if (C::PAGED)  // (dimension, row of 8, half, group of 8 rows, page and head)
            e = enc.template operator()<5>(
                m, i ? a.pv : a.pk, {64, 8, D / 64, groups, (unsigned)(a.n_pages * a.Hkv)},
                {D, 64, 8 * D, (long long)D * a.page}, {64, 8, D / 64, groups < 8 ? groups : 8, 1});
        else  // (dimension, token, head)
            e = enc.template operator()<3>(m, r.p, {D, (unsigned)a.T, (unsigned)a.Hkv},
                                           {a.T > 1 ? r.st : D, a.Hkv > 1 ? r.sh : D},
                                           {64, C::TP, 1});
        if (e)
            return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nsm < kSeqTcCtas ? nsm : kSeqTcCtas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, a, maps, q_tokens);
}

}  // namespace

cudaError_t launch_seq_tc(const SeqAttnArgs &a, int nsm, cudaStream_t st)
{
    SeqAttnArgs b = a;
    seq_group(b, 128);
    const bool few = b.max_tok <= 1 << b.tlog && (long long)b.max_tok * b.group <= 32;
    const auto go = [&](auto d) {
        constexpr int D = decltype(d)::value;
        return !a.pk ? launch_tc<SeqTcCfg<D, false, false>>(b, nsm, st)
               : few ? launch_tc<SeqTcCfg<D, true, true>>(b, nsm, st)
                     : launch_tc<SeqTcCfg<D, true, false>>(b, nsm, st);
    };
    return a.D == 128 ? go(std::integral_constant<int, 128>{}) : go(std::integral_constant<int, 64>{});
}

size_t seq_tc_record_bytes(int D)
{
    // two pieces' records a CTA, and what its streams set aside
    return 2 * (size_t)kSeqTcCtas * (2 * 128 * D + 4 * 128 + 128 * D + 128) * 4;
}

}  // namespace dv
