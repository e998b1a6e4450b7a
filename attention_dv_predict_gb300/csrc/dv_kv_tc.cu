// dv_kv_tc.cu -- attention of 9 to 64 query rows per KV head (drafted trees,
// grouped query heads) over a binary16 or 8-bit cache on tcgen05 (sm_103a).
//
// A unit's 64 query rows fill an M = 128 tile with their binary16 high and
// low parts: TMEM lanes 32 w .. 32 w + 15 hold the high parts of rows 16 w ..
// 16 w + 15, the next 16 lanes their low parts, so the sum of the two lane
// halves has 22 of the query's bits, and the weights, split the same way, give
// the value product the same accuracy.  Both products of a 64-position tile of
// 128 dimensions take 619 tensor cycles (measured alone: 384 and 256), mma.sync
// 2048.  64-token trees of 32 rows at the 175B shape, 2048 cached positions:
// binary16 573 us, where the cache's bytes alone take 519; 8 bits 675 us,
// where those take 282 and the tensor products 220.  No unit is full there (0.60
// of the issue slots, 0.32 of the DRAM throughput, 0.30 of the tensor pipe): the
// 16 softmax and 8 conversion warps wait for loads of tensor memory and for one
// another's hand-overs.  Their 72 registers a thread spill 64 bytes of stores.
//
// Warps of a CTA (one CTA per SM):
//   0-15      softmax: two streams that take turns at the tiles, each with its
//             own output columns in tensor memory; they are merged when a unit
//             ends, so neither waits for the other.  Eight warps of a stream
//             take half of a tile's columns each four: a warp's own latency
//             bounds it.  Four score buffers, whose weights take the scores'
//             place, let scores run ahead
//   16-23     8-bit caches: codes to binary16, raw ring -> operand ring
//   last four one that prepares a unit's queries while the unit before runs,
//             one of tensor-map copies (and scales by cp.async), one whose
//             elected thread issues the scores' MMAs, one the values'
// Keys are the K-major operand of the scores; values, as they lie, the
// MN-major operand of Q = softmax weights (A from tensor memory) x V.
// Hand-overs are mbarriers; every wait has a limit (DV_ERR_TIMEOUT).
//
// A row's reference point only moves when a weight of its own leaves binary16's
// range (dv_kv_tma.cuh), so the output in tensor memory is rarely rescaled and a
// tile's softmax needs no reduction over the row.  Scores that rise steadily
// move their rows one after another: 64 tokens of 8 x 96 heads over 2048 8-bit
// positions take 198 us, 252 where the scores rise by 15 and 329 where by 60
// (binary16: 179, 195, 225).  Taking rows that are halfway to the range's end
// every fourth tile made that 240 and 310, but the 675 us above 760.
#include "dv_kv_tma.cuh"

namespace dv {
namespace {

template <bool I8_, int D_, bool LONG_>
struct TcCfg {
    static constexpr bool I8 = I8_, LONG = LONG_;
    static constexpr int D = D_, RM = 64, TP = kKvTile;
    static constexpr int RB = D * (I8 ? 1 : 2);           // bytes of a cached row
    static constexpr int OPER = TP * D * 2;               // a binary16 operand tile
    static constexpr int NK = I8 ? 2 : (D == 128 ? 4 : 8);  // key operands
    static constexpr int NV = NK + 1;                     // value operands: held longer
    static constexpr int RAW = TP * RB;
    static constexpr int NSR = I8 ? (D == 128 ? 4 : 8) : 0;  // raw stages
    static constexpr int NSC = D == 128 ? 8 : 16;         // scale slots (see the producer)
    static constexpr int QB = 128 * D * 2;
    static constexpr int WARPS = 16 + (I8 ? 8 : 0) + 4, THREADS = 32 * WARPS;
    static constexpr int SOFT = 512;                      // softmax threads
    static constexpr int OFF_OP = 2 * QB;
    static constexpr int OFF_V = OFF_OP + NK * OPER;
    static constexpr int OFF_RAW = OFF_V + NV * OPER;
    static constexpr int OFF_SC = OFF_RAW + NSR * 2 * RAW;
    static_assert(kMergePieces * RM * 4 <= 2 * QB, "the merge's weights fit them");
    static constexpr size_t SMEM = 1024 + OFF_SC + (I8 ? NSC * 2 * TP * 4 : 0);
    // tensor-memory columns
    static constexpr int NS = 4, T_S = 0, T_O = 64 * NS, T_COLS = 512;
    static_assert(TP == 64 && T_O + 2 * 128 <= T_COLS, "score buffers, two outputs");
    // Tiles of a unit whose values tensor memory sums.  The tensor cores cut
    // sums off instead of rounding them, always towards zero: without a limit
    // the outputs of a part of 250 tiles were 6.5e-6 too small, now 2.2e-6 (128
    // steps; terms of chosen sizes show that each cuts 16 products and the sum
    // before off below 2^-25 of the largest, and the new sum below 2^-23: 6e-5
    // beside one term that outweighs the others, 8e-5 at most).
    static constexpr int CHUNK = 64;
};

struct SoftSync {
    DV_DEV static void sync() { asm volatile("bar.sync 1, 512;" ::: "memory"); }
};

DV_DEV void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
DV_DEV void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
DV_DEV void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle: 8-row groups 1024 bytes
// apart; lbo: bytes between 64-element blocks of an MN-major operand.
DV_DEV uint64_t tc_desc(unsigned saddr, unsigned lbo)
{
    return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
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
DV_DEV void tc_commit(unsigned bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}

// 16 lanes x 2 N columns: thread (g, t) = (lane / 4, lane % 4) holds columns 8 j
// + 2 t, + 1 of lanes g (v[4 j], v[4 j + 1]) and g + 8 (v[4 j + 2], v[4 j + 3]).
template <int N>
DV_DEV void tm_ld(unsigned addr, float (&v)[N])
{
    static_assert(N == 16 || N == 8, "32 or 16 columns");
    if constexpr (N == 16)
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
                     : "r"(addr));
    else
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "r"(addr));
}
template <int N>
DV_DEV void tm_st(unsigned addr, const float (&v)[N])
{
    static_assert(N == 16 || N == 8, "32 or 16 columns");
    if constexpr (N == 16)
        asm volatile("tcgen05.st.sync.aligned.16x256b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
                     "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
                     : "memory");
    else
        asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr),
                     "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                     : "memory");
}
// The loads into v have landed (v passes through, so that no use moves before it).
template <int N>
DV_DEV void tm_wait_ld(float (&v)[N])
{
    static_assert(N == 16 || N == 8, "32 or 16 columns");
    if constexpr (N == 16)
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
                     :
                     : "memory");
    else
        asm volatile("tcgen05.wait::ld.sync.aligned;"
                     : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7])
                     :
                     : "memory");
}
DV_DEV void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 16 lanes x 16 columns of binary16 pairs: r[2 j] columns 4 j + t of lane g,
// r[2 j + 1] of lane g + 8.
DV_DEV void tm_st_pairs(unsigned addr, const unsigned (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(
                     addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                 "r"(r[7])
                 : "memory");
}

// Whether any of N threads says so (a barrier among them).
template <int N>
DV_DEV bool any_of(int bar, bool v)
{
    unsigned r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((unsigned)v), "r"(bar), "n"(N)
        : "memory");
    return r != 0;
}
DV_DEV bool stream_any(int stream, bool v) { return any_of<256>(2 + stream, v); }

DV_DEV bool elect_one()
{
    unsigned p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(p));
    return p != 0;
}

// A role's waits: after one has run out the others no longer wait (the
// results are lost, the status says so, every loop still ends).
struct Waiter {
    int *status;
    bool dead = false;
    DV_DEV void operator()(unsigned bar, unsigned parity)
    {
        if (!dead && !bar_wait(bar, parity)) {
            dead = true;
            set_status(status, DV_ERR_TIMEOUT);
        }
    }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    k_kv_tc(const KvAttnArgs a, const __grid_constant__ KvMaps maps)
{
    constexpr int D = C::D, RM = C::RM, TP = C::TP, NK = C::NK, NV = C::NV;
    constexpr bool I8 = C::I8;
    extern __shared__ unsigned char smem_raw[];
    __shared__ SchedSmem sm;
    __shared__ float s_m[2][RM], s_l[4][RM], u_m[RM], u_l[RM];
    __shared__ float c_m[2][RM], c_l[2][RM];  // of a part's chunks so far
    // what the query warp prepares, for two units: beside the operand
    __shared__ float s_inv[2][RM];
    __shared__ unsigned long long s_bits[2][RM];
    __shared__ Unit s_unit[2];
    __shared__ int s_tile0[2], s_n[2];  // first tile; tiles (0: the run is over)
    __shared__ int s_ends[2];           // bit 0: the part's first chunk, bit 1: its last
    __shared__ float s_max[2][2][RM];  // rare: a row's maximum over both halves,
    __shared__ bool s_out[2][2][RM];   // and whether a weight of it is out of range
    __shared__ unsigned s_bad[2][2];  // binary16 edge tiles: positions not finite
    __shared__ __align__(8) uint64_t b_raw_full[I8 ? C::NSR : 1], b_raw_empty[I8 ? C::NSR : 1],
        b_sc_full[C::NSC], b_k_full[NK], b_k_empty[NK], b_v_full[NV], b_v_empty[NV], b_s_full[C::NS],
        b_p_full[C::NS], b_s_free[C::NS], b_q_full[2], b_q_free[2], b_end[2];
    __shared__ unsigned s_tmem;
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const unsigned sbase = smem_addr(smem);
    float *scales = reinterpret_cast<float *>(smem + C::OFF_SC);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int W_PV = C::WARPS - 1, W_QK = C::WARPS - 2, W_LOAD = C::WARPS - 3,
                  W_Q = C::WARPS - 4;

    if (warp == W_PV) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&s_tmem)),
                     "r"(C::T_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < C::NSR; ++i) {
            bar_init(smem_addr(&b_raw_full[i]), 1);
            bar_init(smem_addr(&b_raw_empty[i]), 8);
        }
        for (int i = 0; i < C::NSC; ++i)
            bar_init(smem_addr(&b_sc_full[i]), 32);
        for (int i = 0; i < NV; ++i) {
            if (i < NK) {
                bar_init(smem_addr(&b_k_full[i]), I8 ? 4 : 1);
                bar_init(smem_addr(&b_k_empty[i]), 1);
            }
            bar_init(smem_addr(&b_v_full[i]), I8 ? 4 : 1);
            bar_init(smem_addr(&b_v_empty[i]), 1);
        }
        for (int i = 0; i < C::NS; ++i) {
            bar_init(smem_addr(&b_s_full[i]), 1);
            bar_init(smem_addr(&b_p_full[i]), 8);
            bar_init(smem_addr(&b_s_free[i]), 1);
            if (i < 2) {
                bar_init(smem_addr(&b_q_full[i]), 1);
                bar_init(smem_addr(&b_q_free[i]), 16);
            }
        }
        bar_init(smem_addr(&b_end[0]), 1);
        bar_init(smem_addr(&b_end[1]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    const Run run = sched_init<false>(a, RM, sm);  // (barriers)
    tc_fence_after();
    const unsigned tmem = s_tmem;
    Waiter wait{a.status};

    if (warp == W_LOAD) {
        // ---- copies.  A scale slot is reused 8 tiles later: by then the raw
        // (NSR) and value (NV) rings between have only let the copies this far
        // because the slot's tile has left the softmax.
        static_assert(!I8 || C::NSR + NV <= C::NSC, "scale slots");
        int i = 0;  // tile of the run
        auto boxes = [&](unsigned dst, const CUtensorMap *map, int p, int bh, unsigned bar) {
#pragma unroll
            for (int xb = 0; xb < C::RB; xb += 128)
                tma_load(dst + xb * TP, map, xb, p, bh, bar);
        };
        for (long long w = run.lo; w < run.hi;) {
            const Unit x = sched_unit<false>(a, RM, sm, run, w);
            const long long wend = min(run.hi, x.w1);
            if (x.h < 0) {
                w = wend;
                continue;
            }
            const int bh = unit_bh<false>(a, x);
            for (w = tile_place(x, w); w < wend; ++w, ++i) {
                const int p = tile_of(x, w) * TP;
                if constexpr (I8) {
                    const int slot = i % C::NSR, sc = i % C::NSC;
                    if (i >= C::NSR)
                        wait(smem_addr(&b_raw_empty[slot]), (i / C::NSR - 1) & 1);
                    const unsigned dst = sbase + C::OFF_SC + sc * 2 * TP * 4;
#pragma unroll
                    for (int k = 0; k < 2 * TP; k += 32) {
                        const int r = (k + lane) % TP;
                        const bool on = p + r < a.c.cap;
                        cp4(dst + (k + lane) * 4,
                            (k < TP ? a.c.ks : a.c.vs) + (on ? (size_t)bh * a.c.cap + p + r : 0), on);
                    }
                    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(
                                     smem_addr(&b_sc_full[sc]))
                                 : "memory");
                    if (lane == 0) {
                        const unsigned full = smem_addr(&b_raw_full[slot]);
                        const unsigned raw = sbase + C::OFF_RAW + slot * 2 * C::RAW;
                        bar_expect(full, 2 * C::RAW);
                        boxes(raw, &maps.k, p, bh, full);
                        boxes(raw + C::RAW, &maps.v, p, bh, full);
                    }
                } else {
                    const int sk = i % NK, sv = i % NV;
                    if (i >= NK)
                        wait(smem_addr(&b_k_empty[sk]), (i / NK - 1) & 1);
                    if (lane == 0) {
                        const unsigned full = smem_addr(&b_k_full[sk]);
                        bar_expect(full, C::OPER);
                        boxes(sbase + C::OFF_OP + sk * C::OPER, &maps.k, p, bh, full);
                    }
                    __syncwarp();
                    if (i >= NV)
                        wait(smem_addr(&b_v_empty[sv]), (i / NV - 1) & 1);
                    if (lane == 0) {
                        const unsigned full = smem_addr(&b_v_full[sv]);
                        bar_expect(full, C::OPER);
                        boxes(sbase + C::OFF_V + sv * C::OPER, &maps.v, p, bh, full);
                    }
                }
                __syncwarp();
            }
        }
        // no copy may outlive the CTA
        if constexpr (I8) {
            asm volatile("cp.async.wait_all;" ::: "memory");
            for (int k = max(0, i - C::NSR); k < i; ++k)
                bar_wait(smem_addr(&b_raw_full[k % C::NSR]), (k / C::NSR) & 1);
        } else {
            for (int k = max(0, i - NK); k < i; ++k)
                bar_wait(smem_addr(&b_k_full[k % NK]), (k / NK) & 1);
            for (int k = max(0, i - NV); k < i; ++k)
                bar_wait(smem_addr(&b_v_full[k % NV]), (k / NV) & 1);
        }
    } else if (warp == W_Q) {
        // ---- queries: each unit's, split and in place, a unit ahead
        int k = 0;
        auto take = [&](int buf) {  // buffer `buf` is free (unit k - 2 has left it)
            if (k >= 2)
                wait(smem_addr(&b_q_free[buf]), (k / 2 - 1) & 1);
        };
        for (long long w = run.lo; w < run.hi;) {
            const Unit x = sched_unit<false>(a, RM, sm, run, w);
            const long long wpart = min(run.hi, x.w1), wb = tile_place(x, w);
            const bool first = !C::LONG || w == run.lo || w == x.w0;
            if (x.h < 0) {
                w = wpart;
                continue;
            }
            // a long part is handed out in chunks of like size
            const int rest = (int)(wpart - wb);
            const long long wend =
                C::LONG ? wb + rest / ((rest + C::CHUNK - 1) / C::CHUNK) : wpart;
            w = wend;
            const int buf = k & 1;
            if (first) {  // on their way to L2 while the buffer is waited for
                const int es = a.q.f16 ? 2 : 4;
                for (int r = lane; r < x.nrows; r += 32) {
                    const char *q = static_cast<const char *>(a.q.p) + es * q_at<false>(a, x, r);
                    for (int d = 0; d < D * es; d += 128)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(q + d));
                }
            }
            take(buf);
            if (lane == 0) {
                s_unit[buf] = x;
                s_tile0[buf] = tile_of(x, wb);
                s_n[buf] = (int)(wend - wb);
                s_ends[buf] = first | (wend == wpart) << 1;
            }
            unsigned char *qs = smem + buf * C::QB;
            if (!first) {  // the chunk before has them (and the softmax waits for this copy)
                constexpr int N = 4;
                const uint4 *from = reinterpret_cast<const uint4 *>(smem + (buf ^ 1) * C::QB) + lane;
                uint4 *to = reinterpret_cast<uint4 *>(qs) + lane;
#pragma unroll 1
                for (int i = 0; i < C::QB / 16; i += 32 * N) {
                    uint4 u[N];
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        u[j] = from[i + 32 * j];
#pragma unroll
                    for (int j = 0; j < N; ++j)
                        to[i + 32 * j] = u[j];
                }
                for (int r = lane; r < RM; r += 32) {
                    s_inv[buf][r] = s_inv[buf ^ 1][r];
                    s_bits[buf][r] = s_bits[buf ^ 1][r];
                }
            } else {
                // a row over D / 16 lanes, the next pass's rows on their way
                constexpr int LPR = D / 16, RPP = 32 / LPR;
                const int part = lane % LPR;
                float4 v[4], nx[4];
                auto fetch = [&](int r0, float4 (&to)[4]) {
                    const int r = r0 + lane / LPR;
                    long long at[4];
                    const long long q0 = r < x.nrows ? q_at<false>(a, x, r) + part * 16 : -1;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        at[i] = q0 < 0 ? -1 : q0 + 4 * i;
                    ld_queries(a.q, at, to);
                };
                fetch(0, nx);
#pragma unroll 1
                for (int r0 = 0; r0 < RM; r0 += RPP) {
                    const int r = r0 + lane / LPR;
                    float mx = 0.f;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        v[i] = nx[i];
                        mul2(v[i].x, v[i].y, a.scale, a.scale);
                        mul2(v[i].z, v[i].w, a.scale, a.scale);
                        mx = amax3(amax3(mx, v[i].x, v[i].y), v[i].z, v[i].w);
                    }
                    if (r0 + RPP < RM)
                        fetch(r0 + RPP, nx);
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1)
                        mx = amax2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    float inv;
                    const float al = query_power(mx, &inv);
                    unsigned hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        mul2(v[i].x, v[i].y, al, al);
                        mul2(v[i].z, v[i].w, al, al);
                        hi[2 * i] = h2(v[i].x, v[i].y);
                        hi[2 * i + 1] = h2(v[i].z, v[i].w);
                        lo[2 * i] = h2_rest(v[i].x, v[i].y, hi[2 * i]);
                        lo[2 * i + 1] = h2_rest(v[i].z, v[i].w, hi[2 * i + 1]);
                    }
                    // 64 dimensions a region of 128 rows; a row's low parts 16 rows on, at
                    // the same place in the swizzle
                    const int row = 32 * (r >> 4) + (r & 15), c = 2 * (part & 3);
                    unsigned char *p = qs + (part >> 2) * (128 * 128) + row * 128;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        unsigned char *q = p + (((c + k) ^ (row & 7)) << 4);
                        *reinterpret_cast<uint4 *>(q) =
                            make_uint4(hi[4 * k], hi[4 * k + 1], hi[4 * k + 2], hi[4 * k + 3]);
                        *reinterpret_cast<uint4 *>(q + 16 * 128) =
                            make_uint4(lo[4 * k], lo[4 * k + 1], lo[4 * k + 2], lo[4 * k + 3]);
                    }
                    if (part == 0)
                        s_inv[buf][r] = inv;
                }
                for (int r = lane; r < RM; r += 32)
                    s_bits[buf][r] =
                        r < x.nrows ? seen_bits(a, x, row_token(a, x.row0 + r)) : 0ull;
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0)
                bar_arrive(smem_addr(&b_q_full[buf]));
            ++k;
        }
        take(k & 1);
        if (lane == 0) {
            s_n[k & 1] = 0;
            bar_arrive(smem_addr(&b_q_full[k & 1]));
        }
    } else if (warp == W_QK || warp == W_PV) {
        // ---- products, the scores' and the values' each by a warp.  The warp
        // runs its loop together, so that descriptors stay in uniform
        // registers, and one thread issues (with the loop in one thread,
        // building them took longer than the products).
        constexpr uint32_t ID_S = tc_idesc(TP, false), ID_O = tc_idesc(D, true);
        constexpr unsigned STAGE = C::OPER >> 4;
        const uint64_t dq = tc_desc(sbase, 16), dk0 = tc_desc(sbase + C::OFF_OP, 16),
                       dv0 = tc_desc(sbase + C::OFF_V, TP * 128);
        const bool one = elect_one(), scores = warp == W_QK;
        int st = 0, stp = 0, sb = 0, sbp = 0;  // operand stage, score buffer; their phases
        bool used = false;                     // every score buffer has been used
        for (int k = 0;; ++k) {
            wait(smem_addr(&b_q_full[k & 1]), (k >> 1) & 1);
            const int n = wait.dead ? 0 : __shfl_sync(0xffffffffu, s_n[k & 1], 0);
            if (n == 0)
                break;
            if (scores) {
                const uint64_t da = dq + (uint64_t)(unsigned)(k & 1) * (C::QB >> 4);
                for (int t = 0; t < n; ++t) {
                    if (used)  // the weights that took the buffer's scores' place are read
                        wait(smem_addr(&b_s_free[sb]), sbp ^ 1);
                    wait(smem_addr(&b_k_full[st]), stp);
                    tc_fence_after();
                    const uint64_t dk = dk0 + (uint64_t)(unsigned)st * STAGE;
                    if (one) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc_mma_ss(tmem + C::T_S + sb * 64,
                                      da + (kk / 4) * (128 * 128 >> 4) + (kk % 4) * 2,
                                      dk + (kk / 4) * (TP * 128 >> 4) + (kk % 4) * 2, ID_S, kk > 0);
                        tc_commit(smem_addr(&b_s_full[sb]));
                        tc_commit(smem_addr(&b_k_empty[st]));
                    }
                    __syncwarp();
                    if (++sb == C::NS) {
                        sb = 0;
                        sbp ^= 1;
                        used = true;
                    }
                    if (++st == NK) {
                        st = 0;
                        stp ^= 1;
                    }
                }
            } else {
                for (int t = 0; t < n; ++t) {
                    const int g = t & 1;
                    wait(smem_addr(&b_v_full[st]), stp);
                    wait(smem_addr(&b_p_full[sb]), sbp);
                    tc_fence_after();
                    const uint64_t dv = dv0 + (uint64_t)(unsigned)st * STAGE;
                    if (one) {
#pragma unroll
                        for (int kk = 0; kk < TP / 16; ++kk)
                            tc_mma_ts(tmem + C::T_O + g * 128, tmem + C::T_S + sb * 64 + kk * 8,
                                      dv + kk * (16 * 128 >> 4), ID_O, t > 1 || kk > 0);
                        tc_commit(smem_addr(&b_v_empty[st]));
                        tc_commit(smem_addr(&b_s_free[sb]));
                    }
                    __syncwarp();
                    if (++sb == C::NS) {
                        sb = 0;
                        sbp ^= 1;
                    }
                    if (++st == NV) {
                        st = 0;
                        stp ^= 1;
                    }
                }
            }
        }
        // every product is done before tensor memory goes
        if (one)
            tc_commit(smem_addr(&b_end[scores]));
        __syncwarp();
        bar_wait(smem_addr(&b_end[scores]), 0);
    } else if (I8 && warp >= 16 && warp < 24) {
        // ---- codes to binary16: four warps the keys, four the values
        // A thread keeps its 16-byte chunk c and its row modulo the pass.  Eight
        // lanes that access shared memory together take half of one row's chunks
        // and the other half of the next one's, which keeps the swizzled reads
        // and writes free of bank conflicts.
        constexpr int CPR = C::RB / 16, RPP = 128 / CPR, PASSES = TP / RPP, PQ = PASSES < 4 ? PASSES : 4;
        constexpr int NSR = I8 ? C::NSR : 1;
        const int side = (warp - 16) >> 2;
        const int cw = tid & 127, u = cw % (2 * CPR), odd = (u >> 2) & 1;
        const int c = (u & 3) + (CPR == 8 ? 4 * (odd ^ (u >> 3)) : 0);
        const int r = cw / (2 * CPR) * 2 + odd;
        const unsigned src0 = r * C::RB + ((CPR == 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) << 4);
        const unsigned dst0 = (c >> 2) * (TP * 128) + r * 128 + ((((2 * c) & 7) ^ (r & 7)) << 4);
        const int ns = side ? NV : NK;
        const unsigned ring = sbase + (side ? C::OFF_V : C::OFF_OP);
        uint64_t *const full = side ? b_v_full : b_k_full, *const empty = side ? b_v_empty : b_k_empty;
        int i = 0, fs = 0, ph = 0;  // tile of the run; its slot and phase (counted: a
                                    // division by ns took longer than the codes)
        for (long long w = run.lo; w < run.hi;) {
            const Unit x = sched_unit<false>(a, RM, sm, run, w);
            const long long wend = min(run.hi, x.w1);
            const int n = x.h < 0 ? 0 : (int)(wend - tile_place(x, w));
            w = wend;
            for (int t = 0; t < n; ++t, ++i) {
                const int rs = i % NSR;
                wait(smem_addr(&b_raw_full[rs]), (i / NSR) & 1);
                if (i >= ns)
                    wait(smem_addr(&empty[fs]), ph ^ 1);
                const unsigned src = sbase + C::OFF_RAW + rs * 2 * C::RAW + side * C::RAW + src0;
                const unsigned dst = ring + fs * C::OPER;
#pragma unroll
                for (int p0 = 0; p0 < PASSES; p0 += PQ) {
                    uint4 q[PQ];
#pragma unroll
                    for (int j = 0; j < PQ; ++j)
                        q[j] = lds16(src + (p0 + j) * RPP * C::RB);
#pragma unroll
                    for (int j = 0; j < PQ; ++j) {
                        const unsigned b0 = q[j].x ^ 0x80808080u, b1 = q[j].y ^ 0x80808080u,
                                       b2 = q[j].z ^ 0x80808080u, b3 = q[j].w ^ 0x80808080u;
                        const unsigned at = dst + (p0 + j) * RPP * 128;
                        sts16(at + dst0, codes_lo(b0), codes_hi(b0), codes_lo(b1), codes_hi(b1));
                        sts16(at + (dst0 ^ 16), codes_lo(b2), codes_hi(b2), codes_lo(b3),
                              codes_hi(b3));
                    }
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(smem_addr(&full[fs]));
                    bar_arrive(smem_addr(&b_raw_empty[rs]));
                }
                if (++fs == ns) {
                    fs = 0;
                    ph ^= 1;
                }
            }
        }
    } else if (warp < 16) {
        // ---- softmax: stream sx takes every other tile, half hx of its columns
        constexpr int HC = TP / 2;  // columns of a half
        const int sx = (warp >> 2) & 1, hx = warp >> 3, ww = warp & 3, g = lane >> 2, t4 = lane & 3;
        const unsigned lanes = (unsigned)(32 * ww) << 16, low = 16u << 16;
        const unsigned tO = tmem + lanes + C::T_O + sx * 128;
        Finish<false, RM, C::SOFT, SoftSync> fin;
        int i0 = 0;  // tile of the run
        for (int k = 0;; ++k) {
            const int buf = k & 1;
            wait(smem_addr(&b_q_full[buf]), (k >> 1) & 1);
            // (all end together, or a barrier among them would not)
            const int n = any_of<C::SOFT>(1, wait.dead) ? 0 : s_n[buf], tile0 = s_tile0[buf];
            if (n == 0)
                break;
            const int len = s_unit[buf].len;
            float inv[2], m[2], l[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                inv[r] = s_inv[buf][16 * ww + g + 8 * r];
                m[r] = -INFINITY;
                l[r] = 0.f;
            }

            for (int t = sx; t < n; t += 2) {
                const int p0 = (tile0 + t) * TP;
                const bool edge = p0 + TP > len;
                // (weights overwrite their own scores)
                const int sb = (i0 + t) % C::NS;
                const unsigned tS = tmem + lanes + C::T_S + sb * 64;
                wait(smem_addr(&b_s_full[sb]), ((i0 + t) / C::NS) & 1);
                tc_fence_after();
                const float *sc =
                    scales + ((i0 + t) % C::NSC) * 2 * TP + hx * HC + 2 * t4;
                if (I8)
                    wait(smem_addr(&b_sc_full[(i0 + t) % C::NSC]), ((i0 + t) / C::NSC) & 1);
                unsigned seen[2] = {0xffu, 0xffu};  // bit 2 j + c: column 8 j + 2 t4 + c of the half
                if (edge) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const unsigned long long bits = s_bits[buf][16 * ww + g + 8 * r];
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const int q = p0 + hx * HC + 8 * (e >> 1) + 2 * t4 + (e & 1) - len;
                            if (!(q < 0 || (q < 64 && ((bits >> q) & 1))))
                                seen[r] &= ~(1u << e);
                        }
                    }
                    if (!I8) {
                        // a NaN or an infinity among the values must not reach rows
                        // that do not see it: taken out of the operand here
                        const int st = (i0 + t) % NV, tt = hx * 128 + (tid & 127);
                        wait(smem_addr(&b_v_full[st]), ((i0 + t) / NV) & 1);
                        if (tt < 2)
                            s_bad[sx][tt] = 0u;
                        stream_any(sx, false);
                        unsigned char *vb = smem + C::OFF_V + st * C::OPER;
                        for (int k2 = tt; k2 < C::OPER / 16; k2 += 256) {
                            uint4 *q = reinterpret_cast<uint4 *>(vb) + k2;
                            const uint4 u = *q;
                            const unsigned wd[4] = {u.x, u.y, u.z, u.w};
                            bool bad = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const unsigned z = wd[e] & 0x7c007c00u;
                                bad |= (z & 0xffffu) == 0x7c00u || (z >> 16) == 0x7c00u;
                            }
                            if (bad) {
                                *q = make_uint4(0u, 0u, 0u, 0u);
                                const int row = (k2 >> 3) & (TP - 1);
                                atomicOr(&s_bad[sx][row >> 5], 1u << (row & 31));
                            }
                        }
                        fence_async_smem();
                        stream_any(sx, false);
                    }
                }
                float v[16];
                // scores (without the row's factor): v[4 j + 2 r + c]
                auto scores = [&]() {
                    float lo[16];
                    tm_ld(tS + hx * HC, v);
                    tm_ld(tS + low + hx * HC, lo);
                    tm_wait_ld(v);
                    tm_wait_ld(lo);
#pragma unroll
                    for (int e = 0; e < 16; e += 2)
                        add2(v[e], v[e + 1], lo[e], lo[e + 1]);
                    if (I8) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 k2 = *reinterpret_cast<const float2 *>(sc + 8 * j);
                            mul2(v[4 * j], v[4 * j + 1], k2.x, k2.y);
                            mul2(v[4 * j + 2], v[4 * j + 3], k2.x, k2.y);
                        }
                    }
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (!((seen[(e >> 1) & 1] >> (2 * (e >> 2) + (e & 1))) & 1))
                                v[e] = -INFINITY;
                    }
                };
                // weights under the references; the sums of 2^(s - m) and the
                // largest weight
                auto weights = [&](float m0, float m1, float (&sum)[2], float (&big)[2]) {
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        float s0 = 0.f, s1 = 0.f;
                        big[r] = 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float &p = v[4 * j + 2 * r], &q = v[4 * j + 2 * r + 1];
                            fma2(p, q, inv[r], r ? -m1 : -m0);
                            p = ex2(p);
                            q = ex2(q);
                            add2(s0, s1, p, q);
                            if (I8) {
                                const float2 k2 =
                                    *reinterpret_cast<const float2 *>(sc + TP + 8 * j);
                                mul2(p, q, k2.x, k2.y);
                                if (edge) {
                                    p = (seen[r] >> (2 * j)) & 1 ? p : 0.f;
                                    q = (seen[r] >> (2 * j + 1)) & 1 ? q : 0.f;
                                }
                            }
                            big[r] = fmaxf(fmaxf(big[r], p), q);
                        }
                        sum[r] = s0 + s1;
                    }
                };
                float f[2] = {1.f, 1.f}, sum[2], big[2];
                scores();
                weights(m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1], sum, big);
                bool moved = false;
#pragma unroll
                for (int r = 0; r < 2; ++r)
                    moved |= !(big[r] <= kWeightMax && sum[r] <= kSumMax) || m[r] == -INFINITY;
                moved = stream_any(sx, moved);
                if (moved) {  // a row's first weights, or one out of range: rare
                    // (a row's reference moves for its own sake only, so that no row's
                    // bits depend on what another one sees)
                    bool move[2];
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const bool out =
                            !(big[r] <= kWeightMax && sum[r] <= kSumMax) || m[r] == -INFINITY;
                        move[r] = quad_max(out ? 1.f : 0.f) != 0.f;
                        if (t4 == 0)
                            s_out[sx][hx][16 * ww + g + 8 * r] = move[r];
                    }
                    scores();
                    float mn[2], ms[2];
                    // a row's maximum over both halves, by way of shared memory
                    auto row_max = [&](float (&x)[2], const bool scaled) {
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            x[r] = quad_max(x[r]) * (scaled ? inv[r] : 1.f);
                            if (t4 == 0)
                                s_max[sx][hx][16 * ww + g + 8 * r] = x[r];
                        }
                        stream_any(sx, false);
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const int row = 16 * ww + g + 8 * r;
                            x[r] = fmaxf(x[r], s_max[sx][hx ^ 1][row]);
                            if (scaled)
                                move[r] |= s_out[sx][hx ^ 1][row];
                        }
                        stream_any(sx, false);
                    };
                    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        top[(e >> 1) & 1] = fmaxf(top[(e >> 1) & 1], v[e]);
                    row_max(top, true);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        mn[r] = move[r] ? ref_from_scores(m[r], top[r]) : m[r];
                        ms[r] = mn[r] == -INFINITY ? 0.f : mn[r];
                    }
                    weights(ms[0], ms[1], sum, big);
                    row_max(big, false);
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const float m0 = mn[r];
                        mn[r] = move[r] ? ref_new(m[r], m0, big[r]) : m[r];
                        const float g2 = move[r] ? pow2(m0 - mn[r]) : 1.f;
                        sum[r] *= g2;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mul2(v[4 * j + 2 * r], v[4 * j + 2 * r + 1], g2, g2);
                        const float d = mn[r] == -INFINITY ? 0.f : m[r] - mn[r];
                        f[r] = pow2(d);
                        l[r] = times_pow2(l[r], d);
                        m[r] = mn[r];
                    }
                }
                unsigned ph[8], pl[8];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    l[r] += sum[r];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float p = v[4 * j + 2 * r], q = v[4 * j + 2 * r + 1];
                        ph[2 * j + r] = h2(p, q);
                        const float2 h =
                            __half22float2(*reinterpret_cast<const __half2 *>(&ph[2 * j + r]));
                        float dp = p, dq2 = q;
                        add2(dp, dq2, -h.x, -h.y);
                        pl[2 * j + r] = h2(dp, dq2);
                    }
                }
                if (!I8 && edge) {
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if ((s_bad[sx][hx] >> (8 * j + 2 * t4)) & (seen[r] >> (2 * j)) & 3)
                                l[r] = __int_as_float(0x7fc00000);  // its result is NaN
                }
                // (every score of the buffer was read before stream_any)
                tm_st_pairs(tS + hx * (HC / 2), ph);
                tm_st_pairs(tS + low + hx * (HC / 2), pl);
                if (t >= 2 && moved) {
                    // the output is at rest once the stream's tile before is through
                    wait(smem_addr(&b_s_free[(sb + 2) % C::NS]), ((i0 + t - 2) / C::NS) & 1);
                    tc_fence_after();
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int cb = 0; cb < D / 2; cb += 32) {
                            float o[16];
                            const unsigned at = tO + (half ? low : 0u) + hx * (D / 2) + cb;
                            tm_ld(at, o);
                            tm_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                o[e] *= f[(e >> 1) & 1];
                            tm_st(at, o);
                        }
                }
                tm_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(smem_addr(&b_p_full[sb]));
            }

            // ---- the chunk's end: both streams' outputs
            constexpr int QC = D / 4, NE = QC / 2;
            // (A buffer's phase can be waited for because its next product needs this
            // stream's weights; a count of the stream's products could not: two
            // may be outstanding, and a parity does not tell them apart.)
            const bool have = sx < n;  // this stream took a tile
            const int last = i0 + n - 1 - ((n - 1 - sx) & 1);
            if (have)
                wait(smem_addr(&b_s_free[last % C::NS]), (last / C::NS) & 1);
            i0 += n;
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                if (t4 == 0) {
                    s_m[sx][16 * ww + g + 8 * r] = m[r];
                    s_l[2 * sx + hx][16 * ww + g + 8 * r] = l[r];
                }
            }
            SoftSync::sync();
            // Group (sx, hx) finishes columns hx D / 2 + sx D / 4 and on, D / 4 of
            // them; the other stream's share of them comes through the unit's
            // query operand, whose products are all done.
            if (C::LONG && !(s_ends[buf] >> 1))  // the next chunk's queries are copied from here
                wait(smem_addr(&b_q_full[buf ^ 1]), ((k + 1) >> 1) & 1);
            float fac[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 16 * ww + g + 8 * r;
                const float M = fmaxf(s_m[0][row], s_m[1][row]);
                fac[r] = pow2(m[r] - (M == -INFINITY ? 0.f : M));
            }
            auto load_o = [&](int col, float (&o)[NE]) {
                float lo[NE];
                tm_ld(tO + col, o);
                tm_ld(tO + low + col, lo);
                tm_wait_ld(o);
                tm_wait_ld(lo);
#pragma unroll
                for (int e = 0; e < NE; ++e)
                    o[e] = (o[e] + lo[e]) * fac[(e >> 1) & 1];
            };
            // place of (hx, stream, ww, e / 2, lane): no bank conflicts
            float2 *const xq = reinterpret_cast<float2 *>(smem + buf * C::QB) +
                               (hx * 8 + ww) * (NE / 2) * 32 + lane;
            constexpr int SXS = 4 * (NE / 2) * 32;
            const int c0 = hx * (D / 2);
            float o[NE];
            if (have) {
                load_o(c0 + (sx ^ 1) * QC, o);
#pragma unroll
                for (int e = 0; e < NE / 2; ++e)
                    xq[(sx ^ 1) * SXS + e * 32] = make_float2(o[2 * e], o[2 * e + 1]);
                load_o(c0 + sx * QC, o);
            } else {
#pragma unroll
                for (int e = 0; e < NE; ++e)
                    o[e] = 0.f;
            }
            tc_fence_before();
            SoftSync::sync();
            if (sx == 1 || n > 1) {  // the other stream took a tile
#pragma unroll
                for (int e = 0; e < NE / 2; ++e) {
                    const float2 y = xq[sx * SXS + e * 32];
                    o[2 * e] += y.x;
                    o[2 * e + 1] += y.y;
                }
            }
            const Unit x = s_unit[buf];
            const bool all = fin.whole(run, x), first = !C::LONG || (s_ends[buf] & 1),
                       end = !C::LONG || s_ends[buf] >> 1;
            float *rec = fin.record(a, run, x);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 16 * ww + g + 8 * r;
                if (row >= x.nrows)
                    continue;
                float M = fmaxf(s_m[0][row], s_m[1][row]);
                const float ms = M == -INFINITY ? 0.f : M;
                float L = times_pow2(s_l[0][row] + s_l[1][row], s_m[0][row] - ms) +
                          times_pow2(s_l[2][row] + s_l[3][row], s_m[1][row] - ms);
                float *const part = rec + row * D + c0 + sx * QC + 2 * t4;
                if (!first) {  // what the part's chunks before have left there
                    const float mo = c_m[buf ^ 1][row], top = fmaxf(M, mo);
                    const float ts = top == -INFINITY ? 0.f : top;
                    const float fn = pow2(M - ts), fo = pow2(mo - ts);
                    L = times_pow2(c_l[buf ^ 1][row], mo - ts) + times_pow2(L, M - ts);
                    M = top;
#pragma unroll
                    for (int j = 0; j < QC / 8; ++j) {
                        const float2 y = __ldcg(reinterpret_cast<const float2 *>(part + 8 * j));
                        o[4 * j + 2 * r] = fmaf(y.x, fo, o[4 * j + 2 * r] * fn);
                        o[4 * j + 2 * r + 1] = fmaf(y.y, fo, o[4 * j + 2 * r + 1] * fn);
                    }
                }
                const float rl = L == 0.f ? 0.f : __frcp_rn(L);
                const bool res = all && end;
                float *dst = res ? a.out + out_at<false>(a, x, row) + c0 + sx * QC + 2 * t4 : part;
                const float fr = res ? rl : 1.f;
#pragma unroll
                for (int j = 0; j < QC / 8; ++j) {
                    const float2 y =
                        make_float2(o[4 * j + 2 * r] * fr, o[4 * j + 2 * r + 1] * fr);
                    if (res)
                        *reinterpret_cast<float2 *>(dst + 8 * j) = y;
                    else
                        __stcg(reinterpret_cast<float2 *>(dst + 8 * j), y);
                }
                if (warp < 4 && t4 == 0) {
                    if (!end) {
                        c_m[buf][row] = M;
                        c_l[buf][row] = L;
                    } else if (!all) {
                        __stcg(rec + RM * D + row, M);
                        __stcg(rec + RM * D + RM + row, L);
                    }
                }
            }
            if (end)
                fin.done(a, run, x);
            __syncwarp();  // every lane has read what lies in the buffer
            if (lane == 0)
                bar_arrive(smem_addr(&b_q_free[buf]));
        }
        // (the query operands are at rest)
        fin.end(a, run, sm, u_m, u_l, reinterpret_cast<float(*)[RM]>(smem));
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_PV) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(C::T_COLS)
                     : "memory");
    }
}

template <class C>
cudaError_t launch_tc(const KvAttnArgs &a, int nsm, cudaStream_t st)
{
    auto kern = k_kv_tc<C>;
    static DeviceOnce once;
    cudaError_t e = once.run([&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)C::SMEM);
    });
    if (e != cudaSuccess)
        return e;
    KvMaps maps;
    if ((e = kv_maps(a.c, a.B, C::TP, &maps)))
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nsm < kKvMaxCtas ? nsm : kKvMaxCtas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, a, maps);
}

template <bool I8, int D>
cudaError_t launch_i8(const KvAttnArgs &a, int nsm, cudaStream_t st)
{
    // A cache that holds no part of two chunks is attended without their code:
    // 670 us against 730 for 64-token trees over 32 x 96 heads x 2048 cached 8-bit
    // positions (binary16: 567 and 572).  At 8000 positions of 8 rows, where they
    // are needed: 560 us.  (The lengths are not known here: the capacity stands
    // for them.)
    using L = TcCfg<I8, D, true>;
    return a.c.cap > L::CHUNK * L::TP ? launch_tc<L>(a, nsm, st)
                                      : launch_tc<TcCfg<I8, D, false>>(a, nsm, st);
}

template <int D>
cudaError_t launch_d(const KvAttnArgs &a, int nsm, cudaStream_t st)
{
    return a.c.dtype == DV_I8 ? launch_i8<true, D>(a, nsm, st) : launch_i8<false, D>(a, nsm, st);
}

}  // namespace

cudaError_t launch_kv_tc(const KvAttnArgs &a, int nsm, cudaStream_t st)
{
    if (a.c.D == 128)
        return launch_d<128>(a, nsm, st);
    if (a.c.D == 64)
        return launch_d<64>(a, nsm, st);
    return cudaErrorInvalidValue;
}

}  // namespace dv
