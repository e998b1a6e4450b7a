// dv_kv_tc.cu -- attention of 9 to 64 query rows per KV head (drafted trees,
// grouped query heads) over a binary16 or 8-bit cache on tcgen05 (sm_103a).
//
// A unit's 64 query rows fill an M = 128 tile with their binary16 high and
// low parts: TMEM lanes 32 w .. 32 w + 15 hold the high parts of rows 16 w ..
// 16 w + 15, the next 16 lanes their low parts, so the sum of the two lane
// halves is the score to binary32's last bits, and the weights, split the
// same way, give the value product the same accuracy.  At that shape both
// products of a 64-position tile take about 512 tensor cycles, under the
// tile's time in memory (mma.sync needed 2048: 1959 us for 64-token trees of
// 32 rows at the 175B shape; see the launch rule for this kernel's time).
//
// Warps of a CTA (one CTA per SM):
//   0-3, 4-7  two softmax groups that take turns at the tiles, each with its
//             own score, weight and output columns in tensor memory; they are
//             merged when a unit ends, so neither waits for the other
//   8-11      8-bit caches: codes to binary16, raw ring -> operand ring
//   next      one warp of tensor-map copies (and scales by cp.async)
//   last      one thread issuing the MMAs; its warp owns tensor memory
// Keys are the K-major operand of the scores; values, as they lie, the
// MN-major operand of Q = softmax weights (A from tensor memory) x V.
// Hand-overs are mbarriers; every wait has a limit (DV_ERR_TIMEOUT).
//
// The running max only moves when a row's scores exceed it by 2^8, so the
// output in tensor memory is rarely rescaled; weights are kept below 2^14.
#include "dv_kv_tma.cuh"

namespace dv {
namespace {

template <bool I8_, int D_>
struct TcCfg {
    static constexpr bool I8 = I8_;
    static constexpr int D = D_, RM = 64, TP = kKvTile;
    static constexpr int RB = D * (I8 ? 1 : 2);           // bytes of a cached row
    static constexpr int OPER = TP * D * 2;               // a binary16 operand tile
    static constexpr int NSF = I8 ? 3 : (D == 128 ? 4 : 6);  // operand stages (K and V)
    static constexpr int RAW = TP * RB;
    static constexpr int NSR = I8 ? (D == 128 ? 2 : 4) : 0;   // raw stages
    static constexpr int NSC = 8;                         // scale slots (see the producer)
    static constexpr int QB = 128 * D * 2;
    static constexpr int LDO = D + 4;                     // padded row of the output buffer
    static constexpr int WARPS = 8 + (I8 ? 4 : 0) + 2, THREADS = 32 * WARPS;
    static constexpr int SOFT = 256;                      // softmax threads
    static constexpr int OFF_OP = QB;
    static constexpr int OFF_RAW = OFF_OP + NSF * 2 * OPER;
    static constexpr int OFF_SO = OFF_RAW + NSR * 2 * RAW;
    static constexpr int OFF_SC = OFF_SO + RM * LDO * 4;
    static constexpr size_t SMEM = 1024 + OFF_SC + (I8 ? NSC * 2 * TP * 4 : 0);
    // tensor-memory columns
    static constexpr int T_S = 0, T_O = 128, T_P = 384, T_COLS = 512;
};

struct SoftSync {
    DV_DEV static void sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
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

// 16 lanes x 64 columns: thread (g, t) = (lane / 4, lane % 4) holds columns 8 j
// + 2 t, + 1 of lanes g (v[4 j], v[4 j + 1]) and g + 8 (v[4 j + 2], v[4 j + 3]).
DV_DEV void tm_ld64(unsigned addr, float (&v)[32])
{
    unsigned r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
          "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
          "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
}
// The loads into v have landed (v passes through, so that no use moves before it).
DV_DEV void tm_wait_ld(float (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}
DV_DEV void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
DV_DEV void tm_st64(unsigned addr, const float (&v)[32])
{
    unsigned r[32];
#pragma unroll
    for (int i = 0; i < 32; ++i)
        r[i] = __float_as_uint(v[i]);
    asm volatile(
        "tcgen05.st.sync.aligned.16x256b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
// 16 lanes x 32 columns of binary16 pairs: r[2 j] columns 4 j + t of lane g,
// r[2 j + 1] of lane g + 8.
DV_DEV void tm_st_pairs(unsigned addr, const unsigned (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.16x128b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
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
    constexpr int D = C::D, RM = C::RM, TP = C::TP, NSF = C::NSF;
    constexpr bool I8 = C::I8;
    extern __shared__ unsigned char smem_raw[];
    __shared__ SchedSmem sm;
    __shared__ float s_m[2][RM], s_l[2][RM], u_m[RM], u_l[RM], s_inv[RM];
    __shared__ float wgt[kMergePieces][RM];
    __shared__ unsigned s_bad[2][2];  // binary16 edge tiles: positions not finite
    __shared__ __align__(8) uint64_t b_raw_full[I8 ? C::NSR : 1], b_raw_empty[I8 ? C::NSR : 1],
        b_sc_full[C::NSC], b_kv_full[NSF], b_kv_empty[NSF], b_s_full[2], b_p_full[2],
        b_pv_done[2], b_q_full, b_end;
    __shared__ unsigned s_tmem;
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    const unsigned sbase = smem_addr(smem);
    float *so = reinterpret_cast<float *>(smem + C::OFF_SO);
    float *scales = reinterpret_cast<float *>(smem + C::OFF_SC);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int W_MMA = C::WARPS - 1, W_LOAD = C::WARPS - 2;

    if (warp == W_MMA) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&s_tmem)),
                     "r"(C::T_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < C::NSR; ++i) {
            bar_init(smem_addr(&b_raw_full[i]), 1);
            bar_init(smem_addr(&b_raw_empty[i]), 4);
        }
        for (int i = 0; i < C::NSC; ++i)
            bar_init(smem_addr(&b_sc_full[i]), 32);
        for (int i = 0; i < NSF; ++i) {
            bar_init(smem_addr(&b_kv_full[i]), I8 ? 4 : 1);
            bar_init(smem_addr(&b_kv_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(smem_addr(&b_s_full[i]), 1);
            bar_init(smem_addr(&b_p_full[i]), 4);
            bar_init(smem_addr(&b_pv_done[i]), 1);
        }
        bar_init(smem_addr(&b_q_full), 8);
        bar_init(smem_addr(&b_end), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_fence_before();
    const Run run = sched_init<false>(a, RM, sm);  // (barriers)
    tc_fence_after();
    const unsigned tmem = s_tmem;
    Waiter wait{a.status};

    if (warp == W_LOAD) {
        // ---- copies.  A scale slot is reused 8 tiles later: by then the raw
        // (NSR) and operand (NSF) rings between have only let the copies this
        // far because the slot's tile has left the softmax.
        constexpr int NS = I8 ? C::NSR : NSF, BYTES = I8 ? C::RAW : C::OPER;
        static_assert(!I8 || C::NSR + NSF + 1 <= C::NSC, "scale slots");
        const unsigned ring = sbase + (I8 ? C::OFF_RAW : C::OFF_OP);
        int i = 0;  // tile of the run
        for (long long w = run.lo; w < run.hi;) {
            const Unit x = sched_unit<false>(a, RM, sm, run, w);
            const long long wend = min(run.hi, x.w1);
            if (x.h < 0) {
                w = wend;
                continue;
            }
            const int bh = unit_bh<false>(a, x);
            for (w = tile_place(x, w); w < wend; ++w, ++i) {
                const int slot = i % NS, p = tile_of(x, w) * TP;
                const unsigned full = smem_addr(I8 ? &b_raw_full[slot % (I8 ? C::NSR : 1)]
                                                   : &b_kv_full[slot % NSF]);
                const unsigned empty = smem_addr(I8 ? &b_raw_empty[slot % (I8 ? C::NSR : 1)]
                                                    : &b_kv_empty[slot % NSF]);
                if (i >= NS)
                    wait(empty, (i / NS - 1) & 1);
                if (I8) {
                    const int sc = i % C::NSC;
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
                }
                if (lane == 0) {
                    bar_expect(full, 2 * BYTES);
                    const unsigned dst = ring + slot * 2 * BYTES;
#pragma unroll
                    for (int xb = 0; xb < C::RB; xb += 128) {
                        tma_load(dst + xb * TP, &maps.k, xb, p, bh, full);
                        tma_load(dst + BYTES + xb * TP, &maps.v, xb, p, bh, full);
                    }
                }
                __syncwarp();
            }
        }
        if (I8)
            asm volatile("cp.async.wait_all;" ::: "memory");
        // no copy may outlive the CTA
        for (int k = max(0, i - NS); k < i; ++k)
            bar_wait(smem_addr(I8 ? &b_raw_full[k % (I8 ? C::NSR : 1)] : &b_kv_full[k % NSF]),
                     (k / NS) & 1);
    } else if (warp == W_MMA) {
        // ---- products
        if (lane == 0) {
            constexpr uint32_t ID_S = tc_idesc(TP, false), ID_O = tc_idesc(D, true);
            int i = 0, seg = 0, ph[2] = {0, 0};
            for (long long w = run.lo; w < run.hi;) {
                const Unit x = sched_unit<false>(a, RM, sm, run, w);
                const long long wend = min(run.hi, x.w1);
                if (x.h < 0) {
                    w = wend;
                    continue;
                }
                const int n = (int)(wend - tile_place(x, w));
                w = wend;
                wait(smem_addr(&b_q_full), seg & 1);
                ++seg;
                for (int t = 0; t <= n; ++t) {
                    if (t < n) {
                        const int st = (i + t) % NSF;
                        wait(smem_addr(&b_kv_full[st]), ((i + t) / NSF) & 1);
                        tc_fence_after();
                        const unsigned kb = sbase + C::OFF_OP + st * 2 * C::OPER;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            tc_mma_ss(tmem + C::T_S + (t & 1) * 64,
                                      tc_desc(sbase + (kk / 4) * (128 * 128) + (kk % 4) * 32, 16),
                                      tc_desc(kb + (kk / 4) * (TP * 128) + (kk % 4) * 32, 16), ID_S,
                                      kk > 0);
                        tc_commit(smem_addr(&b_s_full[t & 1]));
                    }
                    if (t > 0) {
                        const int st = (i + t - 1) % NSF, g = (t - 1) & 1;
                        wait(smem_addr(&b_p_full[g]), ph[g] & 1);
                        ++ph[g];
                        tc_fence_after();
                        const unsigned vb = sbase + C::OFF_OP + st * 2 * C::OPER + C::OPER;
#pragma unroll
                        for (int kk = 0; kk < TP / 16; ++kk)
                            tc_mma_ts(tmem + C::T_O + g * 128, tmem + C::T_P + g * 32 + kk * 8,
                                      tc_desc(vb + kk * 16 * 128, TP * 128), ID_O,
                                      t > 2 || kk > 0);
                        tc_commit(smem_addr(&b_pv_done[g]));
                        tc_commit(smem_addr(&b_kv_empty[st]));
                    }
                }
                i += n;
            }
            tc_commit(smem_addr(&b_end));  // every product is done before tensor memory goes
            bar_wait(smem_addr(&b_end), 0);
        }
        __syncwarp();
    } else if (I8 && warp >= 8) {
        // ---- codes to binary16
        const int cw = tid - 256;  // 0 .. 127
        constexpr int CPR = C::RB / 16;
        int i = 0;
        for (long long w = run.lo; w < run.hi;) {
            const Unit x = sched_unit<false>(a, RM, sm, run, w);
            const long long wend = min(run.hi, x.w1);
            const int n = x.h < 0 ? 0 : (int)(wend - tile_place(x, w));
            w = wend;
            for (int t = 0; t < n; ++t, ++i) {
                const int rs = i % (I8 ? C::NSR : 1), fs = i % NSF;
                wait(smem_addr(&b_raw_full[rs]), (i / (I8 ? C::NSR : 1)) & 1);
                if (i >= NSF)
                    wait(smem_addr(&b_kv_empty[fs]), (i / NSF - 1) & 1);
                const unsigned src = sbase + C::OFF_RAW + rs * 2 * C::RAW;
                const unsigned dst = sbase + C::OFF_OP + fs * 2 * C::OPER;
#pragma unroll 4
                for (int id = cw; id < 2 * TP * CPR; id += 128) {
                    const int side = id / (TP * CPR), r = id / CPR % TP, pc = id % CPR;
                    // (the copy swizzled the row's chunks)
                    const int c = C::RB == 64 ? pc ^ ((r >> 1) & 3) : pc ^ (r & 7);
                    const uint4 u = lds16(src + side * C::RAW + r * C::RB + pc * 16);
                    const unsigned b[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u,
                                           u.w ^ 0x80808080u};
                    const unsigned row = dst + side * C::OPER + (c >> 2) * (TP * 128) + r * 128;
                    const unsigned e = row + ((((2 * c) & 7) ^ (r & 7)) << 4);
                    const unsigned o = row + ((((2 * c + 1) & 7) ^ (r & 7)) << 4);
                    const bool odd = c >= 4;  // the halves in turn: no bank conflicts
                    const uint4 lo = make_uint4(codes_lo(b[0]), codes_hi(b[0]), codes_lo(b[1]),
                                                codes_hi(b[1]));
                    const uint4 hi = make_uint4(codes_lo(b[2]), codes_hi(b[2]), codes_lo(b[3]),
                                                codes_hi(b[3]));
                    const uint4 f = odd ? hi : lo, s = odd ? lo : hi;
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(odd ? o : e),
                                 "r"(f.x), "r"(f.y), "r"(f.z), "r"(f.w)
                                 : "memory");
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(odd ? e : o),
                                 "r"(s.x), "r"(s.y), "r"(s.z), "r"(s.w)
                                 : "memory");
                }
                fence_async_smem();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(smem_addr(&b_kv_full[fs]));
                    bar_arrive(smem_addr(&b_raw_empty[rs]));
                }
            }
        }
    } else {
        // ---- softmax
        const int wg = warp >> 2, ww = warp & 3, g = lane >> 2, t4 = lane & 3;
        const unsigned lanes = (unsigned)(32 * ww) << 16, low = 16u << 16;
        const unsigned tS = tmem + lanes + C::T_S + wg * 64, tO = tmem + lanes + C::T_O + wg * 128,
                       tP = tmem + lanes + C::T_P + wg * 32;
        const int G = a.H / a.c.Hkv;
        Finish<false, RM, C::SOFT, SoftSync> fin;
        int i0 = 0, nt = 0;  // tile of the run; this group's tiles so far
        for (long long w = run.lo; w < run.hi;) {
            const Unit x = sched_unit<false>(a, RM, sm, run, w);
            const long long wend = min(run.hi, x.w1), wb = tile_place(x, w);
            w = wend;
            if (x.h < 0)
                continue;
            const int n = (int)(wend - wb), tile0 = tile_of(x, wb);
            // the queries' parts (8 rows a warp)
            for (int r = warp; r < RM; r += 8) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (r < x.nrows && lane * 4 < D)
                    v = ld_row4(a.q, q_at<false>(a, x, r) + lane * 4);
                float inv;
                const SplitQ q = split_row(v, a.scale, &inv);
                if (lane * 4 < D) {
                    const int row = 32 * (r >> 4) + (r & 15), d = lane * 4;
                    unsigned char *p = smem + (d >> 6) * (128 * 128) + row * 128 +
                                       ((((d & 63) >> 3) ^ (row & 7)) << 4) + (d & 4) * 2;
                    *reinterpret_cast<uint2 *>(p) = make_uint2(q.hi01, q.hi23);
                    // (16 rows on: the same place in the swizzle)
                    *reinterpret_cast<uint2 *>(p + 16 * 128) = make_uint2(q.lo01, q.lo23);
                }
                if (lane == 0)
                    s_inv[r] = inv;
            }
            fence_async_smem();
            SoftSync::sync();
            if (lane == 0)
                bar_arrive(smem_addr(&b_q_full));
            float inv[2], m[2], l[2], sg[2];
            unsigned long long bits[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 16 * ww + g + 8 * r;
                inv[r] = s_inv[row];
                bits[r] = row < x.nrows ? seen_bits(a, x, (x.row0 + row) / G) : 0ull;
                m[r] = -INFINITY;
                l[r] = 0.f;
                sg[r] = 1.f;
            }

            for (int t = wg; t < n; t += 2, ++nt) {
                const int p0 = (tile0 + t) * TP;
                const bool edge = p0 + TP > x.len;
                wait(smem_addr(&b_s_full[wg]), nt & 1);
                tc_fence_after();
                float v[32], vl[32];
                tm_ld64(tS, v);
                tm_ld64(tS + low, vl);
                const float *sc = scales + ((i0 + t) % C::NSC) * 2 * TP;
                if (I8)
                    wait(smem_addr(&b_sc_full[(i0 + t) % C::NSC]), ((i0 + t) / C::NSC) & 1);
                tm_wait_ld(v);
                tm_wait_ld(vl);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    v[e] += vl[e];
                if (I8) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float2 k = *reinterpret_cast<const float2 *>(sc + 8 * j + 2 * t4);
                        v[4 * j] *= k.x;
                        v[4 * j + 1] *= k.y;
                        v[4 * j + 2] *= k.x;
                        v[4 * j + 3] *= k.y;
                    }
                }
                unsigned seen[2] = {0xffffu, 0xffffu};  // bit 2 j + c: column 8 j + 2 t4 + c
                if (edge) {
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int q = p0 + 8 * j + 2 * t4 + c - x.len;
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                if (!(q < 0 || (q < 64 && ((bits[r] >> q) & 1)))) {
                                    v[4 * j + 2 * r + c] = -INFINITY;
                                    seen[r] &= ~(1u << (2 * j + c));
                                }
                        }
                    if (!I8) {
                        // a NaN or an infinity among the values must not reach rows
                        // that do not see it: taken out of the operand here
                        const int st = (i0 + t) % NSF;
                        wait(smem_addr(&b_kv_full[st]), ((i0 + t) / NSF) & 1);
                        if (ww == 0 && lane < 2)
                            s_bad[wg][lane] = 0u;
                        asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory");
                        unsigned char *vb = smem + C::OFF_OP + st * 2 * C::OPER + C::OPER;
                        for (int k = tid & 127; k < C::OPER / 16; k += 128) {
                            uint4 *q = reinterpret_cast<uint4 *>(vb) + k;
                            uint4 u = *q;
                            unsigned wd[4] = {u.x, u.y, u.z, u.w};
                            bool bad = false;
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const unsigned z = wd[e] & 0x7c007c00u;
                                bad |= (z & 0xffffu) == 0x7c00u || (z >> 16) == 0x7c00u;
                            }
                            if (bad) {
                                *q = make_uint4(0u, 0u, 0u, 0u);
                                const int row = (k >> 3) & (TP - 1);
                                atomicOr(&s_bad[wg][row >> 5], 1u << (row & 31));
                            }
                        }
                        fence_async_smem();
                        asm volatile("bar.sync %0, 128;" ::"r"(2 + wg) : "memory");
                    }
                }
                float f[2];
                unsigned ph[16], pl[16];
                bool moved = false;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float mx = v[2 * r];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        mx = fmaxf(mx, fmaxf(v[4 * j + 2 * r], v[4 * j + 2 * r + 1]));
                    mx = quad_max(mx) * inv[r];
                    f[r] = 1.f;
                    if (mx > m[r] + 8.f) {
                        f[r] = ex2(m[r] - mx);
                        m[r] = mx;
                    }
                    const float ms = m[r] == -INFINITY ? 0.f : m[r];
                    float sum = 0.f, big = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float &p = v[4 * j + 2 * r + c];
                            p = ex2(fmaf(p, inv[r], -ms));
                            sum += p;
                        }
                    l[r] = fmaf(l[r], f[r], sum);
                    float up = 64.f;
                    if (I8) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const float2 k =
                                *reinterpret_cast<const float2 *>(sc + TP + 8 * j + 2 * t4);
                            float &p = v[4 * j + 2 * r], &q = v[4 * j + 2 * r + 1];
                            p = (seen[r] >> (2 * j)) & 1 ? p * k.x : 0.f;
                            q = (seen[r] >> (2 * j + 1)) & 1 ? q * k.y : 0.f;
                            big = fmaxf(big, fmaxf(p, q));
                        }
                        // weights relative to about the largest so far
                        big = fmaxf(sg[r] * f[r], quad_max(big));
                        if (big >= 256.f * sg[r] || (big < sg[r] * 0x1p-10f && big > 0.f)) {
                            const float now = fmaxf(
                                __uint_as_float(__float_as_uint(big) & 0x7f800000u), 0x1p-100f);
                            f[r] = f[r] * sg[r] / now;
                            sg[r] = now;
                        }
                        up = 64.f / sg[r];
                    }
                    moved |= f[r] != 1.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float w0 = v[4 * j + 2 * r] * up, w1 = v[4 * j + 2 * r + 1] * up;
                        ph[2 * j + r] = h2(w0, w1);
                        pl[2 * j + r] = h2_rest(w0, w1, ph[2 * j + r]);
                    }
                }
                if (!I8 && edge) {
#pragma unroll
                    for (int r = 0; r < 2; ++r)
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const int col = 8 * j + 2 * t4;
                            if ((s_bad[wg][col >> 5] >> (col & 31)) & (seen[r] >> (2 * j)) & 3)
                                l[r] = __int_as_float(0x7fc00000);  // its result is NaN
                        }
                }
                // the group's product before this one is done: weights and output are free
                if (t >= 2)
                    wait(smem_addr(&b_pv_done[wg]), (nt - 1) & 1);
                tc_fence_after();
                tm_st_pairs(tP, ph);
                tm_st_pairs(tP + low, pl);
                if (t >= 2 && __any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int cb = 0; cb < D; cb += 64) {
                            float o[32];
                            const unsigned at = tO + (half ? low : 0u) + cb;
                            tm_ld64(at, o);
                            tm_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] *= f[(e >> 1) & 1];
                            tm_st64(at, o);
                        }
                }
                tm_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(smem_addr(&b_p_full[wg]));
            }
            i0 += n;

            // ---- the unit's (part's) end: both groups' outputs
            const bool have = wg < n;  // this group took a tile
            if (have)
                wait(smem_addr(&b_pv_done[wg]), (nt - 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
                if (t4 == 0) {
                    s_m[wg][16 * ww + g + 8 * r] = m[r];
                    s_l[wg][16 * ww + g + 8 * r] = l[r];
                }
            }
            SoftSync::sync();
            float fac[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 16 * ww + g + 8 * r;
                const float M = fmaxf(s_m[0][row], s_m[1][row]), ms = M == -INFINITY ? 0.f : M;
                fac[r] = ex2(m[r] - ms) * (sg[r] * (1.f / 64.f));
                if (wg == 0 && t4 == 0) {
                    u_m[row] = M;
                    u_l[row] = s_l[0][row] * ex2(s_m[0][row] - ms) +
                               s_l[1][row] * ex2(s_m[1][row] - ms);
                }
            }
            for (int k = 0; k < 2; ++k) {
                if (k == wg && (have || k == 0)) {
#pragma unroll
                    for (int cb = 0; cb < D; cb += 64) {
                        float o[32], ol[32];
                        tm_ld64(tO + cb, o);
                        tm_ld64(tO + low + cb, ol);
                        tm_wait_ld(o);
                        tm_wait_ld(ol);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                float2 *q = reinterpret_cast<float2 *>(
                                    so + (16 * ww + g + 8 * r) * C::LDO + cb + 8 * j + 2 * t4);
                                const int e = 4 * j + 2 * r;
                                float2 val = make_float2((o[e] + ol[e]) * fac[r],
                                                         (o[e + 1] + ol[e + 1]) * fac[r]);
                                if (k) {
                                    const float2 was = *q;
                                    val = make_float2(was.x + val.x, was.y + val.y);
                                }
                                *q = val;
                            }
                    }
                    tc_fence_before();
                }
                SoftSync::sync();
            }
            fin.part(a, run, x, [&](int row, int d) { return so[row * C::LDO + d]; }, u_m, u_l);
        }
        fin.end(a, run, sm, u_m, u_l, wgt);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == W_MMA) {
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

}  // namespace

cudaError_t launch_kv_tc(const KvAttnArgs &a, int nsm, cudaStream_t st)
{
    const bool i8 = a.c.dtype == DV_I8;
    if (a.c.D == 128)
        return i8 ? launch_tc<TcCfg<true, 128>>(a, nsm, st)
                  : launch_tc<TcCfg<false, 128>>(a, nsm, st);
    if (a.c.D == 64)
        return i8 ? launch_tc<TcCfg<true, 64>>(a, nsm, st)
                  : launch_tc<TcCfg<false, 64>>(a, nsm, st);
    return cudaErrorInvalidValue;
}

}  // namespace dv
