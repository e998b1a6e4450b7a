// dv_kv_mma.cu -- attention of up to 8 query rows per KV head over a binary16
// or 8-bit cache (single tokens, small trees, selected blocks) on tensor
// cores (sm_103a).
//
// The arithmetic is near binary32's although the products are mma.sync m16n8k16
// with binary16 operands: cached keys and values are exact in binary16 (8-bit
// codes are whole numbers; their scales multiply the scores and the weights),
// and queries and softmax weights are split into binary16 high and low parts,
// each scaled by a power of two so that the low part keeps its bits (22 of the
// number, dv_kv_tma.cuh).  The two parts of 8 rows fill the 16 rows of an MMA
// (rows 0-7 high, 8-15 low), and their results are added.
//
// Four warps take 16 positions each of a tile of 64, every warp from a ring
// of its own that one of its lanes fills by tensor-map copies (scales by
// 4-byte cp.async), NST tiles deep and on over the ends of units: no barrier
// between warps until a unit ends.  What bounds it is the cache's bytes; an
// 8-bit value costs about 0.7 instructions to become binary16, which is why
// a warp's 16 rows are filled with both parts instead of two products.  One
// token of 32 x 96 heads over 2049 positions: binary16 473 us, the bytes' own
// time; 8 bits 309 us of 245: 0.53 of the issue slots and 0.58 of the DRAM
// throughput are in use, the rest is those instructions' latencies.
//
// Rows are swizzled by the copy, and dimensions are dealt to the fragments so
// that a thread reads 16 contiguous bytes of a cached row at a time: the k
// index of the score product and the n index of the value product are
// permutations of the head dimension that the query fragments and the output
// order repeat.  Columns of the score tile are positions in an order that
// keeps both reads free of bank conflicts, and the weights leave the score
// fragments as the A operand of the value product without a shuffle.
#include "dv_kv_tma.cuh"

namespace dv {
namespace {

DV_DEV void mma(float (&c)[4], const uint4 &a, unsigned b0, unsigned b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// Position (0-7) of column n of a score tile: even columns as they are, odd
// ones with bit 2 flipped.  Rows of adjacent columns then differ in the bit
// that the swizzle needs for the key reads, and the even (odd) columns alone
// cover every even (odd) row for the value reads.
DV_DEV int col_pos(int n) { return (n & 1) ? (n ^ 4) : n; }

template <bool I8_, int D_, int NST_, int MINB_, bool LONG_>
struct Cfg {
    static constexpr bool LONG = LONG_;  // a warp may take more than FLUSH tiles of a unit
    static constexpr bool I8 = I8_;
    static constexpr int D = D_, NST = NST_, MINB = MINB_;
    static constexpr int WARPS = 4, THREADS = 32 * WARPS, RM = 8, PW = kKvTile / WARPS;
    static constexpr int RB = D * (I8 ? 1 : 2);  // bytes of a cached row
    static constexpr int CPR = RB / 16;
    static constexpr int KS = D / 16;            // MMA steps of a score
    static constexpr int NT = D / 8;             // n tiles of the values
    static constexpr int CH = I8 && D == 128 ? 16 : 8;  // contiguous values per thread and chunk
    static constexpr int SIDE = PW * RB;         // a warp's keys (values) of a tile
    static constexpr int RING = WARPS * NST * 2 * SIDE;
    static constexpr int SCALES = WARPS * NST * 2 * PW * 4;
    static constexpr int QF = KS * 32 * 16;
    static constexpr int SO = RM * D * 4;
    static constexpr size_t SMEM = 1024 + (size_t)RING + SCALES + QF + SO;
    static constexpr int FLUSH = 64;  // tiles whose values the tensor cores sum
    static_assert(PW == 16, "one k step of the value product");
};

// Byte offset of 16-byte chunk c of row r of a side.
template <class C>
DV_DEV int swz(int r, int c)
{
    if (C::RB == 64)
        return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
    return (c >> 3) * (C::PW * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

template <class C, bool BLOCK>
__global__ void __launch_bounds__(C::THREADS, C::MINB)
    k_kv_mma(const KvAttnArgs a, const __grid_constant__ KvMaps maps)
{
    constexpr int D = C::D, NT = C::NT, CH = C::CH, RM = C::RM, WP = C::WARPS;
    extern __shared__ unsigned char smem_raw[];
    __shared__ SchedSmem sm;
    __shared__ float s_m[WP][RM], s_l[WP][RM], u_m[RM], u_l[RM], s_inv[RM];
    __shared__ float wgt[kMergePieces][RM];
    __shared__ __align__(8) uint64_t s_bar[WP][C::NST];
    __shared__ int s_pos[WP][C::NST];
    unsigned char *smem = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    float *scales = reinterpret_cast<float *>(smem + C::RING);
    uint4 *qf = reinterpret_cast<uint4 *>(smem + C::RING + C::SCALES);
    float *so = reinterpret_cast<float *>(smem + C::RING + C::SCALES + C::QF);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    if (lane == 0) {
        for (int i = 0; i < C::NST; ++i)
            bar_init(smem_addr(&s_bar[warp][i]), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    const Run run = sched_init<BLOCK>(a, RM, sm);
    if (run.lo >= run.hi)
        return;
    Finish<BLOCK, RM, C::THREADS> fin;

    // ---- this warp's loads, NST - 1 tiles ahead of its products
    const unsigned ring = smem_addr(smem) + warp * C::NST * 2 * C::SIDE;
    const unsigned sring = smem_addr(scales) + warp * C::NST * 2 * C::PW * 4;
    Unit xl = sched_unit<BLOCK>(a, RM, sm, run, run.lo);
    int bhl = xl.h < 0 ? 0 : unit_bh<BLOCK>(a, xl);
    long long wl = tile_place(xl, run.lo);
    int sl = 0;  // its slot
    // block mode: the list entry of the next load, asked for one load ahead
    auto entry = [&](int tile) {
        const int e = (tile * kKvTile + warp * C::PW) >> a.blog;
        return e < xl.ent ? __ldg(a.idx + ((size_t)xl.b * a.H + xl.h) * a.k + e) : -1;
    };
    int jl = BLOCK ? entry(tile_of(xl, wl)) : 0;
    auto issue = [&]() {
        if (wl < run.hi) {
            if (wl >= xl.w1) {
                xl = sched_unit<BLOCK>(a, RM, sm, run, wl);
                wl = tile_place(xl, wl);
                bhl = xl.h < 0 ? 0 : unit_bh<BLOCK>(a, xl);
                if (BLOCK)
                    jl = entry(0);
            }
            const int tile = tile_of(xl, wl);
            int p = tile * kKvTile + warp * C::PW;
            if (BLOCK) {
                if (jl < 0 || jl > (xl.len - 1) >> a.blog) {
                    if (jl != -1 && lane == 0)
                        set_status(a.status, DV_ERR_DEVICE_INDEX);
                    p = -1;
                } else {
                    p = (jl << a.blog) + (p & (a.c.block - 1));
                }
                p = p < xl.len ? p : -1;
                if (wl + 1 < xl.w1)
                    jl = entry(tile + 1);
            } else {
                p = xl.h >= 0 && p < xl.len + xl.ntok ? p : -1;
            }
            if (lane == 0)
                s_pos[warp][sl] = p;
            if (p >= 0) {
                if (C::I8) {
                    const int i = lane & 15;
                    const size_t row = (size_t)bhl * a.c.cap + p + i;
                    cp4(sring + (sl * 2 + (lane >> 4)) * C::PW * 4 + i * 4,
                        (lane < 16 ? a.c.ks : a.c.vs) + (p + i < a.c.cap ? row : 0),
                        p + i < a.c.cap);
                }
                if (lane == 0) {
                    const unsigned bar = smem_addr(&s_bar[warp][sl]);
                    const unsigned dst = ring + sl * 2 * C::SIDE;
                    bar_expect(bar, 2 * C::SIDE);
#pragma unroll
                    for (int x = 0; x < C::RB; x += 128) {
                        tma_load(dst + x * C::PW, &maps.k, x, p, bhl, bar);
                        tma_load(dst + C::SIDE + x * C::PW, &maps.v, x, p, bhl, bar);
                    }
                }
            }
            ++wl;
            sl = sl + 1 == C::NST ? 0 : sl + 1;
        }
        if (C::I8)
            cp_commit();
    };
    __syncwarp();
#pragma unroll
    for (int i = 0; i < C::NST - 1; ++i)
        issue();

    const int pc0 = col_pos(2 * t), pc1 = col_pos(2 * t + 1);  // positions of this thread's columns
    const int kr = col_pos(g);                                 // key row of this thread
    int sc = 0;             // slot of the next tile
    unsigned phases = 0;    // its barriers' parities
    bool timed_out = false;

    for (long long w = run.lo; w < run.hi;) {
        const Unit x = sched_unit<BLOCK>(a, RM, sm, run, w);
        const long long wend = min(run.hi, x.w1);
        // ---- queries: scaled, split, in fragment order (two rows a warp)
        if (x.h >= 0) {
            constexpr int N = RM / WP;
            long long at[N];
            float4 v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int r = warp + WP * i;
                at[i] = r < x.nrows && lane * 4 < D ? q_at<BLOCK>(a, x, r) + lane * 4 : -1;
            }
            ld_queries(a.q, at, v);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int r = warp + WP * i;
                float inv;
                const SplitQ q = split_row(v[i], a.scale, &inv);
                constexpr int EPC = C::I8 ? 16 : 8, SPC = EPC / 4;  // steps per 16-byte chunk
                const int c = lane * 4 / EPC, s = SPC * (c / 4) + lane % SPC;
                if (lane * 4 < D)
                    qf[s * 32 + r * 4 + c % 4] = make_uint4(q.hi01, q.lo01, q.hi23, q.lo23);
                if (lane == 0)
                    s_inv[r] = inv;
            }
        }
        __syncthreads();
        const float inv = x.h >= 0 ? s_inv[g] : 0.f;
        const unsigned long long bits =
            !BLOCK && g < x.nrows ? seen_bits(a, x, row_token(a, x.row0 + g)) : 0ull;

        float o[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
            o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m = -INFINITY, l = 0.f;  // reference point, sum
        // Tensor cores cut their sums off instead of rounding them: every step
        // takes up to 2^-23 of a value, always towards zero.  So the values of
        // FLUSH tiles at a time are added here in binary32 (in local memory,
        // on purpose: as registers they would cost a CTA per SM).
        volatile float acc[NT * 2 + 1];  // values; sum
        int steps = 0;
        bool flushed = false;

        for (w = tile_place(x, w); w < wend; ++w) {
            if (C::I8)
                cp_wait<C::NST - 2>();
            __syncwarp();
            issue();  // into the slot of the tile before this one
            const int slot = sc;
            sc = sc + 1 == C::NST ? 0 : sc + 1;
            const int p0 = s_pos[warp][slot];
            if (p0 < 0)
                continue;
            if (!timed_out && !bar_wait(smem_addr(&s_bar[warp][slot]), (phases >> slot) & 1)) {
                timed_out = true;
                set_status(a.status, DV_ERR_TIMEOUT);
            }
            phases ^= 1u << slot;
            const unsigned st = ring + slot * 2 * C::SIDE;
            const bool edge = p0 + C::PW > x.len;  // some position may be unseen

            // ---- scores: 16 positions (columns), rows 0-7 high parts, 8-15 low
            float s[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
                s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
            for (int i = 0; i < C::CPR / 4; ++i) {
                unsigned kc[2][4];
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const uint4 u = lds16(st + swz<C>(8 * nt + kr, t + 4 * i));
                    kc[nt][0] = u.x;
                    kc[nt][1] = u.y;
                    kc[nt][2] = u.z;
                    kc[nt][3] = u.w;
                }
                if (C::I8) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 q = qf[(4 * i + j) * 32 + lane];
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt) {
                            const unsigned u = kc[nt][j] ^ 0x80808080u;
                            mma(s[nt], q, codes_lo(u), codes_hi(u));
                        }
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 q = qf[(2 * i + j) * 32 + lane];
#pragma unroll
                        for (int nt = 0; nt < 2; ++nt)
                            mma(s[nt], q, kc[nt][2 * j], kc[nt][2 * j + 1]);
                    }
                }
            }
            // row g: columns 2t, 2t + 1 of both halves
            float v[4], vs[4];
            const float *sp = scales + ((size_t)warp * C::NST + slot) * 2 * C::PW;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int ps = 8 * (e >> 1) + ((e & 1) ? pc1 : pc0);
                vs[e] = C::I8 ? sp[C::PW + ps] : 1.f;
                v[e] = (s[e >> 1][e & 1] + s[e >> 1][2 + (e & 1)]) * (C::I8 ? inv * sp[ps] : inv);
            }
            unsigned seen = 15u;
            if (edge) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = p0 + 8 * (e >> 1) + ((e & 1) ? pc1 : pc0) - x.len;
                    const bool on = j < 0 || (!BLOCK && j < 64 && ((bits >> j) & 1));
                    if (!on) {
                        v[e] = -INFINITY;
                        seen &= ~(1u << e);
                    }
                }
            }
            // ---- weights under the row's reference point (no reduction over the row)
            float p[4], sum, big;
            auto weights = [&](float ms) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p[e] = ex2(v[e] - ms);
                sum = (p[0] + p[1]) + (p[2] + p[3]);
                if (C::I8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        p[e] = (seen >> e) & 1 ? p[e] * vs[e] : 0.f;
                }
                big = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
            };
            weights(m == -INFINITY ? 0.f : m);
            const bool range = big <= kWeightMax && sum <= kSumMax && m != -INFINITY;
            if (!__all_sync(0xffffffffu, range)) {  // first weights, or one out of range: rare
                // (a row's reference moves for its own sake only, so that no row's
                // bits depend on what another one sees)
                const bool move = quad_max(range ? 0.f : 1.f) != 0.f;
                const float top = quad_max(fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])));
                const float m0 = move ? ref_from_scores(m, top) : m;
                weights(m0 == -INFINITY ? 0.f : m0);
                big = quad_max(big);
                const float mn = move ? ref_new(m, m0, big) : m, g2 = move ? pow2(m0 - mn) : 1.f;
                sum *= g2;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    p[e] *= g2;
                const float d = mn == -INFINITY ? 0.f : m - mn, f = pow2(d);
                m = mn;
                l = times_pow2(l, d);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    o[i][0] *= f;
                    o[i][1] *= f;
                    o[i][2] *= f;
                    o[i][3] *= f;
                }
                if (flushed) {
#pragma unroll
                    for (int i = 0; i < 2 * NT; ++i)
                        acc[i] = acc[i] * f;
                    acc[2 * NT] = times_pow2(acc[2 * NT], d);
                }
            }
            l += sum;
            unsigned hh[2], ll[2];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                hh[nt] = h2(p[2 * nt], p[2 * nt + 1]);
                ll[nt] = h2_rest(p[2 * nt], p[2 * nt + 1], hh[nt]);
            }
            const uint4 pw = make_uint4(hh[0], ll[0], hh[1], ll[1]);
            // ---- values
            unsigned bad = 0;  // edge tiles of binary16: positions not finite
            const int pos[4] = {pc0, pc1, 8 + pc0, 8 + pc1};
            constexpr int VI = NT / CH;  // 16-byte (or half) chunks per row
#pragma unroll
            for (int i = 0; i < VI; ++i) {
                unsigned vw[4][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (C::I8 && D == 64) {
                        const uint2 u =
                            lds8(st + C::SIDE + swz<C>(pos[e], g >> 1) + 8 * (g & 1));
                        vw[e][0] = u.x;
                        vw[e][1] = u.y;
                        vw[e][2] = vw[e][3] = 0u;
                    } else {
                        const uint4 u = lds16(st + C::SIDE + swz<C>(pos[e], g + 8 * i));
                        vw[e][0] = u.x;
                        vw[e][1] = u.y;
                        vw[e][2] = u.z;
                        vw[e][3] = u.w;
                    }
                }
                if (!C::I8 && edge) {
                    // a NaN or an infinity must not reach rows that do not see it:
                    // taken out of the product here, given back below
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const unsigned u = vw[e][j] & 0x7c007c00u;
                            if ((u & 0xffffu) == 0x7c00u || (u >> 16) == 0x7c00u) {
                                vw[e][j] = 0u;
                                bad |= 1u << e;
                            }
                        }
                }
                constexpr int WV = C::I8 ? CH / 4 : 4;  // words per chunk
#pragma unroll
                for (int j = 0; j < WV; ++j) {
                    if (C::I8) {
                        const unsigned x0 = vw[0][j] ^ 0x80808080u, x1 = vw[1][j] ^ 0x80808080u;
                        const unsigned x2 = vw[2][j] ^ 0x80808080u, x3 = vw[3][j] ^ 0x80808080u;
                        const unsigned a01 = __byte_perm(x0, x1, 0x5140);
                        const unsigned a23 = __byte_perm(x0, x1, 0x7362);
                        const unsigned b01 = __byte_perm(x2, x3, 0x5140);
                        const unsigned b23 = __byte_perm(x2, x3, 0x7362);
                        mma(o[i * CH + 4 * j], pw, codes_lo(a01), codes_lo(b01));
                        mma(o[i * CH + 4 * j + 1], pw, codes_hi(a01), codes_hi(b01));
                        mma(o[i * CH + 4 * j + 2], pw, codes_lo(a23), codes_lo(b23));
                        mma(o[i * CH + 4 * j + 3], pw, codes_hi(a23), codes_hi(b23));
                    } else {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mma(o[i * CH + 2 * j + k], pw,
                                __byte_perm(vw[0][j], vw[1][j], k ? 0x7632 : 0x5410),
                                __byte_perm(vw[2][j], vw[3][j], k ? 0x7632 : 0x5410));
                    }
                }
            }
            if (!C::I8 && edge) {
                bad |= __shfl_xor_sync(0xffffffffu, bad, 4);
                bad |= __shfl_xor_sync(0xffffffffu, bad, 8);
                bad |= __shfl_xor_sync(0xffffffffu, bad, 16);
                if (bad & seen)
                    l = __int_as_float(0x7fc00000);  // the row's result is NaN
            }
            if (C::LONG && ++steps == C::FLUSH) {
                steps = 0;
#pragma unroll
                for (int i = 0; i < 2 * NT; ++i) {
                    float *p = o[i >> 1];
                    const float val = p[i & 1] + p[2 + (i & 1)];
                    acc[i] = flushed ? acc[i] + val : val;
                    p[i & 1] = p[2 + (i & 1)] = 0.f;
                }
                acc[2 * NT] = flushed ? acc[2 * NT] + l : l;
                l = 0.f;
                flushed = true;
            }
        }
        if (x.h < 0)
            continue;

        // ---- merge the warps
        if (flushed)
            l += acc[2 * NT];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t == 0) {
            s_m[warp][g] = m;
            s_l[warp][g] = l;
        }
        __syncthreads();
        float M = -INFINITY;
#pragma unroll
        for (int i = 0; i < WP; ++i)
            M = fmaxf(M, s_m[i][g]);
        const float ms = M == -INFINITY ? 0.f : M;
        const float fac = pow2(m - ms);
        if (warp == 0 && t == 0) {
            float L = 0.f;
#pragma unroll
            for (int i = 0; i < WP; ++i)
                L += times_pow2(s_l[i][g], s_m[i][g] - ms);
            u_m[g] = M;
            u_l[g] = L;
        }
        // so[n tile][column parity][lane], warps in order
        for (int i = 0; i < WP; ++i) {
            if (warp == i && g < x.nrows) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float *q = so + (n * 2 + c) * 32 + lane;
                        const float sum = o[n][c] + o[n][2 + c];
                        const float val = (flushed ? acc[2 * n + c] + sum : sum) * fac;
                        *q = i ? *q + val : val;
                    }
            }
            __syncthreads();
        }
        fin.part(a, run, x, [&](int row, int d) {
            const int n = d / CH % 8, nt = d / (8 * CH) * CH + d % CH;
            return so[(nt * 2 + (n & 1)) * 32 + row * 4 + n / 2];
        }, u_m, u_l);
    }
    if (C::I8)
        cp_wait<0>();
    if (timed_out)  // no copy may outlive the CTA (a wait with the same limit)
        for (int i = 0; i < C::NST; ++i)
            bar_wait(smem_addr(&s_bar[warp][i]), ~(phases >> i) & 1);
    fin.end(a, run, sm, u_m, u_l, wgt);
}

template <class C, bool BLOCK>
cudaError_t launch_cfg(const KvAttnArgs &a, int nsm, cudaStream_t st)
{
    auto kern = k_kv_mma<C, BLOCK>;
    static DeviceOnce once;
    static int per_sm[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if ((e = once.run([&] { return kv_occupancy(kern, C::THREADS, C::SMEM, &per_sm[dev]); })))
        return e;
    KvMaps maps;
    if ((e = kv_maps(a.c, a.B, C::PW, &maps)))
        return e;
    cudaLaunchConfig_t cfg = {};
    const int grid = nsm * per_sm[dev];
    cfg.gridDim = dim3(grid < kKvMaxCtas ? grid : kKvMaxCtas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, a, maps);
}

template <bool I8, int D>
cudaError_t launch_d(const KvAttnArgs &a, int nsm, cudaStream_t st)
{
    // rings of 48 KB (8 bits) and 96 KB: room for a third CTA per SM, and for two
    constexpr int NST = 3 * (128 / D), MINB = I8 ? 3 : 2;
    // Units of at most FLUSH tiles have no use for the code that adds the
    // outputs up in between: 32 rows of 2049 8-bit positions of 96 heads take
    // 309 us without it, 360 with it (binary16: 473 and 476).  Where it is needed, at
    // 8000 positions of 8 rows: 329 us.  (The lengths are not known here: the capacity
    // stands for them.)
    using L = Cfg<I8, D, NST, MINB, true>;
    using S = Cfg<I8, D, NST, MINB, false>;
    const long long listed = a.idx ? (long long)a.k * a.c.block : a.c.cap;
    const bool longer = (listed < a.c.cap ? listed : a.c.cap) > L::FLUSH * kKvTile;
    if (a.idx)
        return longer ? launch_cfg<L, true>(a, nsm, st) : launch_cfg<S, true>(a, nsm, st);
    return longer ? launch_cfg<L, false>(a, nsm, st) : launch_cfg<S, false>(a, nsm, st);
}

}  // namespace

cudaError_t launch_kv_mma(const KvAttnArgs &a, int nsm, cudaStream_t st)
{
    const bool i8 = a.c.dtype == DV_I8;
    if (a.c.D == 128)
        return i8 ? launch_d<true, 128>(a, nsm, st) : launch_d<false, 128>(a, nsm, st);
    if (a.c.D == 64)
        return i8 ? launch_d<true, 64>(a, nsm, st) : launch_d<false, 64>(a, nsm, st);
    return cudaErrorInvalidValue;
}

}  // namespace dv
