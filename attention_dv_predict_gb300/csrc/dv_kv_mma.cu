// dv_kv_mma.cu -- attention over a binary16 or 8-bit KV cache for drafted
// trees and selected blocks on tensor cores (sm_103a).
//
// The arithmetic is binary32 to its last bits although the products are
// mma.sync m16n8k16 with binary16 operands: cached keys and values are exact
// in binary16 (8-bit codes are whole numbers; their scales multiply the
// scores and the weights), and queries and softmax weights are split into
// binary16 high and low parts, each scaled by a power of two so that the low
// part keeps its bits.  Up to 8 query rows put both parts into the 16 rows
// of one MMA (rows 0-7 high, 8-15 low); more rows take two MMAs.
//
// Tiles of 64 positions come into shared memory by 16-byte cp.async
// (swizzled, so that every fragment read is free of bank conflicts), NST
// deep; loads run ahead over the ends of units.  Positions without a row are
// filled with zeros.  Dimensions are dealt to the fragments so that a thread
// reads 16 contiguous bytes of a cached row at a time: the k index of the
// score product and the n index of the value product are permutations of the
// head dimension that the query fragments and the output order repeat.
// Likewise columns of the score tile are positions in an order r(n) that
// keeps both reads conflict-free, and the weights leave the score fragments
// as the A operand of the value product without a shuffle.
#include <cuda_fp16.h>

#include "dv_kv_sched.cuh"

namespace dv {
namespace {

DV_DEV void cp16(unsigned dst, const void *src, bool on)
{
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 16 : 0)
                 : "memory");
}
DV_DEV void cp4(unsigned dst, const void *src, bool on)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(on ? 4 : 0)
                 : "memory");
}
DV_DEV void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
DV_DEV void cp_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

DV_DEV uint4 lds16(unsigned a)
{
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "r"(a));
    return r;
}
DV_DEV uint2 lds8(unsigned a)
{
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
    return r;
}

DV_DEV void mma(float (&c)[4], const uint4 &a, unsigned b0, unsigned b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

DV_DEV unsigned h2(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&h);
}
// The part of (a, b) that the binary16 pair `hi` leaves.
DV_DEV unsigned h2_rest(float a, float b, unsigned hi)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return h2(a - f.x, b - f.y);
}

DV_DEV float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
DV_DEV float quad_max(float v)
{
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// Position (0-7) of column n of a score tile: even columns as they are, odd
// ones with bit 2 flipped.  Rows of adjacent columns then differ in the bit
// that the swizzle needs for the key reads, and the even (odd) columns alone
// cover every even (odd) row for the value reads.
DV_DEV int col_pos(int n) { return (n & 1) ? (n ^ 4) : n; }

template <bool I8_, int D_, int WM_, int WP_, bool PACK_, int NST_, int MINB_>
struct Cfg {
    static constexpr bool I8 = I8_, PACK = PACK_;
    static constexpr int D = D_, WM = WM_, WP = WP_, NST = NST_, MINB = MINB_;
    static constexpr int THREADS = 32 * WM * WP;
    static constexpr int RW = PACK ? 8 : 16;   // query rows per warp
    static constexpr int RM = WM * RW;         // per unit
    static constexpr int PW = kKvTile / WP;    // positions of a tile per warp
    static constexpr int RB = D * (I8 ? 1 : 2);  // bytes of a cached row
    static constexpr int CPR = RB / 16;
    static constexpr int KS = D / 16;          // MMA steps of a score
    static constexpr int NT = D / 8;           // n tiles of the values
    static constexpr int CH = I8 && D == 128 ? 16 : 8;  // contiguous values per thread and chunk
    static constexpr int TILE = kKvTile * RB;
    static constexpr int STAGE = 2 * TILE + 3 * kKvTile * 4;  // K, V, scales, mask
    static constexpr int QF = WM * KS * (PACK ? 1 : 2) * 32 * 16;
    static constexpr int SO = RM * D * 4;
    static constexpr size_t SMEM = (size_t)NST * STAGE + QF + SO;
};

// Byte offset of 16-byte chunk c of tile row r.
template <class C>
DV_DEV int swz(int r, int c)
{
    return C::CPR >= 8 ? r * C::RB + ((c ^ (r & 7)) << 4)
                       : r * C::RB + ((c ^ ((r >> 1) & 3)) << 4);
}

// One tile of unit x into a stage; WM == 1: the calling warp's positions only.
template <class C, bool BLOCK>
DV_DEV void load_tile(const KvAttnArgs &a, const Unit &x, size_t base, int tile, unsigned stage)
{
    constexpr bool OWN = C::WM == 1;
    constexpr int ROWS = OWN ? C::PW : kKvTile, N = OWN ? 32 : C::THREADS;
    const int r0 = OWN ? (int)(threadIdx.x >> 5) * C::PW : 0;
    const int id0 = OWN ? threadIdx.x & 31 : threadIdx.x;
    const int end = x.len + x.ntok;
    const char *K = static_cast<const char *>(a.c.k);
    const char *V = static_cast<const char *>(a.c.v);
    static_assert(N % C::CPR == 0, "a thread keeps its chunk");
    const int c = id0 % C::CPR;
#pragma unroll
    for (int i = 0; i < (ROWS * C::CPR + N - 1) / N; ++i) {
        const int r = r0 + id0 / C::CPR + i * (N / C::CPR);
        if ((ROWS * C::CPR) % N != 0 && r >= r0 + ROWS)
            break;
        int p;
        if (BLOCK) {
            p = block_pos(a, x, tile * kKvTile + r);
        } else {
            p = tile * kKvTile + r;
            p = p < end ? p : -1;
        }
        const bool on = p >= 0;
        const size_t row = on ? base + p : base;
        const unsigned dst = stage + swz<C>(r, c);
        cp16(dst, K + row * C::RB + c * 16, on);
        cp16(dst + C::TILE, V + row * C::RB + c * 16, on);
        if (C::I8 && c < 2)
            cp4(stage + 2 * C::TILE + c * kKvTile * 4 + r * 4, (c ? a.c.vs : a.c.ks) + row, on);
        if (BLOCK && c == C::CPR - 1) {
            const unsigned m = stage + 2 * C::TILE + 2 * kKvTile * 4 + r * 4;
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(m), "f"(on ? 0.f : -INFINITY)
                         : "memory");
        }
    }
}

template <class C, bool BLOCK>
__global__ void __launch_bounds__(C::THREADS, C::MINB) k_kv_mma(const KvAttnArgs a)
{
    constexpr int D = C::D, KS = C::KS, NT = C::NT, CH = C::CH, RM = C::RM, WP = C::WP;
    constexpr int NR = C::PACK ? 1 : 2;  // query rows per thread
    constexpr int PS = C::PW < 32 ? C::PW : 32, NTL = PS / 8, NV = 2 * NTL;  // positions a step
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ SchedSmem sm;
    __shared__ float s_m[WP][RM], s_l[WP][RM], u_m[RM], u_l[RM], s_al[RM], s_inv[RM];
    __shared__ unsigned long long s_bits[RM];
    __shared__ float wgt[kMergePieces][RM];
    uint4 *qf = reinterpret_cast<uint4 *>(smem + (size_t)C::NST * C::STAGE);
    float *so = reinterpret_cast<float *>(smem + (size_t)C::NST * C::STAGE + C::QF);
    const unsigned ring = (unsigned)__cvta_generic_to_shared(smem);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int wm = warp % C::WM, wp = warp / C::WM;
    const int G = a.H / a.c.Hkv;
    const Run run = sched_init<BLOCK>(a, RM, sm);
    if (run.lo >= run.hi)
        return;

    // loads run C::NST - 1 tiles ahead of the products
    Unit xl = sched_unit<BLOCK>(a, RM, sm, run, run.lo);
    auto unit_base = [&](const Unit &u) {
        return ((size_t)u.b * a.c.Hkv + (BLOCK ? u.h / G : u.h)) * (size_t)a.c.cap;
    };
    long long wl = run.lo;
    size_t bl = unit_base(xl);
    unsigned sl = ring;  // stage of the next load
    auto issue = [&]() {
        if (wl < run.hi) {
            if (wl >= xl.w1) {
                xl = sched_unit<BLOCK>(a, RM, sm, run, wl);
                bl = unit_base(xl);
            }
            if (xl.h >= 0)
                load_tile<C, BLOCK>(a, xl, bl, (int)(wl - xl.w0), sl);
            ++wl;
            sl = sl + C::STAGE == ring + C::NST * C::STAGE ? ring : sl + C::STAGE;
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < C::NST - 1; ++i)
        issue();

    // a tile is shared by the warps of different query rows, or a warp's own
    auto sync_tile = [&]() {
        if (C::WM > 1)
            __syncthreads();
        else
            __syncwarp();
    };
    unsigned st_next = ring;  // stage of the next tile
    const int pc0 = col_pos(2 * t), pc1 = col_pos(2 * t + 1);  // positions of this thread's columns
    const int kr = col_pos(g);                                 // key row of this thread

    for (long long w = run.lo; w < run.hi;) {
        const Unit x = sched_unit<BLOCK>(a, RM, sm, run, w);
        const long long wend = min(run.hi, x.w1);
        if (x.h < 0) {
            for (; w < wend; ++w) {
                cp_wait<C::NST - 2>();
                sync_tile();
                issue();
                st_next = st_next + C::STAGE == ring + C::NST * C::STAGE ? ring
                                                                        : st_next + C::STAGE;
            }
            continue;
        }
        // ---- queries: power-of-two scaled, split, in fragment order
        for (int r = warp; r < RM; r += C::THREADS / 32) {
            float mx = 0.f;
            if (r < x.nrows)
                for (int d = lane * 4; d < D; d += 128) {
                    const float4 v = ld_row4(a.q, q_at<BLOCK>(a, x, r) + d);
                    mx = amax2(mx, amax2(amax2(v.x, v.y), amax2(v.z, v.w)));
                }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                mx = amax2(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (lane == 0) {
                mx *= fabsf(a.scale);
                int e = 0;
                if (mx > 0.f && mx <= 3.402823466e38f)
                    frexpf(mx, &e);
                e = min(max(14 - e, -126), 100);  // largest element into [2^13, 2^14)
                s_al[r] = ldexpf(1.f, e);
                s_inv[r] = ldexpf(1.f, -e);
                s_bits[r] = !BLOCK && r < x.nrows ? seen_bits(a, x, (x.row0 + r) / G) : 0ull;
            }
        }
        __syncthreads();
        for (int i = tid; i < C::WM * KS * 32; i += C::THREADS) {
            const int ln = i & 31, s = (i >> 5) % KS, m = (i >> 5) / KS;
            constexpr int SPC = C::I8 ? 4 : 2;  // steps per 16-byte chunk
            const int d = ((ln & 3) + 4 * (s / SPC)) * (C::I8 ? 16 : 8) + 4 * (s % SPC);
            unsigned hi[2][2] = {}, lo[2][2] = {};
#pragma unroll
            for (int hr = 0; hr < NR; ++hr) {
                const int r = m * C::RW + (ln >> 2) + 8 * hr;
                if (r < x.nrows) {
                    const float4 v = ld_row4(a.q, q_at<BLOCK>(a, x, r) + d);
                    const float al = s_al[r], sc = a.scale;
                    const float e0 = v.x * sc * al, e1 = v.y * sc * al, e2 = v.z * sc * al,
                                e3 = v.w * sc * al;
                    hi[hr][0] = h2(e0, e1);
                    hi[hr][1] = h2(e2, e3);
                    lo[hr][0] = h2_rest(e0, e1, hi[hr][0]);
                    lo[hr][1] = h2_rest(e2, e3, hi[hr][1]);
                }
            }
            if (C::PACK) {
                qf[i] = make_uint4(hi[0][0], lo[0][0], hi[0][1], lo[0][1]);
            } else {
                const int at = ((m * KS + s) * 2) * 32 + ln;
                qf[at] = make_uint4(hi[0][0], hi[1][0], hi[0][1], hi[1][1]);
                qf[at + 32] = make_uint4(lo[0][0], lo[1][0], lo[0][1], lo[1][1]);
            }
        }
        __syncthreads();
        float inv[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r)
            inv[r] = s_inv[wm * C::RW + g + 8 * r];

        float o[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
            o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[NR], l[NR], sg[NR];  // max, sum, power of two the weights are taken over
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
            sg[r] = 1.f;
        }

        for (; w < wend; ++w) {
            cp_wait<C::NST - 2>();
            sync_tile();
            issue();  // into the stage of the tile before this one
            const unsigned st = st_next;
            st_next = st_next + C::STAGE == ring + C::NST * C::STAGE ? ring : st_next + C::STAGE;
            const int p0 = (int)(w - x.w0) * kKvTile;
            const bool edge = !BLOCK && p0 + kKvTile > x.len;  // some position may be unseen
            // ---- PS positions at a time
#pragma unroll 1
            for (int pb = wp * C::PW; pb < (wp + 1) * C::PW; pb += PS) {
                float s[NTL][4], sl2[C::PACK ? 1 : NTL][4];
#pragma unroll
                for (int nt = 0; nt < NTL; ++nt) {
                    s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
                    if (!C::PACK)
                        sl2[nt][0] = sl2[nt][1] = sl2[nt][2] = sl2[nt][3] = 0.f;
                }
                const uint4 *qw = qf + wm * KS * (C::PACK ? 1 : 2) * 32 + lane;
                auto step = [&](int ks, const unsigned (&b0)[NTL], const unsigned (&b1)[NTL]) {
                    const uint4 q = qw[ks * (C::PACK ? 1 : 2) * 32];
#pragma unroll
                    for (int nt = 0; nt < NTL; ++nt)
                        mma(s[nt], q, b0[nt], b1[nt]);
                    if (!C::PACK) {
                        const uint4 ql = qw[(ks * 2 + 1) * 32];
#pragma unroll
                        for (int nt = 0; nt < NTL; ++nt)
                            mma(sl2[nt], ql, b0[nt], b1[nt]);
                    }
                };
#pragma unroll
                for (int i = 0; i < C::CPR / 4; ++i) {
                    unsigned kc[NTL][4];
#pragma unroll
                    for (int nt = 0; nt < NTL; ++nt) {
                        const uint4 u = lds16(st + swz<C>(pb + 8 * nt + kr, t + 4 * i));
                        kc[nt][0] = u.x;
                        kc[nt][1] = u.y;
                        kc[nt][2] = u.z;
                        kc[nt][3] = u.w;
                    }
                    unsigned b0[NTL], b1[NTL];
                    if (C::I8) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
#pragma unroll
                            for (int nt = 0; nt < NTL; ++nt) {
                                const unsigned u = kc[nt][j] ^ 0x80808080u;
                                b0[nt] = codes_lo(u);
                                b1[nt] = codes_hi(u);
                            }
                            step(4 * i + j, b0, b1);
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
#pragma unroll
                            for (int nt = 0; nt < NTL; ++nt) {
                                b0[nt] = kc[nt][2 * j];
                                b1[nt] = kc[nt][2 * j + 1];
                            }
                            step(2 * i + j, b0, b1);
                        }
                    }
                }
                // ---- scores of row g (and g + 8): columns 2t, 2t + 1 of each tile
                float v[NR][NV];
#pragma unroll
                for (int nt = 0; nt < NTL; ++nt) {
                    if (C::PACK) {
                        v[0][2 * nt] = s[nt][0] + s[nt][2];
                        v[0][2 * nt + 1] = s[nt][1] + s[nt][3];
                    } else {
                        v[0][2 * nt] = s[nt][0] + sl2[nt][0];
                        v[0][2 * nt + 1] = s[nt][1] + sl2[nt][1];
                        v[NR - 1][2 * nt] = s[nt][2] + sl2[nt][2];
                        v[NR - 1][2 * nt + 1] = s[nt][3] + sl2[nt][3];
                    }
                }
                const float *sc = reinterpret_cast<const float *>(
                    smem + (st - ring) + 2 * C::TILE) + pb;
                float vs[NV];
#pragma unroll
                for (int e = 0; e < NV; ++e) {
                    const int ps = 8 * (e >> 1) + ((e & 1) ? pc1 : pc0);
                    const float kscl = C::I8 ? sc[ps] : 1.f;
                    vs[e] = C::I8 ? sc[kKvTile + ps] : 1.f;
                    const float add = BLOCK ? sc[2 * kKvTile + ps] : 0.f;
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        const float f = C::I8 ? inv[r] * kscl : inv[r];
                        v[r][e] = BLOCK ? fmaf(v[r][e], f, add) : v[r][e] * f;
                    }
                }
                unsigned seen[NR];
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    seen[r] = (1u << NV) - 1;
                if (edge) {
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        const unsigned long long bits = s_bits[wm * C::RW + g + 8 * r];
#pragma unroll
                        for (int e = 0; e < NV; ++e) {
                            const int j = p0 + pb + 8 * (e >> 1) + ((e & 1) ? pc1 : pc0) - x.len;
                            const bool on = j < 0 || (j < 64 && ((bits >> j) & 1));
                            if (!on) {
                                v[r][e] = -INFINITY;
                                seen[r] &= ~(1u << e);
                            }
                        }
                    }
                }
                // ---- running max, weights, their power of two
                float f[NR];
                unsigned hh[NR][NTL], ll[NR][NTL];  // weights, high and low parts
                bool moved = false;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    float mx = v[r][0];
#pragma unroll
                    for (int e = 1; e < NV; ++e)
                        mx = fmaxf(mx, v[r][e]);
                    mx = quad_max(mx);
                    const float mn = fmaxf(m[r], mx), ms = mn == -INFINITY ? 0.f : mn;
                    f[r] = ex2(m[r] - ms);
                    m[r] = mn;
                    float p[NV], sum = 0.f;
#pragma unroll
                    for (int e = 0; e < NV; ++e) {
                        p[e] = ex2(v[r][e] - ms);
                        sum += p[e];
                    }
                    l[r] = fmaf(l[r], f[r], sum);
                    float up = 16384.f;
                    if (C::I8) {
                        float big = 0.f;
#pragma unroll
                        for (int e = 0; e < NV; ++e) {
                            p[e] = (seen[r] >> e) & 1 ? p[e] * vs[e] : 0.f;
                            big = fmaxf(big, p[e]);
                        }
                        // weights relative to the largest so far: the low part keeps
                        // its bits whatever the scales are
                        big = fmaxf(sg[r] * f[r], quad_max(big));
                        if (big >= 2.f * sg[r] || (big < sg[r] * 0x1p-10f && big > 0.f)) {
                            const float now = fmaxf(
                                __uint_as_float(__float_as_uint(big) & 0x7f800000u), 0x1p-100f);
                            f[r] = f[r] * sg[r] / now;
                            sg[r] = now;
                        }
                        up = 16384.f / sg[r];
                    }
                    moved |= f[r] != 1.f;
#pragma unroll
                    for (int nt = 0; nt < NTL; ++nt) {
                        const float w0 = p[2 * nt] * up, w1 = p[2 * nt + 1] * up;
                        hh[r][nt] = h2(w0, w1);
                        ll[r][nt] = h2_rest(w0, w1, hh[r][nt]);
                    }
                }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        o[i][0] *= f[0];
                        o[i][1] *= f[0];
                        // (PACK: rows 8-15 are the low parts of the same rows)
                        o[i][2] *= f[NR - 1];
                        o[i][3] *= f[NR - 1];
                    }
                }
                // ---- values, 16 positions a product
                unsigned bad = 0;  // edge tiles of binary16: positions not finite
#pragma unroll
                for (int kk = 0; kk < NTL / 2; ++kk) {
                    uint4 ph, pl;
                    if (C::PACK) {
                        ph = make_uint4(hh[0][2 * kk], ll[0][2 * kk], hh[0][2 * kk + 1],
                                        ll[0][2 * kk + 1]);
                    } else {
                        ph = make_uint4(hh[0][2 * kk], hh[NR - 1][2 * kk], hh[0][2 * kk + 1],
                                        hh[NR - 1][2 * kk + 1]);
                        pl = make_uint4(ll[0][2 * kk], ll[NR - 1][2 * kk], ll[0][2 * kk + 1],
                                        ll[NR - 1][2 * kk + 1]);
                    }
                    const int pos[4] = {pb + 16 * kk + pc0, pb + 16 * kk + pc1,
                                        pb + 16 * kk + 8 + pc0, pb + 16 * kk + 8 + pc1};
                    constexpr int VI = NT / CH;  // 16-byte (or half) chunks per row
#pragma unroll
                    for (int i = 0; i < VI; ++i) {
                        unsigned vw[4][4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (C::I8 && D == 64) {
                                const uint2 u = lds8(st + C::TILE + swz<C>(pos[e], g >> 1) +
                                                     8 * (g & 1));
                                vw[e][0] = u.x;
                                vw[e][1] = u.y;
                                vw[e][2] = vw[e][3] = 0u;
                            } else {
                                const uint4 u = lds16(st + C::TILE + swz<C>(pos[e], g + 8 * i));
                                vw[e][0] = u.x;
                                vw[e][1] = u.y;
                                vw[e][2] = u.z;
                                vw[e][3] = u.w;
                            }
                        }
                        if (!C::I8 && !BLOCK && edge) {
                            // a NaN or an infinity must not reach rows that do not see it:
                            // taken out of the product here, given back below
#pragma unroll
                            for (int e = 0; e < 4; ++e)
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const unsigned u = vw[e][j] & 0x7c007c00u;
                                    if ((u & 0xffffu) == 0x7c00u || (u >> 16) == 0x7c00u) {
                                        vw[e][j] = 0u;
                                        bad |= 1u << (4 * kk + e);
                                    }
                                }
                        }
                        constexpr int WV = C::I8 ? CH / 4 : 4;  // words per chunk
#pragma unroll
                        for (int j = 0; j < WV; ++j) {
                            if (C::I8) {
                                const unsigned x0 = vw[0][j] ^ 0x80808080u,
                                               x1 = vw[1][j] ^ 0x80808080u,
                                               x2 = vw[2][j] ^ 0x80808080u,
                                               x3 = vw[3][j] ^ 0x80808080u;
                                const unsigned a01 = __byte_perm(x0, x1, 0x5140);
                                const unsigned a23 = __byte_perm(x0, x1, 0x7362);
                                const unsigned b01 = __byte_perm(x2, x3, 0x5140);
                                const unsigned b23 = __byte_perm(x2, x3, 0x7362);
                                const unsigned b0[4] = {codes_lo(a01), codes_hi(a01),
                                                        codes_lo(a23), codes_hi(a23)};
                                const unsigned b1[4] = {codes_lo(b01), codes_hi(b01),
                                                        codes_lo(b23), codes_hi(b23)};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    mma(o[i * CH + 4 * j + k], ph, b0[k], b1[k]);
                                    if (!C::PACK)
                                        mma(o[i * CH + 4 * j + k], pl, b0[k], b1[k]);
                                }
                            } else {
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const unsigned b0 =
                                        __byte_perm(vw[0][j], vw[1][j], k ? 0x7632 : 0x5410);
                                    const unsigned b1 =
                                        __byte_perm(vw[2][j], vw[3][j], k ? 0x7632 : 0x5410);
                                    mma(o[i * CH + 2 * j + k], ph, b0, b1);
                                    if (!C::PACK)
                                        mma(o[i * CH + 2 * j + k], pl, b0, b1);
                                }
                            }
                        }
                    }
                }
                if (!C::I8 && !BLOCK && edge) {
                    bad |= __shfl_xor_sync(0xffffffffu, bad, 4);
                    bad |= __shfl_xor_sync(0xffffffffu, bad, 8);
                    bad |= __shfl_xor_sync(0xffffffffu, bad, 16);
#pragma unroll
                    for (int r = 0; r < NR; ++r)
                        if (bad & seen[r])
                            l[r] = __int_as_float(0x7fc00000);  // its result is NaN
                }
            }
        }

        // ---- merge the warps of a row group
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            if (t == 0) {
                s_m[wp][wm * C::RW + g + 8 * r] = m[r];
                s_l[wp][wm * C::RW + g + 8 * r] = l[r];
            }
        }
        __syncthreads();
        float fac[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            const int row = wm * C::RW + g + 8 * r;
            float M = -INFINITY;
#pragma unroll
            for (int i = 0; i < WP; ++i)
                M = fmaxf(M, s_m[i][row]);
            const float ms = M == -INFINITY ? 0.f : M;
            fac[r] = ex2(m[r] - ms) * (sg[r] * (1.f / 16384.f));
            if (wp == 0 && t == 0) {
                float L = 0.f;
#pragma unroll
                for (int i = 0; i < WP; ++i)
                    L += s_l[i][row] * ex2(s_m[i][row] - ms);
                u_m[row] = M;
                u_l[row] = L;
            }
        }
        // so[wm][n tile][row half][column parity][lane], warps in order
        float *mine = so + wm * NT * NR * 64 + lane;
        for (int i = 0; i < WP; ++i) {
            if (wp == i) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float val =
                                (C::PACK ? o[n][c] + o[n][2 + c] : o[n][2 * r + c]) * fac[r];
                            float *p = mine + ((n * NR + r) * 2 + c) * 32;
                            *p = i ? *p + val : val;
                        }
            }
            __syncthreads();
        }
        finish_unit<BLOCK, RM, C::THREADS>(
            a, run, x, sm, so, u_m, u_l, wgt,
            [](int row, int d) {
                const int n = d / CH % 8, nt = d / (8 * CH) * CH + d % CH;
                const int gr = row % 8, r = row / 8 % NR, wr = row / C::RW;
                return (((wr * NT + nt) * NR + r) * 2 + (n & 1)) * 32 + gr * 4 + n / 2;
            },
            [](int i) { return i / (NT * NR * 64) * C::RW + i / 64 % NR * 8 + i % 32 / 4; });
    }
    cp_wait<0>();
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
    e = once.run([&] {
        cudaError_t r = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)C::SMEM);
        if (r == cudaSuccess)
            r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm[dev], kern, C::THREADS,
                                                              C::SMEM);
        return r;
    });
    if (e != cudaSuccess)
        return e;
    if (per_sm[dev] < 1)
        return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    const int grid = nsm * per_sm[dev];
    cfg.gridDim = dim3(grid < kKvMaxCtas ? grid : kKvMaxCtas);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <bool I8, int D>
cudaError_t launch_d(const KvAttnArgs &a, int rows, int nsm, cudaStream_t st)
{
    constexpr int NST = (I8 ? 3 : 2) * (128 / D) + (I8 ? 0 : 1);
    constexpr int N2 = !I8 && D == 128 ? 2 : NST;  // two CTAs per SM
    constexpr int MB = I8 || D == 64 ? 3 : 2;
    if (a.idx)
        return launch_cfg<Cfg<I8, D, 1, 4, true, NST, MB>, true>(a, nsm, st);
    switch (rows) {
    case 8: return launch_cfg<Cfg<I8, D, 1, 4, true, NST, MB>, false>(a, nsm, st);
    case 16: return launch_cfg<Cfg<I8, D, 1, 4, false, N2, 2>, false>(a, nsm, st);
    case 32: return launch_cfg<Cfg<I8, D, 2, 2, false, N2, 2>, false>(a, nsm, st);
    case 64: return launch_cfg<Cfg<I8, D, 4, 2, false, NST, 1>, false>(a, nsm, st);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_kv_mma(const KvAttnArgs &a, int rows, int nsm, cudaStream_t st)
{
    const bool i8 = a.c.dtype == DV_I8;
    if (a.c.D == 128)
        return i8 ? launch_d<true, 128>(a, rows, nsm, st) : launch_d<false, 128>(a, rows, nsm, st);
    if (a.c.D == 64)
        return i8 ? launch_d<true, 64>(a, rows, nsm, st) : launch_d<false, 64>(a, rows, nsm, st);
    return cudaErrorInvalidValue;
}

}  // namespace dv
