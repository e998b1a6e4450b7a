// dv_rope_steps.cpp -- angles of rotation per position in units of 2^-64 turns
// (host).  See include/dv.h.
//
// A kernel multiplies a step by positions up to 2^31, so a step is worth no more
// than its last bits: in binary64 the fastest pairs would be off by some hundred
// units (2^-25 of a turn at position 2^30).  Everything is held in binary128
// (113 bits) and rounded once.  g++ computes binary128 in software on x86 and on Arm
// (where it is long double), so the steps are the same on both.
#include <cmath>

#include "dv.h"

namespace {

#if __LDBL_MANT_DIG__ == 113
typedef long double f128;
#else
typedef __float128 f128;
#endif

const f128 kTau = 2 * ((f128)3.141592653589793116 + (f128)1.2246467991473531772e-16);

// x^(-1 / n) of x >= 1: a binary64 power and two Newton steps of y^n x = 1 (its
// relative error of up to 2^-43, for exponents near 700, falls to n 2^-86, then
// below binary128's roundings).
f128 inverse_root(double x, int n)
{
    f128 y = std::pow(x, -1.0 / n);
    for (int step = 0; step < 2; ++step) {
        f128 p = x;
        for (int i = 0; i < n; ++i)
            p *= y;
        y -= y * (p - 1) / n;
    }
    return y;
}

// The pair that makes `turns` turns over the trained length.
double dim_of_turns(double turns, int rot, double theta, double orig)
{
    return rot * std::log(orig / (turns * 2 * 3.14159265358979323846)) / (2 * std::log(theta));
}

}  // namespace

extern "C" int dv_rope_steps(int rot_dim, double theta, int scaling, double factor,
                             double orig_len, double low, double high, uint64_t *steps)
{
    if (rot_dim < 2 || rot_dim % 2 || rot_dim > 256 || !(theta > 1) || !std::isfinite(theta) ||
        !steps || scaling < DV_ROPE_NONE || scaling > DV_ROPE_RAMP_INDEX)
        return DV_ERR_INVALID_ARG;
    if (scaling != DV_ROPE_NONE && (!(factor >= 1) || !std::isfinite(factor)))
        return DV_ERR_INVALID_ARG;
    const bool ramp = scaling == DV_ROPE_RAMP || scaling == DV_ROPE_RAMP_INDEX;
    if (ramp && (!(orig_len > 0) || !std::isfinite(orig_len) || !(low < high) || !(low > 0) ||
                 !std::isfinite(high)))
        return DV_ERR_INVALID_ARG;
    if (scaling == DV_ROPE_BASE && rot_dim == 2)
        return DV_ERR_INVALID_ARG;
    const int pairs = rot_dim / 2;
    f128 ratio = inverse_root(theta, pairs);  // of a pair's angle to the one before
    if (scaling == DV_ROPE_BASE)  // (factor^(rot / (rot - 2)))^(-2 / rot)
        ratio *= inverse_root(factor, pairs - 1);
    double i0 = 0, i1 = 0;
    if (scaling == DV_ROPE_RAMP_INDEX) {
        i0 = std::fmax(std::floor(dim_of_turns(high, rot_dim, theta, orig_len)), 0);
        i1 = std::fmin(std::ceil(dim_of_turns(low, rot_dim, theta, orig_len)), rot_dim - 1);
        if (i0 == i1)
            i1 += 0.001;
    }
    f128 f = 1;
    for (int i = 0; i < pairs; ++i, f *= ratio) {
        f128 w = 1;
        if (scaling == DV_ROPE_RAMP)
            w = (orig_len * f / kTau - low) / ((f128)high - low);
        if (scaling == DV_ROPE_RAMP_INDEX)
            w = 1 - (i - (f128)i0) / ((f128)i1 - i0);
        w = w > 0 ? w < 1 ? w : 1 : 0;
        f128 angle = f;
        if (scaling == DV_ROPE_LINEAR)
            angle /= factor;
        else if (ramp)
            angle *= w + (1 - w) / factor;
        steps[i] = (uint64_t)(angle / kTau * 0x1p64 + (f128)0.5);
    }
    return DV_OK;
}
