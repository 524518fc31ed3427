// rope.cpp -- the plan of rotary positions: each pair's turns a position, with
// the scalings for contexts longer than the model's own, worked out on the host
// in 80-bit floating point (64 bits of mantissa, as many as a step has).
#include <algorithm>
#include <cmath>
#include <string>

#include "lw.h"

lw_status lw_fail(lw_status s, const std::string &msg);   // bundle.cpp

extern "C" lw_status lw_rope_make(const lw_rope_opts *o, lw_rope_plan *plan)
{
    if (!o || !plan) return lw_fail(LW_E_ARG, "null options or plan");
    const double most = 0x1p64;
    auto within = [](double x, double lo, double hi) { return x >= lo && x <= hi; };         // (false for NaN)
    if (o->pairs < 1 || o->pairs > LW_ROPE_MOST) return lw_fail(LW_E_ARG, "pairs must be in 1..256");
    if (o->layout != LW_ROPE_HALVES && o->layout != LW_ROPE_PAIRS) return lw_fail(LW_E_ARG, "unknown layout");
    if (o->scaling < LW_ROPE_PLAIN || o->scaling > LW_ROPE_TURNS) return lw_fail(LW_E_ARG, "unknown scaling");
    if (!std::isfinite(o->amplitude)) return lw_fail(LW_E_ARG, "amplitude must be finite");
    if (!within(o->base, 1.0, most)) return lw_fail(LW_E_ARG, "base must be in 1..2^64");
    if (o->scaling != LW_ROPE_PLAIN && !within(o->factor, 1.0 / most, most))
        return lw_fail(LW_E_ARG, "factor must be in 2^-64..2^64");
    if (o->scaling == LW_ROPE_BASE && o->pairs < 2) return lw_fail(LW_E_ARG, "a scaled base needs two pairs");
    if (o->scaling == LW_ROPE_INDEX || o->scaling == LW_ROPE_TURNS) {
        if (!(o->original > 0.0) || o->original > most) return lw_fail(LW_E_ARG, "original must be positive, at most 2^64");
        if (!(o->low >= 0.0) || o->low > most || !within(o->high, 0.0, most))
            return lw_fail(LW_E_ARG, "low and high must be in 0..2^64");
        if (o->scaling == LW_ROPE_TURNS && !(o->low < o->high)) return lw_fail(LW_E_ARG, "low must be below high");
        if (o->scaling == LW_ROPE_INDEX && !(o->base > 1.0 && o->low > 0.0 && o->high > 0.0))
            return lw_fail(LW_E_ARG, "base must be above 1, low and high positive");
    }
    typedef long double R;
    const int n = o->pairs;
    const R two_pi = 2 * 3.14159265358979323846264338327950288L;
    const R factor = o->scaling == LW_ROPE_PLAIN ? 1 : (R)o->factor;
    R base = o->base, lo = 0, hi = 1;
    if (o->scaling == LW_ROPE_BASE) base *= powl(factor, (R)n / (n - 1));
    if (o->scaling == LW_ROPE_INDEX) {
        // (at's arithmetic in 64 bits, as models' own programs have it: floor
        // and ceil are to fall the same way; so are the ends, each kept on one
        // side, also where that leaves hi below lo)
        auto at = [&](double turns) {
            return n * std::log(o->original / (turns * (2 * 3.14159265358979323846))) / std::log(o->base);
        };
        lo = std::max(std::floor(at(o->high)), 0.0);
        if (!std::isfinite(lo)) return lw_fail(LW_E_ARG, "original / (2 pi high) is past what 64 bits hold");
        hi = std::min(std::ceil(at(o->low)), 2.0 * n - 1);
        if (hi == lo) hi = lo + 0.001L;
    }
    plan->amplitude = o->amplitude;
    plan->pairs = n;
    plan->layout = o->layout;
    for (int i = 0; i < LW_ROPE_MOST; i++) {
        plan->step[i] = 0;
        if (i >= n) continue;
        R f = powl(base, -(R)i / n);
        if (o->scaling == LW_ROPE_LINEAR) f /= factor;
        if (o->scaling == LW_ROPE_INDEX) {
            const R r = std::min(std::max((i - lo) / (hi - lo), (R)0), (R)1);
            f *= 1 - r + r / factor;
        }
        if (o->scaling == LW_ROPE_TURNS) {
            const R s = std::min(std::max(((R)o->original * f / two_pi - o->low) / ((R)o->high - o->low), (R)0), (R)1);
            f *= s + (1 - s) / factor;
        }
        const R turn = f / two_pi, part = turn - floorl(turn);              // whole turns are none
        const R step = nearbyintl(part * 0x1p64L);
        plan->step[i] = step >= 0x1p64L ? 0 : (uint64_t)step;
    }
    return LW_OK;
}
