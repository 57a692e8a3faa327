// Host side of the operators around the quantized product: argument checks
// and tables that need no GPU.
#include <cmath>

#include "q4_internal.h"

namespace q4 {

q4_status check_cache(const q4_cache* c, const char* who)
{
    if (!c || !c->k || !c->v) return fail(Q4_ERR_INVALID_ARG, "%s: null cache or cache pointer", who);
    if (c->pages < 1 || c->kv_heads < 1 || c->page_size < 1 || c->dim < 1)
        return fail(Q4_ERR_INVALID_ARG, "%s: cache of %d pages, %d heads, %d rows a page, %d values", who, c->pages,
                    c->kv_heads, c->page_size, c->dim);
    if ((long long)c->pages * c->page_size > 0x7fffffffLL)
        return fail(Q4_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 rows in the cache", who);
    return Q4_OK;
}

}  // namespace q4

extern "C" q4_status q4_rotary_plan(int dim, int rot, int scaling, double base, double factor, int original_length,
                                    double low, double high, uint64_t* turns, float* magnitude)
{
    const char* who = "q4_rotary";
    if (!turns || !magnitude) return q4::fail(Q4_ERR_INVALID_ARG, "%s: null output", who);
    if (dim < 2 || rot < 2 || rot % 2 || rot > dim)
        return q4::fail(Q4_ERR_INVALID_ARG, "%s: %d rotated values (even, 2 .. dim) of a head of %d", who, rot, dim);
    if (dim > Q4_ROTARY_MAX_DIM)
        return q4::fail(Q4_ERR_UNSUPPORTED, "%s: heads of %d values (at most %d)", who, dim, Q4_ROTARY_MAX_DIM);
    if (!(base > 1.0) || !std::isfinite(base)) return q4::fail(Q4_ERR_INVALID_ARG, "%s: base %g is not above 1", who, base);
    if (scaling < Q4_ROTARY_NONE || scaling > Q4_ROTARY_BY_PARTS)
        return q4::fail(Q4_ERR_INVALID_ARG, "%s: unknown scaling %d", who, scaling);
    if (scaling != Q4_ROTARY_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
        return q4::fail(Q4_ERR_INVALID_ARG, "%s: factor %g is not 1 or more", who, factor);
    if (scaling == Q4_ROTARY_BASE && rot < 4)
        return q4::fail(Q4_ERR_INVALID_ARG, "%s: a scaled base needs at least 4 rotated values", who);
    if (scaling == Q4_ROTARY_BY_PARTS && (original_length < 1 || !(high > low) || !std::isfinite(low) || !std::isfinite(high)))
        return q4::fail(Q4_ERR_INVALID_ARG, "%s: by parts needs original_length >= 1 and low < high", who);
    // long double: 64 bits of mantissa, as many as the table keeps
    const long double pi2 = 6.283185307179586476925286766559L;
    const int n = rot / 2;
    long double b = base;
    const long double f = factor;
    if (scaling == Q4_ROTARY_BASE) b *= powl(f, (long double)rot / (rot - 2));
    for (int i = 0; i < n; ++i) {
        long double w = powl(b, -(long double)i / n);     // radians a position
        if (scaling == Q4_ROTARY_LINEAR) w /= f;
        if (scaling == Q4_ROTARY_BY_PARTS) {
            long double keep = (original_length * w / pi2 - low) / ((long double)high - low);
            keep = keep < 0 ? 0 : keep > 1 ? 1 : keep;
            w = w * keep + w / f * (1 - keep);
        }
        turns[i] = (uint64_t)roundl(w / pi2 * 18446744073709551616.0L);
    }
    *magnitude = scaling == Q4_ROTARY_BY_PARTS ? (float)(0.1L * logl(f) + 1.0L) : 1.f;
    return Q4_OK;
}
