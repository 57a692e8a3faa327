// Host side of the operators around the quantized product: argument checks
// and tables that need no GPU.
#include <cmath>

#include "q4_cache4_host.h"

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

q4_status check_cache4(const q4_cache4* c, const char* who)
{
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return fail(Q4_ERR_INVALID_ARG, "%s: null cache or cache pointer", who);
    if (c->pages < 1 || c->kv_heads < 1 || c->page_size < 1 || c->dim < 1)
        return fail(Q4_ERR_INVALID_ARG, "%s: cache of %d pages, %d heads, %d rows a page, %d values", who, c->pages,
                    c->kv_heads, c->page_size, c->dim);
    if ((long long)c->pages * c->page_size > 0x7fffffffLL)
        return fail(Q4_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 rows in the cache", who);
    if (c->dim % 32 || c->dim > 256)
        return fail(Q4_ERR_UNSUPPORTED, "%s: heads of %d values (a multiple of 32, at most 256)", who, c->dim);
    if ((c->group != 32 && c->group != 64 && c->group != 128 && c->group != 256) || c->dim % c->group)
        return fail(Q4_ERR_UNSUPPORTED, "%s: groups of %d values (32, 64, 128 or 256, a divisor of %d)", who, c->group, c->dim);
    for (int i = 0; i < 3; ++i) {
        if (c->k_stride[i] < 0 || c->v_stride[i] < 0 || c->k_stride[i] % 16 || c->v_stride[i] % 16)
            return fail(Q4_ERR_UNSUPPORTED, "%s: strides of the codes must be multiples of 16 bytes", who);
        if (c->k_scale_stride[i] < 0 || c->v_scale_stride[i] < 0 || c->k_scale_stride[i] % 4 || c->v_scale_stride[i] % 4)
            return fail(Q4_ERR_UNSUPPORTED, "%s: strides of the scales must be multiples of 4 bytes", who);
    }
    if (c->k_stride[2] > (1 << 26) || c->v_stride[2] > (1 << 26) || c->k_scale_stride[2] > (1 << 26) || c->v_scale_stride[2] > (1 << 26))
        return fail(Q4_ERR_UNSUPPORTED, "%s: rows of a page more than 2^26 bytes apart", who);
    auto off = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; };
    if (off(c->k, 16) || off(c->v, 16) || off(c->k_scale, 4) || off(c->v_scale, 4))
        return fail(Q4_ERR_UNSUPPORTED, "%s: codes must be 16-byte, scales 4-byte aligned", who);
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

extern "C" q4_status q4_check_cache4(const q4_cache4* c)
{
    const char* who = "q4_check_cache4";
    if (q4_status st = q4::check_cache4(c, who); st != Q4_OK) return st;
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < i; ++j)
            if (q4::meet(q4::cache4_view(c, i & 1, i & 2), q4::cache4_view(c, j & 1, j & 2)))
                return q4::fail(Q4_ERR_INVALID_ARG, "%s: keys, values and their scales overlap", who);
    return Q4_OK;
}
