// q4::meet against bytes counted out, for random small views, and the layouts
// that the operators' arguments come in.
#include <cstdio>
#include <random>
#include <set>

#include "q4_meet.h"

using q4::View;

static std::set<int64_t> bytes_of(const View& v)
{
    std::set<int64_t> s;
    for (int64_t a = 0; a < v.dim[0].count; ++a)
        for (int64_t b = 0; b < v.dim[1].count; ++b)
            for (int64_t c = 0; c < v.dim[2].count; ++c)
                for (int64_t i = 0; i < v.inner; ++i)
                    s.insert((int64_t)(uintptr_t)v.at + a * v.dim[0].stride + b * v.dim[1].stride + c * v.dim[2].stride + i);
    return s;
}

static const void* at(int64_t a) { return reinterpret_cast<const void*>((uintptr_t)a); }

static View heads(int64_t where, int64_t token, int64_t head, int tokens, int n, int dim)
{
    return View{at(where), dim * 2, {{tokens, token * 2}, {n, head * 2}, {1, 0}}};
}

#define EXPECT(x) \
    if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; }

int main()
{
    std::mt19937 rng(5);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    int yes = 0, no = 0;
    for (int n = 0; n < 60000; ++n) {
        View v[2];
        const int shared = pick(1, 40);
        for (auto& w : v) {
            w.at = at(4096 + pick(0, 60));
            w.inner = pick(0, 9) ? pick(1, 6) : 0;
            for (auto& d : w.dim) {
                d.count = pick(0, 30) ? pick(1, 4) : 0;
                d.stride = pick(0, 2) ? pick(0, 30) : shared;
                if (!pick(0, 9)) d.stride = -d.stride;
            }
        }
        const auto a = bytes_of(v[0]), b = bytes_of(v[1]);
        bool want = false;
        for (int64_t x : a) want = want || b.count(x);
        (want ? yes : no)++;
        EXPECT(q4::meet(v[0], v[1]) == want);
        EXPECT(q4::meet(v[1], v[0]) == want);
    }
    EXPECT(yes > 5000 && no > 5000);
    // q, k and v as parts of one fused row of 12 heads of 64: 8, 2 and 2
    const int T = 1 << 20, D = 64, row = 12 * D;
    const View q = heads(1 << 20, row, D, T, 8, D), k = heads((1 << 20) + 8 * D * 2, row, D, T, 2, D);
    EXPECT(!q4::meet(q, k) && !q4::meet(k, q));
    EXPECT(q4::meet(heads((1 << 20) + D * 2, row, D, T, 8, D), k));
    EXPECT(q4::meet(q, q));
    EXPECT(!q4::meet(q, heads((1 << 20) + (int64_t)T * row * 2, row, D, T, 8, D)));
    // one token, whose stride is any
    EXPECT(!q4::meet(heads(4096, 7, D, 1, 8, D), heads(4096 + 8 * D * 2, 999, D, 1, 2, D)));
    // a cache whose layers are neighbours in a row of an arena; the same with another stride of the other side
    const View layer0{at(1 << 20), 2 * D, {{9000, 4 * 16 * D * 2}, {4, 16 * D * 2}, {4, D * 2}}};
    const View layer1{at((1 << 20) + 4 * D * 2), 2 * D, {{9000, 4 * 16 * D * 2}, {4, 16 * D * 2}, {4, D * 2}}};
    EXPECT(!q4::meet(layer0, layer1));
    EXPECT(!q4::meet(layer0, heads((1 << 20) + 4 * D * 2, 32 * D, D, 100, 8, D)));
    EXPECT(q4::meet(layer0, heads((1 << 20) + 4 * D * 2, 31 * D, D, 100, 8, D)));
    std::puts("ok");
    return 0;
}
