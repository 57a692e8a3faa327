// Whether an output meets an input: views of strided memory.
#pragma once

#include <algorithm>
#include <cstdint>
#include <new>
#include <utility>
#include <vector>

namespace q4 {

// Memory that an argument takes: `inner` bytes at each of up to three counts of strides.
struct View {
    const void* at;
    int64_t inner;
    struct {
        int64_t count, stride;     // stride in bytes
    } dim[3];
};

namespace detail {

// A view as pieces: dimensions of more than one entry, longest stride first, those
// that run on into each other joined.
struct Pieces {
    int64_t at = 0, inner = 0, count[3], stride[3];
    int dims = 0;
    bool empty = false;

    explicit Pieces(const View& v) : at((int64_t) reinterpret_cast<uintptr_t>(v.at)), inner(v.inner)
    {
        if (inner <= 0) empty = true;
        for (const auto& d : v.dim) {
            if (d.count <= 0) empty = true;
            if (d.count <= 1 || d.stride == 0) continue;
            if (d.stride < 0) at += (d.count - 1) * d.stride;
            count[dims] = d.count;
            stride[dims++] = d.stride < 0 ? -d.stride : d.stride;
        }
        for (int i = 1; i < dims; ++i)
            for (int j = i; j > 0 && stride[j] > stride[j - 1]; --j) {
                std::swap(stride[j], stride[j - 1]);
                std::swap(count[j], count[j - 1]);
            }
        while (dims && stride[dims - 1] <= inner) {
            --dims;
            inner += (count[dims] - 1) * stride[dims];
        }
    }
    int64_t span() const
    {
        int64_t n = inner;
        for (int i = 0; i < dims; ++i) n += (count[i] - 1) * stride[i];
        return n;
    }
    Pieces without(int d) const
    {
        Pieces p = *this;
        for (int i = d; i + 1 < dims; ++i) {
            p.count[i] = count[i + 1];
            p.stride[i] = stride[i + 1];
        }
        --p.dims;
        return p;
    }
    int64_t number() const
    {
        int64_t n = 1;
        for (int i = 0; i < dims; ++i) n *= count[i];
        return n;
    }
    std::vector<int64_t> starts() const
    {
        std::vector<int64_t> s{at};
        for (int i = 0; i < dims; ++i) {
            const size_t n = s.size();
            for (int64_t c = 1; c < count[i]; ++c)
                for (size_t j = 0; j < n; ++j) s.push_back(s[j] + c * stride[i]);
        }
        std::sort(s.begin(), s.end());
        return s;
    }
};

constexpr int64_t kMostPieces = 1 << 20;

inline bool meet(const Pieces& a, const Pieces& b)
{
    if (a.at >= b.at + b.span() || b.at >= a.at + a.span()) return false;
    if (!a.dims && !b.dims) return true;
    // A stride that both have, and that holds what is below it of each: apart
    // if one period of each is, wherever the other's lies against it (views of one
    // wider row; nothing is counted out).
    for (int i = 0; i < a.dims; ++i)
        for (int j = 0; j < b.dims; ++j) {
            const int64_t s = a.stride[i];
            Pieces x = a.without(i), y = b.without(j);
            if (s != b.stride[j] || x.span() > s || y.span() > s) continue;
            const int64_t d = ((y.at - x.at) % s + s) % s;
            y.at = x.at + d;
            if (meet(x, y)) continue;
            y.at -= s;
            if (!meet(x, y)) return false;
        }
    const int64_t na = a.number(), nb = b.number();
    if (na > kMostPieces || nb > kMostPieces) return true;
    const std::vector<int64_t> p = a.starts(), q = b.starts();
    for (size_t i = 0, j = 0; i < p.size() && j < q.size();) {
        if (p[i] + a.inner <= q[j]) ++i;
        else if (q[j] + b.inner <= p[i]) ++j;
        else return true;
    }
    return false;
}

}  // namespace detail

// Whether two views have a byte in common. Exact, but for views of more than 2^20
// pieces whose strides have nothing in common: those meet if their ranges do.
inline bool meet(const View& a, const View& b)
{
    // (mostly their ranges do not meet: seen without taking them apart)
    int64_t from[2], to[2];
    for (int i = 0; i < 2; ++i) {
        const View& v = i ? b : a;
        from[i] = (int64_t) reinterpret_cast<uintptr_t>(v.at);
        to[i] = from[i] + v.inner;
        for (const auto& d : v.dim) (d.stride < 0 ? from[i] : to[i]) += (d.count - 1) * d.stride;
    }
    if (from[0] >= to[1] || from[1] >= to[0]) return false;
    const detail::Pieces p(a), q(b);
    if (p.empty || q.empty) return false;
    try {
        return detail::meet(p, q);
    } catch (const std::bad_alloc&) {
        return true;
    }
}

}  // namespace q4
