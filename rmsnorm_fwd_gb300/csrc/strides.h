// strides.h -- host-side tests for overlapping strided layouts.
#pragma once

#include <algorithm>
#include <cstdint>

namespace rmsnorm {

inline bool bytes_overlap(uintptr_t a, int64_t abytes, uintptr_t b, int64_t bbytes)
{
    return a < b + static_cast<uintptr_t>(bbytes) && b < a + static_cast<uintptr_t>(abytes);
}

inline int64_t floor_div(int64_t x, int64_t y)
{
    return x >= 0 ? x / y : -((-x + y - 1) / y);
}

// Whether two strided sets can share a byte: set A is {a + t * sa + [0, la)}
// and set B {b + t * sb + [0, lb)}, t < n (bytes).  Exact for equal strides;
// sets that interleave with different strides count as overlapping.
inline bool strided_overlap(uintptr_t a, int64_t sa, int64_t la, uintptr_t b, int64_t sb,
                            int64_t lb, int64_t n)
{
    if (n <= 0 || la <= 0 || lb <= 0)
        return false;
    const int64_t ea = (n - 1) * sa + la, eb = (n - 1) * sb + lb;
    if (!bytes_overlap(a, ea, b, eb))
        return false; // the whole extents are apart
    if (sa != sb || sa <= 0)
        return true; // interleaved with different strides: refuse
    // Equal strides P: some pair collides iff d + m P lies in (-lb, la) for
    // an integer |m| < n, with d = b - a.
    const int64_t d = static_cast<int64_t>(b - a), P = sa;
    int64_t m_lo = floor_div(-lb - d, P) + 1;    // smallest m with d + mP > -lb
    int64_t m_hi = -floor_div(-(la - d), P) - 1; // largest m with d + mP < la
    m_lo = std::max(m_lo, -(n - 1));
    m_hi = std::min(m_hi, n - 1);
    return m_lo <= m_hi;
}

// Whether the interval [w, w + wb) meets {a + t * P + [0, la)}, t < n.
inline bool interval_hits_strided(uintptr_t a, int64_t P, int64_t la, int64_t n, uintptr_t w,
                                  int64_t wb)
{
    if (n <= 0 || la <= 0 || wb <= 0)
        return false;
    const int64_t d = static_cast<int64_t>(w - a);
    if (P <= 0) // a single interval
        return d < la && -d < wb;
    // t P < d + wb and d < t P + la, for an integer t in [0, n)
    int64_t t_lo = floor_div(d - la, P) + 1;     // smallest t with t P > d - la
    int64_t t_hi = -floor_div(-(d + wb), P) - 1; // largest t with t P < d + wb
    t_lo = std::max<int64_t>(t_lo, 0);
    t_hi = std::min<int64_t>(t_hi, n - 1);
    return t_lo <= t_hi;
}

} // namespace rmsnorm
