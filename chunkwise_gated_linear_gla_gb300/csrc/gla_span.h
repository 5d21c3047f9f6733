// Host-side checks of tensors shared by the entry points: alignment, the bytes a tensor spans, overlap.
#pragma once

#include <cstddef>
#include <cstdint>
#include <utility>

namespace gla {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The bytes a strided [B,H,T,d] tensor spans (strides may be zero or negative).
struct Span { uintptr_t lo, hi; };
inline Span span(const void* p, const long long* st, int B, int H, int T, int d, size_t e)
{
    if (!p || B <= 0 || H <= 0 || T <= 0) return Span{0, 0};
    long long lo = 0, hi = d;
    const long long n[3] = {B - 1LL, H - 1LL, T - 1LL};
    for (int i = 0; i < 3; ++i) (st[i] < 0 ? lo : hi) += st[i] * n[i];
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a + (uintptr_t)(lo * (long long)e), a + (uintptr_t)(hi * (long long)e)};
}
inline Span flat(const void* p, size_t bytes)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return p ? Span{a, a + bytes} : Span{0, 0};
}
inline bool overlap(Span a, Span b) { return a.lo != a.hi && b.lo != b.hi && a.lo < b.hi && b.lo < a.hi; }

// Whether the rows of a strided output are apart: dimension by dimension, from the smallest
// stride, each steps past everything that the ones before it cover.
inline bool apart(const long long* st, int B, int H, int T, int d)
{
    long long n[3] = {B, H, T}, s[3];
    for (int i = 0; i < 3; ++i) s[i] = st[i] < 0 ? -st[i] : st[i];
    for (int i = 0; i < 2; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i]) { std::swap(s[i], s[j]); std::swap(n[i], n[j]); }
    long long cover = d;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        if (s[i] < cover) return false;
        cover += s[i] * (n[i] - 1);
    }
    return true;
}

}  // namespace gla
