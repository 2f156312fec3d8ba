// Host-side checks shared by the C ABI's entry points.  Nothing here touches
// device memory.
#pragma once

#include <stdint.h>
#include <string.h>
#include <initializer_list>
#include <utility>
#include <hip/hip_runtime_api.h>

#include "sconv.h"

namespace sconv {

// Byte range [lo, hi) covered by a strided bf16 tensor; empty when a size is 0.
struct Span {
    uintptr_t lo = 0, hi = 0;
    bool empty() const { return hi <= lo; }
};

inline Span span_of(const void *p, std::initializer_list<int64_t> sizes,
             std::initializer_list<int64_t> strides, int64_t elem = 2) {
    Span s;
    if (!p) return s;
    int64_t last = 0;
    auto st = strides.begin();
    for (int64_t n : sizes) {
        if (n <= 0) return s;
        last += (n - 1) * *st++;
    }
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + uintptr_t((last + 1) * elem);
    return s;
}

inline bool overlap(const Span &a, const Span &b) {
    return !a.empty() && !b.empty() && a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// No two elements of a strided tensor share an address: taken in order of
// stride, every dimension of size > 1 steps past the whole span of the
// smaller ones.  Outputs and written caches must pass (their elements are
// written by different lanes); inputs may be any view, broadcasts included.
inline bool non_overlapping(std::initializer_list<int64_t> sizes, std::initializer_list<int64_t> strides) {
    int64_t n[4], st[4];
    int k = 0;
    auto sp = strides.begin();
    for (int64_t s : sizes) {
        const int64_t d = *sp++;
        if (s <= 1) continue;
        int i = k++;
        for (; i > 0 && st[i - 1] > d; --i) { n[i] = n[i - 1]; st[i] = st[i - 1]; }
        n[i] = s;
        st[i] = d;
    }
    int64_t span = 1;          // one past the largest offset of the dimensions so far
    for (int i = 0; i < k; ++i) {
        if (st[i] < span) return false;
        span += st[i] * (n[i] - 1);
    }
    return true;
}

inline bool negative(std::initializer_list<int64_t> v) {
    for (int64_t x : v)
        if (x < 0) return true;
    return false;
}

// Every stride a multiple of n elements (dimensions of one element aside) and
// the base aligned to n elements of `elem` bytes.
inline bool groups_of(const void *p, int n, int elem, std::initializer_list<int64_t> sizes,
                      std::initializer_list<int64_t> strides) {
    auto st = strides.begin();
    for (int64_t s : sizes) {
        const int64_t d = *st++;
        if (s > 1 && d % n) return false;
    }
    return aligned(p, uintptr_t(n) * uintptr_t(elem));
}

// The word that holds an argument, as that argument.
template <class A>
A from_word(const unsigned char *w) {
    static_assert(sizeof(A) == 4 || sizeof(A) == 8, "an argument fits a word");
    A a;                               // (little endian: a shorter one is the low half)
    memcpy(&a, w, sizeof(A));
    return a;
}
template <class... A, size_t... I>
int call_words(int (*f)(A...), const unsigned char *w, std::index_sequence<I...>) {
    return f(from_word<A>(w + 8 * I)...);
}
template <class... A>
int call_words(int (*f)(A...), const void *words) {
    if (!words) return SCONV_ERR_NULL;
    return call_words(f, static_cast<const unsigned char *>(words), std::index_sequence_for<A...>{});
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? SCONV_OK : SCONV_ERR_LAUNCH; }

}  // namespace sconv
