// rn_boxes.h -- what memory a strided tensor of rows covers, and whether two of them
// share any (plain C++: the host tests compile it by itself).
#pragma once

#include <cstdint>

namespace rn {

constexpr int64_t kMaxElems = (int64_t)1 << 61;

// Runs of `run` bytes at every combination of three strides (bytes). Empty where a count is 0.
struct Box {
    const void* p;
    int64_t count[3], stride[3], run;
};
inline Box flat(const void* p, int64_t bytes) { return {p, {1, 1, 1}, {0, 0, 0}, bytes}; }
inline bool empty(const Box& b) {
    return !b.p || b.run <= 0 || b.count[0] <= 0 || b.count[1] <= 0 || b.count[2] <= 0;
}
inline int64_t extent(const Box& b) {
    int64_t n = b.run;
    for (int i = 0; i < 3; ++i) n += (b.count[i] - 1) * b.stride[i];
    return n;
}
// Whether the box's last byte is within the element limit (its strides are >= 0).
inline bool fits(const Box& b) {
    int64_t n = b.run;
    for (int i = 0; i < 3; ++i) {
        int64_t m;
        if (b.stride[i] < 0) return false;
        if (b.count[i] <= 1) continue;
        if (__builtin_mul_overflow(b.count[i] - 1, b.stride[i], &m) || m > kMaxElems ||
            (n += m) > kMaxElems)
            return false;
    }
    return true;
}
// Whether no two of the box's runs share a byte, for strides that nest (each at least the
// extent of the smaller ones).
inline bool runs_apart(const Box& b) {
    int order[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (b.stride[order[j]] > b.stride[order[j + 1]]) {
                const int t = order[j];
                order[j] = order[j + 1];
                order[j + 1] = t;
            }
    int64_t n = b.run;
    for (int k : order) {
        if (b.count[k] <= 1) continue;
        if (b.stride[k] < n) return false;
        n += (b.count[k] - 1) * b.stride[k];
    }
    return true;
}
// Whether two boxes are shown to share no byte: by their ranges, or, as column blocks of one
// matrix, by where they lie within a stride m that both have: strides that are multiples of m
// change nothing there, and the rest of each box must be a part of one m.
inline bool apart(const Box& a, const Box& b) {
    if (empty(a) || empty(b)) return true;
    const uintptr_t pa = (uintptr_t)a.p, pb = (uintptr_t)b.p;
    if (pa + (uintptr_t)extent(a) <= pb || pb + (uintptr_t)extent(b) <= pa) return true;
    for (int i = 0; i < 3; ++i) {
        if (a.count[i] <= 1 || a.stride[i] <= 0) continue;
        const int64_t m = a.stride[i];
        int64_t ea = a.run, eb = b.run;
        for (int k = 0; k < 3; ++k) {
            if (a.count[k] > 1 && a.stride[k] % m) ea += (a.count[k] - 1) * a.stride[k];
            if (b.count[k] > 1 && b.stride[k] % m) eb += (b.count[k] - 1) * b.stride[k];
        }
        if (ea > m || eb > m) continue;
        const int64_t ra = (int64_t)(pa % (uintptr_t)m), rb = (int64_t)(pb % (uintptr_t)m);
        const int64_t ab = rb >= ra ? rb - ra : rb - ra + m;   // from a's place on to b's
        const int64_t ba = ab == 0 ? 0 : m - ab;
        if (ab >= ea && ba >= eb) return true;
    }
    return false;
}
template <int NO, int NI>
bool aliased(const Box (&outs)[NO], const Box (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        if (!empty(outs[i]) && !runs_apart(outs[i])) return true;
        for (int j = 0; j < NI; ++j)
            if (!apart(outs[i], ins[j])) return true;
        for (int j = i + 1; j < NO; ++j)
            if (!apart(outs[i], outs[j])) return true;
    }
    return false;
}

}  // namespace rn
