// Whether strided tensors share memory: for the checks that an output meets no
// input.  Host code without CUDA.  Internal to the library.
#pragma once

#include <cstdint>

namespace kv {

// Rows and heads of `bytes` bytes each, `row` and `head` bytes apart (>= 0).
struct Strided {
    const void *at;
    int64_t rows, row, heads, head, bytes;
};

namespace strided {

using Wide = __int128;  // 2^31 rows of 2^42 bytes

// an axis of one element, or expanded, is none
inline Strided plain(Strided a) {
    if (a.rows == 1 || a.row == 0) a.rows = 1, a.row = 0;
    if (a.heads == 1 || a.head == 0) a.heads = 1, a.head = 0;
    return a;
}
inline bool none(const Strided &a) { return a.rows <= 0 || a.heads <= 0 || a.bytes <= 0; }
// bytes from the first to the last
inline Wide reach(const Strided &a) { return static_cast<Wide>(a.rows - 1) * a.row + static_cast<Wide>(a.heads - 1) * a.head + a.bytes; }

// Whether D + t S lies strictly between -below and above for a t of lo .. hi (S >= 0).
template <typename T>
bool hits(T D, T S, T lo, T hi, T below, T above) {
    if (S == 0) return lo <= 0 && 0 <= hi && -below < D && D < above;
    const T x = -below - D;  // the least t with t S > x
    T t = (x >= 0 ? x / S : -((-x + S - 1) / S)) + 1;
    if (t < lo) t = lo;
    return t <= hi && D + t * S < above;
}

// b begins `from` bytes behind a
template <typename T>
bool meet(const Strided &a, const Strided &b, T from) {
    const T S = a.row != 0 ? a.row : b.row, lo = -(a.rows - 1), hi = b.rows - 1;
    if (a.head == b.head || a.head == 0 || b.head == 0) {  // pairs of heads by their distance
        const T step = a.head != 0 ? a.head : b.head;
        for (int64_t d = 1 - a.heads; d < b.heads; ++d)
            if (hits<T>(from + d * step, S, lo, hi, b.bytes, a.bytes)) return true;
        return false;
    }
    if (a.heads * b.heads > 65536) return true;
    for (int64_t i = 0; i < a.heads; ++i)
        for (int64_t j = 0; j < b.heads; ++j)
            if (hits<T>(from + static_cast<T>(j) * b.head - static_cast<T>(i) * a.head, S, lo, hi, b.bytes, a.bytes)) return true;
    return false;
}

}  // namespace strided

// Whether two share a byte.  Exact where their rows are equally far apart, one of them has one row, or the memory from the
// first byte to the last is apart; true for others, which cannot be told apart in a short time.
inline bool meet(Strided a, Strided b) {
    using namespace strided;
    if (none(a) || none(b)) return false;
    a = plain(a);
    b = plain(b);
    const Wide from = static_cast<Wide>(reinterpret_cast<uintptr_t>(b.at)) - static_cast<Wide>(reinterpret_cast<uintptr_t>(a.at));
    const Wide ra = reach(a), rb = reach(b);
    if (from >= ra || -from >= rb) return false;
    if (a.row != 0 && b.row != 0 && a.row != b.row) return true;
    if (ra < (static_cast<Wide>(1) << 60) && rb < (static_cast<Wide>(1) << 60))  // (divisions of 64 bits are quicker)
        return strided::meet<int64_t>(a, b, static_cast<int64_t>(from));
    return strided::meet<Wide>(a, b, from);
}

// Whether two rows or heads of one share a byte.
inline bool folds(const Strided &a) {
    using namespace strided;
    if (none(a)) return false;
    const Wide S = a.rows > 1 ? a.row : 0, T = a.heads > 1 ? a.head : 0, most = a.rows - 1;
    if (a.rows > 1 && S < a.bytes) return true;
    if (a.heads == 1) return false;
    // a row's heads side by side, or a head's rows
    if (T >= a.bytes && (a.rows == 1 || S >= (a.heads - 1) * T + a.bytes || T >= most * S + a.bytes)) return false;
    for (int64_t d = 1; d < a.heads; ++d)
        if (hits<Wide>(d * T, S, -most, most, a.bytes, a.bytes)) return true;
    return false;
}

}  // namespace kv
