// Whether two operands share memory, decided on the host from their rows' addresses.
#pragma once

#include <stdint.h>

#include <initializer_list>
#include <utility>

namespace la {

// B N rows of `row` bytes at p + b bs + n ts (strides in bytes).
struct Rows {
    const void* p;
    int64_t B, N, row, bs, ts;
};

// Rows of `values` elements of eb bytes, strides in elements.
inline Rows rows_of(const void* p, int64_t B, int64_t N, int64_t values, int64_t bs, int64_t ts, int64_t eb) {
    return {p, B, N, values * eb, bs * eb, ts * eb};
}
inline Rows block_of(const void* p, int64_t bytes) { return {p, 1, 1, bytes, 0, 0}; }

// Whether lo < b bs + n ts < hi for some 0 <= b < B, 0 <= n < N.
inline bool lands(int64_t B, int64_t bs, int64_t N, int64_t ts, int64_t lo, int64_t hi) {
    for (auto [count, stride] : {std::pair<int64_t, int64_t*>{B, &bs}, {N, &ts}})
        if (*stride < 0) {                       // counted from the other end
            lo -= (count - 1) * *stride, hi -= (count - 1) * *stride;
            *stride = -*stride;
        }
    if (B > N) std::swap(B, N), std::swap(bs, ts);
    for (int64_t b = 0; b < B; ++b, lo -= bs, hi -= bs) {
        if (hi <= 0) return false;
        const int64_t n = lo < 0 || ts == 0 ? 0 : lo / ts + 1;   // the first past lo
        if (n < N && lo < n * ts && n * ts < hi) return true;
    }
    return false;
}

// Whether rows of x and of y share a byte. Exact where the two have the same strides or one
// of them is a single range of memory; of other pairs that lie within one another, up to 2^16
// comparisons are made, and what they do not show counts as apart.
inline bool overlap(Rows x, Rows y) {
    for (Rows* r : {&x, &y}) {
        if (!r->p || r->B < 1 || r->N < 1 || r->row < 1) return false;
        if (r->bs == 0) r->B = 1;                // the same rows again
        if (r->ts == 0) r->N = 1;
        if (r->B == 1) r->bs = 0;
        if (r->N == 1) r->ts = 0;
    }
    auto low = [](const Rows& r) { return (r.bs < 0 ? (r.B - 1) * r.bs : 0) + (r.ts < 0 ? (r.N - 1) * r.ts : 0); };
    auto high = [](const Rows& r) { return (r.bs > 0 ? (r.B - 1) * r.bs : 0) + (r.ts > 0 ? (r.N - 1) * r.ts : 0) + r.row; };
    const int64_t d = (int64_t)(reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p));
    if (d + low(y) >= high(x) || low(x) >= d + high(y)) return false;
    // Rows that follow one another without a gap are one row.
    auto joined = [](Rows r) {
        for (int k = 0; k < 2; ++k) {
            if (r.B > 1 && r.bs == r.row) r.row *= r.B, r.B = 1, r.bs = 0;
            if (r.N > 1 && r.ts == r.row) r.row *= r.N, r.N = 1, r.ts = 0;
        }
        return r;
    };
    const Rows jx = joined(x), jy = joined(y);
    if (jy.B * jy.N == 1) return lands(jx.B, jx.bs, jx.N, jx.ts, d - jx.row, d + jy.row);
    if (jx.B * jx.N == 1) return lands(jy.B, jy.bs, jy.N, jy.ts, -d - jy.row, -d + jx.row);
    if (x.B == y.B && x.N == y.N && x.bs == y.bs && x.ts == y.ts) {
        const int64_t first = d - (x.B - 1) * x.bs - (x.N - 1) * x.ts;   // of the rows' distances
        return lands(2 * x.B - 1, x.bs, 2 * x.N - 1, x.ts, -y.row - first, x.row - first);
    }
    const int64_t each = jx.B < jx.N ? jx.B : jx.N;
    if (jy.B * jy.N > 65536 / each) return false;
    for (int64_t b = 0; b < jy.B; ++b)
        for (int64_t n = 0; n < jy.N; ++n) {
            const int64_t e = d + b * jy.bs + n * jy.ts;
            if (lands(jx.B, jx.bs, jx.N, jx.ts, e - jx.row, e + jy.row)) return true;
        }
    return false;
}

inline bool overlaps_any(const Rows& out, std::initializer_list<Rows> others) {
    for (const Rows& r : others)
        if (overlap(out, r)) return true;
    return false;
}

// The same rows: an output in its input's place.
inline bool same_rows(const Rows& x, const Rows& y) {
    return x.p == y.p && x.row == y.row && (x.B <= 1 || x.bs == y.bs) && (x.N <= 1 || x.ts == y.ts);
}

}  // namespace la
