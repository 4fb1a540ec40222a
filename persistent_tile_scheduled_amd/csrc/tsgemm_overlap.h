// Whether two matrices in memory share a byte: plain C++, for the argument checks
// of the C ABI.
#pragma once

#include <stdint.h>

#include <initializer_list>

namespace tsg {

struct Region {
    const void* at;        // NULL: not there
    int64_t rows, bytes;   // of a row
    int64_t pitch;         // bytes between rows' beginnings, >= bytes
};

typedef __int128 wide;  // a distance between rows has no bound of its own

inline wide address(const Region& r) { return (wide)reinterpret_cast<uintptr_t>(r.at); }
inline wide end_of(const Region& r) { return address(r) + (wide)(r.rows - 1) * r.pitch + r.bytes; }

// Does one of r's rows reach into [from, to)?
inline bool meets(const Region& r, wide from, wide to) {
    const wide past = from - address(r) - r.bytes, row = past < 0 ? 0 : past / r.pitch + 1;  // the first that ends after `from`
    return row < r.rows && address(r) + row * r.pitch < to;
}

// The first byte and the one after the last (or as far as addresses go).
struct Extent {
    uint64_t from, to;
};
inline Extent extent(const Region& r) {
    if (!r.at || r.rows <= 0 || r.bytes <= 0) return {~0ull, 0};
    const wide end = end_of(r);
    return {(uint64_t)reinterpret_cast<uintptr_t>(r.at), end >> 64 ? ~0ull : (uint64_t)end};
}

inline bool overlap(Region a, Region b) {
    if (!a.at || !b.at || a.rows <= 0 || b.rows <= 0 || a.bytes <= 0 || b.bytes <= 0) return false;
    for (Region* r : {&a, &b})
        if (r->rows == 1 || r->pitch == r->bytes) *r = {r->at, 1, r->rows * r->bytes, r->rows * r->bytes};
    if (a.rows > b.rows) {
        const Region t = a;
        a = b;
        b = t;
    }
    if (!meets(b, address(a), end_of(a)) || !meets(a, address(b), end_of(b))) return false;  // one between the other's rows
    if (a.rows == 1) return true;
    if (a.pitch == b.pitch) {
        // a's row i and b's row j lie d + (j - i) pitch apart: less than a row for
        // at most two values of j - i, those about -d / pitch
        const wide d = address(b) - address(a), t0 = -(d >= 0 ? (d + a.pitch - 1) / a.pitch : -(-d / a.pitch));
        for (wide t = t0; t <= t0 + 1; ++t) {
            const wide apart = d + t * a.pitch;
            if (t > -a.rows && t < b.rows && apart < a.bytes && -apart < b.bytes) return true;
        }
        return false;
    }
    for (int64_t i = 0; i < a.rows; ++i)  // rare: two distances between rows in one stretch of memory
        if (meets(b, address(a) + (wide)i * a.pitch, address(a) + (wide)i * a.pitch + a.bytes)) return true;
    return false;
}

}  // namespace tsg
