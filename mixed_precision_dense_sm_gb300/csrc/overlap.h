// overlap.h -- whether two row-pitched matrices share memory.
#pragma once
#include <cstdint>

namespace gemm103 {

// `rows` rows of `bytes` bytes, the first at `at`, each `pitch` bytes (at least
// `bytes`) behind the one before.  Nothing where `at` is NULL.
struct Region {
    const void* at;
    int64_t rows, pitch, bytes;
};

namespace overlap_detail {
// Addresses are below 2^57: rows that lie beyond 2^61 are none (and no product here
// overflows).
inline Region bounded(Region r) {
    if (r.at == nullptr || r.rows <= 0 || r.bytes <= 0) return Region{nullptr, 0, 1, 0};
    if (r.rows > 1 && r.pitch == r.bytes && r.rows <= (int64_t{1} << 61) / r.bytes) r.bytes *= r.rows, r.rows = 1;
    if (r.rows > 1 && r.rows > (int64_t{1} << 61) / r.pitch) r.rows = (int64_t{1} << 61) / r.pitch;
    if (r.rows <= 1) r.rows = 1, r.pitch = r.bytes;
    return r;
}
inline int64_t address(const Region& r) { return static_cast<int64_t>(reinterpret_cast<uintptr_t>(r.at)); }
inline int64_t end(const Region& r) { return address(r) + (r.rows - 1) * r.pitch + r.bytes; }
}  // namespace overlap_detail

// Columns of one buffer, or every other row of it, are apart although the spans that
// they lie in are not: rows are looked at then, those of the one with fewer.
inline bool overlap(Region a, Region b) {
    using namespace overlap_detail;
    a = bounded(a), b = bounded(b);
    if (a.at == nullptr || b.at == nullptr || end(a) <= address(b) || end(b) <= address(a)) return false;
    if (a.pitch == b.pitch && a.rows > 1) {
        int64_t off = (address(b) - address(a)) % a.pitch;           // of b's rows behind a's
        if (off < 0) off += a.pitch;
        if (off >= a.bytes && off + b.bytes <= a.pitch) return false;
    }
    if (a.rows > b.rows) {
        const Region t = a;
        a = b, b = t;
    }
    const int64_t b0 = address(b);
    for (int64_t i = 0; i < a.rows; ++i) {
        const int64_t s = address(a) + i * a.pitch, e = s + a.bytes;
        // b's first row that ends behind s
        const int64_t j = s < b0 + b.bytes ? 0 : (s - b0 - b.bytes) / b.pitch + 1;
        if (j < b.rows && b0 + j * b.pitch < e) return true;
    }
    return false;
}

}  // namespace gemm103
