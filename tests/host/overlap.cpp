// Whether two pitched matrices share a byte, against a map of the bytes.
#include <cstdio>
#include <random>
#include <vector>

#include "overlap.h"

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

using gemm103::Region;
using gemm103::overlap;

static Region at(int64_t a, int64_t rows, int64_t pitch, int64_t bytes) {
    return Region{reinterpret_cast<const void*>(static_cast<uintptr_t>(a)), rows, pitch, bytes};
}

int main() {
    std::mt19937 rng(7);
    auto pick = [&](int lo, int hi) { return static_cast<int64_t>(rng() % (hi - lo + 1) + lo); };
    int met = 0, apart = 0;
    for (int n = 0; n < 200000; ++n) {
        Region r[2];
        std::vector<char> used(1200, 0);
        bool want = false;
        for (int k = 0; k < 2; ++k) {
            const int64_t bytes = pick(0, 9), pitch = bytes + (n % 3 == 0 ? 12 - bytes : pick(0, 12));
            r[k] = at(pick(100, 200), pick(0, 12), pitch < 1 ? 1 : pitch, bytes);
            for (int64_t i = 0; i < r[k].rows; ++i)
                for (int64_t j = 0; j < r[k].bytes; ++j) {
                    char& u = used[reinterpret_cast<uintptr_t>(r[k].at) + i * r[k].pitch + j];
                    if (k == 1 && u) want = true;
                    if (k == 0) u = 1;
                }
        }
        CHECK(overlap(r[0], r[1]) == want && overlap(r[1], r[0]) == want);
        (want ? met : apart) += 1;
    }
    CHECK(met > 20000 && apart > 20000);
    // NULL and empty
    CHECK(!overlap(at(0, 5, 8, 8), at(0, 5, 8, 8)) && !overlap(at(64, 0, 8, 8), at(64, 5, 8, 8)));
    // columns of one buffer, of the most rows; their padding; every other row
    const int64_t big = int64_t{1} << 30;
    CHECK(!overlap(at(4096, big, 64, 32), at(4096 + 32, big, 64, 32)));
    CHECK(overlap(at(4096, big, 64, 33), at(4096 + 32, big, 64, 32)));
    CHECK(!overlap(at(4096, 1000, 128, 64), at(4096 + 64, 1000, 128, 64)));
    // pitches whose products pass 64 bits
    const int64_t wide = int64_t{1} << 42;
    CHECK(overlap(at(4096, big, wide, 64), at(4096 + 63, 3, 64, 64)));
    CHECK(!overlap(at(4096, big, wide, 64), at(4096 + 64, 3, 64, 64)));
    CHECK(overlap(at(4096, big, wide, 64), at(4096, big, wide, 64)));
    CHECK(!overlap(at(4096, big, wide, 64), at(4096 + 64, big, wide, 64)));
    // the end of the address space is not passed
    CHECK(!overlap(at((int64_t{1} << 57) - 64, 1, 64, 64), at(4096, 1, 64, 64)));
    return 0;
}
