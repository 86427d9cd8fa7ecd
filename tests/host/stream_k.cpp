// Stream-K kernels that share a GPU all come to their end: blocks are started in
// order, each of them on an SM of its own, in any interleaving of two grids, and a
// tile's finisher waits on its SM for the other units of the tile.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "stream_k.h"

struct Grid {
    int tiles, KB, L, units;
    int started = 0, ended = 0;
    std::vector<int> stored;                     // sums of other units, per tile
    std::vector<std::vector<int>> left;          // per unit: its tiles still to do, last first
    Grid(int t, int k, int l) : tiles(t), KB(k), L(l), units(static_cast<int>((static_cast<int64_t>(t) * k + l - 1) / l)),
                                stored(t, 0), left(units) {
        for (int u = 0; u < units; ++u) {
            const int64_t b = static_cast<int64_t>(u) * L;
            int64_t e = b + L;
            if (e > static_cast<int64_t>(tiles) * KB) e = static_cast<int64_t>(tiles) * KB;
            for (int t = static_cast<int>((e - 1) / KB); t >= static_cast<int>(b / KB); --t) left[u].push_back(t);
        }
    }
    // One step of a unit; true where it moved.
    bool step(int u) {
        const int t = left[u].back();
        const int first = gemm103::stream_k_first(t, KB, L), last = gemm103::stream_k_last(t, KB, L);
        if (u < first || u > last) std::abort();
        if (u == first && stored[t] < last - first) return false;          // waits
        if (u != first) ++stored[t];
        left[u].pop_back();
        return true;
    }
};

int main() {
    std::mt19937 rng(7);
    auto pick = [&](int lo, int hi) { return static_cast<int>(lo + rng() % static_cast<unsigned>(hi - lo + 1)); };
    for (int round = 0; round < 4000; ++round) {
        const int sms = pick(1, 12);
        std::vector<Grid> g;
        for (int i = 0; i < 2; ++i) {
            const int tiles = pick(1, 10), KB = pick(1, 12);
            const int64_t work = static_cast<int64_t>(tiles) * KB;
            const int L = static_cast<int>((work + sms - 1) / sms);        // no more units than SMs
            g.emplace_back(tiles, KB, L);
        }
        std::vector<std::pair<int, int>> on;     // (grid, unit) on an SM
        for (;;) {
            while (static_cast<int>(on.size()) < sms) {
                int i = pick(0, 1);
                if (g[i].started == g[i].units) i ^= 1;
                if (g[i].started == g[i].units) break;
                on.push_back({i, gemm103::stream_k_unit(g[i].started++, g[i].units)});
            }
            if (on.empty()) break;
            bool moved = false;
            for (size_t k = 0; k < on.size();) {
                Grid& q = g[on[k].first];
                const int u = on[k].second;
                while (!q.left[u].empty() && q.step(u)) moved = true;
                if (q.left[u].empty()) {
                    ++q.ended;
                    on[k] = on.back();
                    on.pop_back();
                    moved = true;
                } else {
                    ++k;
                }
            }
            if (!moved) {
                std::printf("round %d: %d of %d and %d of %d units ended on %d SMs, the rest wait for ever\n", round,
                            g[0].ended, g[0].units, g[1].ended, g[1].units, sms);
                return 1;
            }
        }
        for (const Grid& q : g)
            if (q.ended != q.units) return 1;
    }
    return 0;
}
