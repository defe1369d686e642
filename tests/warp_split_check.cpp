// Host replay of the split of a decode whose warps run alone (warp_split.h):
// random batches of units
// are cut over CTAs and warps as the kernels cut them; every subtile must be
// used once, every unit written once, and the pieces joined must be exactly
// the unit's.
#include <array>
#include <cstdio>
#include <map>
#include <random>
#include <set>
#include <vector>

#include "warp_split.h"

using namespace pkv;

struct Piece { int tu = 0, nu = 0, from = 0, to = 0; };

static bool run(const std::vector<int> &units, int C, int W, int cost) {
    int NV = 0;
    std::vector<int> start;                        // a unit's first place
    for (int n : units) { start.push_back(NV); NV += n + cost; }
    const int CT = split_active_ctas(NV, C, W, cost);
    if (CT > C || (NV > 0) != (CT > 0)) return false;
    std::map<int, int> covered, written;           // first subtile's place -> subtiles, outputs
    std::map<int, std::vector<std::pair<int, int>>> parts;   // -> (cta, side)
    std::map<int, int> part_subtiles, length;
    for (size_t u = 0; u < units.size(); ++u) length[start[u] + cost] = units[u];
    int expect = 0;
    for (int c = 0; c < CT; ++c) {
        const int A = split_cta_cut(c, NV, CT), Z = split_cta_cut(c + 1, NV, CT);
        if (A != expect || Z <= A) return false;
        expect = Z;
        std::vector<std::array<Piece, 2>> piece(W);
        int at = A;
        for (int w = 0; w < W; ++w) {
            const int a = split_warp_cut(w, A, Z, W, cost), z = split_warp_cut(w + 1, A, Z, W, cost);
            if (a != at || z < a) return false;
            if (w == 0 && z == a) return false;     // the first warp has work
            at = z;
            if (a == z) continue;
            size_t u = 0;
            while (u + 1 < units.size() && start[u + 1] <= a) ++u;
            int ci = a - start[u] - cost;
            if (ci < 0) ci = 0;
            int used = 0;
            while (u < units.size()) {
                const int tu = start[u] + cost, n = units[u];
                const int to = z - tu < n ? z - tu : n;
                if (to <= ci) {
                    if (ci < n) break;              // the share ends before the unit's first subtile
                    ci = 0;                         // (a share cannot begin past a unit's end)
                    return false;
                }
                for (int i = ci; i < to; ++i)
                    if (split_owner(tu + i, NV, CT) != c) return false;
                covered[tu] += to - ci;
                used += to - ci;
                if (ci == 0 && to == n) {
                    ++written[tu];
                } else {
                    Piece &p = piece[w][ci ? 0 : 1];
                    if (p.nu) return false;         // a place is used once
                    p = {tu, n, ci, to};
                }
                ci = 0;
                if (++u < units.size() && start[u] >= z) break;
            }
            if (used == 0) return false;
        }
        if (at != Z) return false;
        bool open[2] = {false, false};
        for (int w = 0; w < W; ++w)
            for (int sl = w == 0 ? 0 : 1; sl < 2; ++sl) {
                const Piece pc = piece[w][sl];
                if (!pc.nu) continue;
                int last = w, sum = pc.to - pc.from;
                while (last + 1 < W && piece[last + 1][0].nu && piece[last + 1][0].tu == pc.tu) {
                    ++last;
                    sum += piece[last][0].to - piece[last][0].from;
                }
                const bool done = pc.tu >= A && pc.tu + pc.nu <= Z;
                if (done) {
                    if (sum != pc.nu) return false;
                    ++written[pc.tu];
                } else {
                    const int side = pc.tu < A ? 0 : 1;
                    if (open[side]) return false;
                    open[side] = true;
                    parts[pc.tu].push_back({c, side});
                    part_subtiles[pc.tu] += sum;
                }
            }
    }
    if (expect != NV) return false;
    std::set<int> counters;
    for (auto &kv : parts) {
        const int tu = kv.first, nu = length[tu];
        const int first = split_owner(tu, NV, CT), n = split_owner(tu + nu - 1, NV, CT) - first + 1;
        if ((int)kv.second.size() != n || part_subtiles[tu] != nu) return false;
        if (!counters.insert(first).second) return false;        // a counter serves one unit
        for (int k = 0; k < n; ++k)
            if (kv.second[k].first != first + k || kv.second[k].second != (k == 0 ? 1 : 0)) return false;
        ++written[tu];
    }
    for (auto &kv : length)
        if (covered[kv.first] != kv.second || written[kv.first] != 1) return false;
    return true;
}

int main() {
    std::mt19937 rng(1);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    for (int i = 0; i < 4000; ++i) {
        std::vector<int> units(pick(1, 60));
        const int most = i % 4 == 0 ? 1 : i % 4 == 1 ? 5 : i % 4 == 2 ? 40 : 900;
        for (int &n : units) n = pick(1, most);
        const int C = i % 3 == 0 ? pick(1, 4) : i % 3 == 1 ? 152 : pick(1, 600);
        bool ok = true;
        for (int W : {8, 10, 12, 16})
            for (int cost : {0, 1, 2}) ok = ok && run(units, C, W, cost);
        if (!ok) {
            std::printf("FAIL at %d\n", i);
            return 1;
        }
    }
    std::puts("OK");
    return 0;
}
