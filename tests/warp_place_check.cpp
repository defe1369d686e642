// Host replay of how a decode whose warps run alone finds its work (warp_split.h): from the
// sequences' lengths, empty ones among them, through the form and the cost that the kernel
// chooses, to each warp's subtiles. Every subtile of every unit is used once; where units
// have a CTA each, a unit lies in its own.
#include <cstdint>
#include <cstdio>
#include <random>
#include <vector>

#include "warp_split.h"

using namespace pkv;

static int alone_seen = 0, even_seen = 0;

static bool run(const std::vector<int> &len, int U, int C, int W, int sub, int unit_cost) {
    const int S = (int)len.size();
    int total = 0, longest = 0;
    for (int L : len) {
        const int n = (L + sub - 1) / sub;
        total += n;
        if (n > longest) longest = n;
    }
    const int cost = split_unit_cost(total * U, C, W, unit_cost);
    std::vector<int> prefix(S + 1, 0);
    std::vector<uint16_t> nonempty(S + 1, 0);
    for (int s = 0; s < S; ++s) {
        prefix[s + 1] = prefix[s] + (len[s] ? (len[s] + sub - 1) / sub + cost : 0);
        nonempty[s + 1] = (uint16_t)(nonempty[s] + (len[s] > 0));
    }
    const int units = nonempty[S] * U, NV = prefix[S] * U;
    const bool alone = split_units_alone(cost, units, longest, C, W);
    const int CT = alone ? units : split_active_ctas(NV, C, W, cost);
    if (CT > C || (total > 0) != (CT > 0)) return false;
    (alone ? alone_seen : even_seen)++;
    std::vector<std::vector<int>> used(S * U);
    for (int s = 0; s < S; ++s)
        for (int u = 0; u < U; ++u) used[s * U + u].assign((len[s] + sub - 1) / sub, 0);
    for (int c = 0; c < CT; ++c) {
        int A, Z;
        if (alone) {
            const int s = split_unit_sequence(nonempty.data(), S, U, c);
            if (s < 0 || s >= S || len[s] == 0) return false;
            split_unit_share(prefix.data(), s, U, c, A, Z);
        } else {
            A = split_cta_cut(c, NV, CT);
            Z = split_cta_cut(c + 1, NV, CT);
        }
        if (A < 0 || Z > NV || A >= Z) return false;
        int own = -1;
        for (int w = 0; w < W; ++w) {
            const int a = split_warp_cut(w, A, Z, W, cost), z = split_warp_cut(w + 1, A, Z, W, cost);
            if (a >= z) continue;
            const int first = split_sequence(S, [&](int lo, int n, int step) {
                int k = 0;
                for (int lane = 0; lane < 32; ++lane)
                    if (lane * step < n) k += prefix.at(lo + lane * step) * U <= a;
                return k;
            });
            if (first < 0 || first >= S || len[first] == 0) return false;
            SplitPlace at = split_place(prefix.data(), first, U, a, cost);
            for (;;) {
                if (at.s < 0 || at.s >= S || at.u < 0 || at.u >= U) return false;
                const int n = at.nv - cost;
                if (n != (int)used[at.s * U + at.u].size()) return false;
                if (at.tu != prefix[at.s] * U + at.u * at.nv + cost) return false;
                const int count = (n < z - at.tu ? n : z - at.tu) - at.i;
                if (count <= 0) break;
                if (alone && own >= 0 && own != at.s * U + at.u) return false;
                own = at.s * U + at.u;
                for (int i = at.i; i < at.i + count; ++i) ++used[own].at(i);
                if (!split_next_unit(prefix.data(), len.data(), U, at, z)) break;
            }
        }
        if (alone && own < 0) return false;
    }
    for (auto &u : used)
        for (int k : u)
            if (k != 1) return false;
    return true;
}

int main() {
    std::mt19937 rng(2);
    auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    int at = 0;
    auto check = [&](const std::vector<int> &len, int U, int C) {
        ++at;
        for (int W : {10, 16})
            for (int sub : {16, 32})
                if (!run(len, U, C, W, sub, 2)) {
                    std::printf("FAIL at %d: %d sequences, %d units each, %d CTAs, %d warps, subtiles of %d\n", at,
                                (int)len.size(), U, C, W, sub);
                    return false;
                }
        return true;
    };
    // units at, one below and one past the CTAs; lengths at and one past a CTA's own
    for (int C : {1, 2, 7, 152, 600})
        for (int U : {1, 2, 8})
            for (int d : {-1, 0, 1})
                for (int W : {10, 16})
                    for (int sub : {16, 32})
                        for (int more : {-1, 0, 1}) {
                            const int S = (C + d * U + U - 1) / U;
                            if (S < 1) continue;
                            std::vector<int> len(S, 5);
                            len[S / 2] = split_one_cta(W) * sub + more;
                            if (!check(len, U, C)) return 1;
                            len.insert(len.begin(), 0);
                            len.push_back(0);
                            if (!check(len, U, C)) return 1;
                        }
    for (int i = 0; i < 3000; ++i) {
        std::vector<int> len(i % 5 == 0 ? pick(900, 2048) : pick(1, 70));
        const int most = i % 4 == 0 ? 3 : i % 4 == 1 ? 100 : i % 4 == 2 ? 700 : 30000;
        const int empty = i % 3 == 0 ? 0 : i % 3 == 1 ? 30 : 95;         // in a hundred
        for (int &L : len) L = pick(1, 100) <= empty ? 0 : pick(0, most);
        if (!check(len, i % 7 == 0 ? pick(9, 40) : pick(1, 8), i % 3 == 0 ? 152 : pick(1, 600))) return 1;
    }
    if (alone_seen < 1000 || even_seen < 1000) return 1;
    std::puts("OK");
    return 0;
}
