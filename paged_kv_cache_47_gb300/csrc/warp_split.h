// How a decode whose warps run alone splits its work over CTAs and their warps
// (W a CTA). Plain integer arithmetic, shared by the kernels and a host replay.
//
// The list: each unit (sequence, kv head, chunk of q heads) takes `cost` places
// and then one for each of its n subtiles, units end to end, NV places in all.
// CTAs and warps take even shares of the places, so a warp that starts more
// units gets fewer subtiles. Subtile i of a unit whose places begin at v has
// place v + cost + i; a cut among a unit's first places falls before its first
// subtile.
#pragma once

#if defined(__CUDACC__)
#define PKV_SPLIT_FN __host__ __device__ __forceinline__
#define PKV_SPLIT_WARP_FN __device__ __forceinline__       // given what a warp finds together
#else
#define PKV_SPLIT_FN inline
#define PKV_SPLIT_WARP_FN inline
#endif

namespace pkv {

// Where warps get fewer subtiles than this the time is that of one chain, and
// unit starts are not counted.
constexpr int kSplitFewSubtiles = 4;

// The cost to count units with, for NT subtiles on C CTAs.
PKV_SPLIT_FN int split_unit_cost(int NT, int C, int W, int cost) {
    return NT < C * W * kSplitFewSubtiles ? 0 : cost;
}

// Few units, none longer than this many subtiles: a CTA each, nothing to join
// between CTAs.
PKV_SPLIT_FN int split_one_cta(int W) { return 4 * W; }
PKV_SPLIT_FN bool split_units_alone(int cost, int units, int longest, int C, int W) {
    return cost == 0 && units <= C && longest <= split_one_cta(W);
}

// Of that form, the sequence of unit k of all (U a sequence that has tokens):
// nonempty[s] sequences before s have some, k < nonempty[S] * U.
template <typename T>
PKV_SPLIT_FN int split_unit_sequence(const T *nonempty, int S, int U, int k) {
    int lo = 0, hi = S - 1;                          // the last with at most k / U before it
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int)nonempty[mid] <= k / U) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// And its share of the places, [A, Z). prefix[s]: places before sequence s, for
// one unit a sequence.
PKV_SPLIT_FN void split_unit_share(const int *prefix, int s, int U, int k, int &A, int &Z) {
    const int n = prefix[s + 1] - prefix[s];
    A = prefix[s] * U + k % U * n;
    Z = A + n;
}

// CTAs with work, of C launched: a full CTA has a subtile for every warp (a
// share of cost + 1 places holds one).
PKV_SPLIT_FN int split_active_ctas(int NV, int C, int W, int cost) {
    const int most = NV / (W * (cost + 1));
    const int ct = most < C ? most : C;
    return NV == 0 ? 0 : ct < 1 ? 1 : ct;
}

// First place of CTA c of CT.
PKV_SPLIT_FN int split_cta_cut(int c, int NV, int CT) {
    return (int)((long long)c * NV / CT);
}

// The CTA whose share holds place v.
PKV_SPLIT_FN int split_owner(int v, int NV, int CT) {
    return (int)((((long long)v + 1) * CT - 1) / NV);
}

// First place of warp w in a CTA's share [A, Z), A < Z. The warps with work
// come first.
PKV_SPLIT_FN int split_warp_cut(int w, int A, int Z, int W, int cost) {
    const int fit = (Z - A) / (cost + 1);
    const int nw = fit < 1 ? 1 : fit < W ? fit : W;
    return A + (int)((long long)(w < nw ? w : nw) * (Z - A) / nw);
}

// A subtile's place: sequence, unit, subtile of the unit; places of a unit of
// the sequence; place of the unit's first subtile.
struct SplitPlace {
    int s, u, i, nv, tu;
};

// The last of S sequences whose units begin at or before place a (of equal
// prefixes, the empty sequences come first), 32 ways at a time:
// found(lo, n, step) of the places lo, lo + step, .. < lo + n, at most 32, begin
// there or before.
template <typename Found>
PKV_SPLIT_WARP_FN int split_sequence(int S, Found found) {
    int lo = 0;
    for (int n = S; n > 1;) {
        const int step = (n + 31) / 32, skip = (found(lo, n, step) - 1) * step;
        lo += skip;
        n = step < n - skip ? step : n - skip;
    }
    return lo;
}

// The first subtile at or after place a, which lies in sequence s.
PKV_SPLIT_FN SplitPlace split_place(const int *prefix, int s, int U, int a, int cost) {
    SplitPlace w;
    w.nv = prefix[s + 1] - prefix[s];
    const int r = a - prefix[s] * U;
    w.s = s;
    w.u = r / w.nv;
    w.tu = a - (r - w.u * w.nv) + cost;
    w.i = a > w.tu ? a - w.tu : 0;
    return w;
}

// The next unit, if its first subtile lies before place z. len: sequences' tokens.
PKV_SPLIT_FN bool split_next_unit(const int *prefix, const int *len, int U, SplitPlace &w, int z) {
    w.i = 0;
    w.tu += w.nv;
    if (w.tu >= z) return false;
    if (++w.u == U) {
        w.u = 0;
        do ++w.s; while (len[w.s] == 0);             // (there is one: the list goes on)
        w.nv = prefix[w.s + 1] - prefix[w.s];
    }
    return true;
}

}  // namespace pkv
