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
#else
#define PKV_SPLIT_FN inline
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

}  // namespace pkv
