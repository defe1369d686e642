// How the 4-bit decode splits its list of NT subtiles over CTAs and their
// warps. Plain integer arithmetic, shared by the kernel and a host replay.
#pragma once

#if defined(__CUDACC__)
#define PKV_SPLIT_FN __host__ __device__ __forceinline__
#else
#define PKV_SPLIT_FN inline
#endif

namespace pkv {

constexpr int kQ4Warps = 16;

// CTAs with work, of C launched: at least a subtile a warp while there is more
// than one, so that a short list stays on few CTAs and is joined on chip.
PKV_SPLIT_FN int q4_active_ctas(int NT, int C) {
    const int most = NT / kQ4Warps;
    const int ct = most < C ? most : C;
    return NT == 0 ? 0 : ct < 1 ? 1 : ct;
}

// First subtile of CTA c of CT.
PKV_SPLIT_FN int q4_cta_cut(int c, int NT, int CT) {
    return (int)((long long)c * NT / CT);
}

// The CTA whose range holds subtile t.
PKV_SPLIT_FN int q4_owner(int t, int NT, int CT) {
    return (int)((((long long)t + 1) * CT - 1) / NT);
}

// First subtile of warp w in a CTA's range [A, Z), A < Z. The warps with work
// come first, each with at least one subtile.
PKV_SPLIT_FN int q4_warp_cut(int w, int A, int Z) {
    const int nw = Z - A < kQ4Warps ? Z - A : kQ4Warps;
    return A + (int)((long long)(w < nw ? w : nw) * (Z - A) / nw);
}

}  // namespace pkv
