"""Plain implementations, in numpy, of the step operators around the decode: device block
tables, rotary positions, the 4-bit cache and block selection. Test infrastructure only.

Values are computed in 64 bits from the formulas in include/pkv_tables.h, pkv_rope.h,
pkv_q4.h and pkv_sparse.h; where a header fixes a decision in fp32 (codes, scores), it is
taken in fp32 here too. Pool layouts are the library's.
"""
from __future__ import annotations

import math

import numpy as np

F32 = np.float32


# ------------------------------------------------------------------ device block tables
def tables_release(tab, lens, released, free, num_free, B):
    """(lens, free, num_free) after the release; None if the call is refused."""
    lens, free = lens.copy(), free.copy()
    held = [(-(-int(L) // B) if r else 0) for L, r in zip(lens, released)]
    if any(L < 0 or L > tab.shape[1] * B for L in lens) or not 0 <= num_free <= len(free):
        return None
    if num_free + sum(held) > len(free):
        return None
    for s, n in enumerate(held):
        for j in range(n):
            free[num_free] = tab[s, j]
            num_free += 1
        if released[s]:
            lens[s] = 0
    return lens, free, num_free


def tables_append(tab, lens, add, free, num_free, B, max_tokens):
    """(tab, lens, num_free, slots, positions, offsets); None if the call is refused."""
    tab, S = tab.copy(), len(lens)
    if any(L < 0 or a < 0 or int(L) + int(a) > tab.shape[1] * B for L, a in zip(lens, add)):
        return None
    need = sum(-(-(int(L) + int(a)) // B) - -(-int(L) // B) for L, a in zip(lens, add))
    if need > num_free or int(np.sum(add, dtype=np.int64)) > max_tokens or not 0 <= num_free <= len(free):
        return None
    slots, pos, offs = np.full(max_tokens, -1, np.int64), np.zeros(max_tokens, np.int32), [0]
    i = 0
    for s in range(S):
        for p in range(int(lens[s]), int(lens[s]) + int(add[s])):
            if p % B == 0:
                num_free -= 1
                tab[s, p // B] = free[num_free]
            slots[i], pos[i] = int(tab[s, p // B]) * B + p % B, p
            i += 1
        offs.append(i)
    return tab, lens + add, num_free, slots, pos, np.array(offs, np.int32)


# --------------------------------------------------------------------- rotary positions
def rope_frequencies(rotary_dim, base, scaling="none", factor=1.0, original_len=0, low_freq_factor=1.0,
                     high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0, attention_factor=0.0):
    """(radians a position of each pair, amplitude)."""
    if scaling == "base":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    out = []
    for i in range(rotary_dim // 2):
        w = base ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            w /= factor
        elif scaling == "bands":
            turns = original_len * w / (2 * math.pi)
            t = min(1.0, max(0.0, (turns - low_freq_factor) / (high_freq_factor - low_freq_factor)))
            w = t * w + (1 - t) * w / factor
        elif scaling == "yarn":
            dim = lambda r: rotary_dim * math.log(original_len / (2 * math.pi * r)) / (2 * math.log(base))  # noqa: E731
            lo, hi = max(0, math.floor(dim(beta_fast))), min(rotary_dim - 1, math.ceil(dim(beta_slow)))
            u = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            w = (1 - u) * w + u * w / factor
        out.append(w)
    amp = (attention_factor or 0.1 * math.log(max(1.0, factor)) + 1) if scaling == "yarn" else 1.0
    return np.array(out), amp


def axes_frequencies(sections, order, frequencies, base, **scaling):
    """(axis of each pair, radians a position of each pair, amplitude) of a rotary embedding over several axes."""
    axis, left = [], list(sections)
    a = 0
    while sum(left):
        while left[a] == 0:
            a = (a + 1) % len(left)
        axis.append(a)
        left[a] -= 1
        if order == "cycled":
            a = (a + 1) % len(left)
    w, amp = rope_frequencies(2 * len(axis), base, **scaling)
    if frequencies == "own":
        own = [rope_frequencies(2 * n, base, **scaling)[0] for n in sections]
        used = [0] * len(sections)
        for i, a in enumerate(axis):
            w[i] = own[a][used[a]]
            used[a] += 1
    return np.array(axis), w, amp


def rope(x, positions, w, amp, layout):
    """x [T][H][D] float64, turned; and, element by element, |x_a| + |x_b| of its pair."""
    y, size = x.copy(), np.abs(x)
    n = len(w)
    pos = positions.astype(np.float64)
    ang = (pos if pos.ndim == 2 else pos[:, None]) * w           # 2-D: a position for each pair
    c, s = (np.cos(ang) * amp)[:, None], (np.sin(ang) * amp)[:, None]
    a, b = ((slice(0, n), slice(n, 2 * n)) if layout == "half" else
            (slice(0, 2 * n, 2), slice(1, 2 * n, 2)))
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


# -------------------------------------------------------------------------- 4-bit cache
def q4_quantize(x):
    """x [..., D] fp32: codes [..., D] uint8, scales and minima [..., NG] fp16."""
    g = x.astype(F32).reshape(*x.shape[:-1], -1, 32)
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)
        m = np.clip(lo, F32(-65504), F32(65504)).astype(np.float16)
        s = np.minimum((hi - lo) * F32(1 / 15), F32(65504)).astype(np.float16)
        bad = ~np.isfinite(g).all(-1)
        m[bad] = s[bad] = np.nan
        c = np.clip(np.rint((g - m.astype(F32)[..., None]) / s.astype(F32)[..., None]), 0, 15)
        c = np.where(s.astype(F32)[..., None] > 0, c, 0)
    return np.nan_to_num(c).astype(np.uint8).reshape(x.shape), s, m


def _nibbles(D, rows):
    """Nibble of a row's bytes that holds each element."""
    d, n = np.arange(D), 8 if rows else 4
    return ((d % 32 // n) * (D // 32) + d // 32) * n + d % n


def q4_pack(codes, rows):
    D = codes.shape[-1]
    nib = np.zeros(codes.shape, np.uint8)
    nib[..., _nibbles(D, rows)] = codes
    return nib[..., 0::2] | nib[..., 1::2] << 4


def q4_unpack(packed, rows):
    nib = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)
    return nib[..., _nibbles(nib.shape[-1], rows)]


def q4_values(codes, s, m):
    """codes [..., D], s and m [..., NG]: values in 64 bits."""
    rep = lambda a: np.repeat(a.astype(np.float64), 32, -1)  # noqa: E731
    return codes * rep(s) + rep(m)


def q4_append(k, v, slots, kc, vc, kp, vp):
    """Write the rows into copies of the four pools, and return those."""
    kc, vc, kp, vp = (a.copy() for a in (kc, vc, kp, vp))
    B = kc.shape[2]
    for i, slot in enumerate(slots):
        if slot < 0:
            continue
        b, o = divmod(int(slot), B)
        for x, codes, params, rows in ((k, kc, kp, True), (v, vc, vp, False)):
            c, s, m = q4_quantize(x[i])
            codes[b, :, o] = q4_pack(c, rows)
            if rows:
                params[b, :, o] = np.concatenate([s, m], -1)
            else:
                params[b, :, :, o] = np.concatenate([s, m], -1)
    return kc, vc, kp, vp


def q4_rows(tab_row, L, kc, vc, kp, vp):
    """K and V values [Hk][L][D] of one sequence."""
    B, NG = kc.shape[2], kp.shape[3] // 2
    blk = tab_row[: -(-L // B)].astype(np.int64)
    out = []
    for codes, params, rows in ((kc[blk], kp[blk], True), (vc[blk], vp[blk].swapaxes(2, 3), False)):
        x = q4_values(q4_unpack(codes, rows), params[..., :NG], params[..., NG:])
        out.append(x.transpose(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[-1])[:, :L])
    return out


def attend(q, k, v, scale):
    """q [Hq][D], k and v [Hk][L][D], 64 bits: (out [Hq][D], log2 denominators, weights [Hq][L])."""
    G = q.shape[0] // k.shape[0]
    k, v = np.repeat(k, G, 0), np.repeat(v, G, 0)
    z = np.einsum("hd,hld->hl", q, k) * scale
    mx = z.max(-1, keepdims=True)
    p = np.exp(z - mx)
    den = p.sum(-1, keepdims=True)
    p = p / den
    return np.einsum("hl,hld->hd", p, v), ((mx + np.log(den)) / math.log(2))[:, 0], p


# --------------------------------------------------------------------- block selection
def block_mean(rows, to):
    """rows [..., B, D] fp32: their mean, added in order in fp32, rounded by `to`."""
    total = rows[..., 0, :].astype(F32)
    for t in range(1, rows.shape[-2]):
        total = (total + rows[..., t, :]).astype(F32)
    return to(total * F32(1.0 / rows.shape[-2]))


def block_scores(q, means):
    """q [G][D], means [n][D] fp32: [n] scores, fp32 in the defined order."""
    prod = (q[None] * means[:, None]).astype(F32)
    acc = prod[..., 0::8]
    for e in range(1, 8):
        acc = (acc + prod[..., e::8]).astype(F32)
    while acc.shape[-1] > 1:
        acc = (acc[..., 0::2] + acc[..., 1::2]).astype(F32)
    acc = acc[..., 0]
    return np.where(np.isnan(acc), F32(np.inf), acc).max(-1)


def select(score, n, top, first, last):
    """Ascending list of the blocks read, of n."""
    mid = [j for j in range(first, n - last)]
    best = sorted(mid, key=lambda j: (-float(score[j]), j))[:top] if len(mid) > top else mid
    return sorted(set(best) | {j for j in range(n) if j < first or j >= n - last})
