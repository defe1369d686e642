"""How near the 4-bit decode comes to 64 bits where operands of fewer bits would show: queries with a
few large channels, weights far below the largest, V scales from 1e-7 to thousands side by side.

Tolerances. A score is off by
  - the sums of D exact products and NG scaled partial sums in fp32, below (D / 8 + 8) 2^-23 of
    A = |scale| sum |q| (|s c| + |m|) for any order within the matrix instructions;
  - the operands: an element of q by at most 2^-35 of the head's largest, a group's sum of q (a pair
    of fp16) by 2^-22 of itself, which the first term's constant covers, and 2^-34 of the largest
    element: 2^-33 |scale| max|q| sum (|s c| + |m|) for both.
A weight's exponent is the score z in log2 units times a constant rounded twice, less the reference,
at most three roundings more: 2^-21 |z|, and the exponential 2^-21. The joins' weights have the
same from the denominators' logarithms. A weight is kept to 2^-22, at least to 2^-25 where
the largest is at 2^10 or above: 2^-35 of the largest. A weight times a V scale is kept to 2^-20, at
least to 2^-24 of the unit that the group's largest scale S (in half or more of it) has:
2 S 2^-34 of the largest weight, 15 times that for a code; scales of less than 2^-14 S to 2^-24 S.
Sums over tokens: a warp adds its own, two products for 16 of them, and up to 64 additions join the
warps' pieces: (n / 8 + 64) 2^-23 of sum p (|s c| + |m|) for n tokens a warp, for the denominator the
same of itself. Then half a step of the output's type."""
import math

import numpy as np
import pytest
import torch

from oracle import step_ops as O
from paged_kv_cache_47_gb300 import binding as b
from test_gpu_q4 import Batch, DT, dev, randn

pytestmark = pytest.mark.gpu


def sizes(t, s):
    """|s c| + |m| of sequence s's K and V elements at most, and the V scales' largest: [Hk][L][D] twice, [Hk][D]."""
    NG, L = t.D // 32, int(t.lens[s])
    blk = t.tab[s, : -(-L // t.B)].astype(np.int64)
    size, top = [], None
    for par in (t.kp[blk], t.vp[blk].swapaxes(2, 3)):
        par = par.transpose(1, 0, 2, 3).reshape(t.Hk, -1, 2 * NG)[:, :L].astype(np.float64)
        size.append(np.repeat(15 * np.abs(par[..., :NG]) + np.abs(par[..., NG:]), 32, -1))
        top = np.repeat(np.abs(par[..., :NG]).max(1), 32, -1)
    return size[0], size[1], top


def score_error(t, q, size, scale):
    """Of one sequence, [Hq][L]; q [Hq][D] in 64 bits."""
    size = np.repeat(size, q.shape[0] // t.Hk, 0)
    a = np.einsum("hd,hld->hl", np.abs(q), size) * (t.D / 8 + 8) * 2.0 ** -23
    return abs(scale) * (a + size.sum(-1) * np.abs(q).max(-1)[:, None] * 2.0 ** -33)


def check(t, q, scale, **kw):
    """q [S][Hq][D], CPU. Output in fp32 and denominators within the tolerances above."""
    S, Hq, _ = q.shape
    G = Hq // t.Hk
    lse = torch.full((S, Hq), 7.0, device="cuda")
    out = b.decode_attention_q4(q.cuda(), t.cache, dev(t.tab), dev(t.lens), scale, out_dtype=torch.float32, lse_out=lse, **kw)
    assert b.get_error() == 0
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    # tokens a warp has of one context: an even share of all subtiles of 32, a unit's start counted as two
    warps = 16 * (kw.get("num_ctas") or torch.cuda.get_device_properties(0).multi_processor_count)
    units = t.Hk * -(-G // 8)
    share = 32 * (-(-int(sum(-(-int(n) // 32) + 2 for n in t.lens)) * units // warps) + 1)
    if kw.get("num_ctas", 0) == 0:
        share = max(share, 4 * 32)                   # few short units: a CTA each
    for s in range(S):
        L = int(t.lens[s])
        k, v = O.q4_rows(t.tab[s], L, t.kc, t.vc, t.kp, t.vp)
        qs = q[s].double().numpy()
        want, wl, p = O.attend(qs, k, v, scale)
        ks, vs, top = sizes(t, s)
        z = np.abs(wl)[:, None] + np.abs(np.log2(np.maximum(p, 1e-300)))    # |log2 units| of a score, at most
        weight = score_error(t, qs, ks, scale) + (z + 1) * 2.0 ** -21 + 2.0 ** -22
        sums = (min(L, share) / 8 + 64) * 2.0 ** -23
        vs, top, v = (np.repeat(x, G, 0) for x in (vs, top, v))
        tol = np.zeros_like(want)
        for h in range(Hq):
            move = np.abs(v[h] - want[h])
            tol[h] = 2 * (p[h] * weight[h]) @ move + (p[h] @ vs[h]) * (2 * sums + 2.0 ** -20)
            tol[h] += L * 2.0 ** -35 * p[h].max() * move.max(0)
            tol[h] += 15 * top[h] * (L * 2.0 ** -33 * p[h].max() + 2.0 ** -24)
        tol += np.abs(want) * 2.0 ** -24
        err = np.abs(out[s] - want)
        assert (err <= tol).all(), (s, float((err / tol).max()), float(err.max()))
        lt = 1.5 * ((p * weight).sum(-1) + sums + L * 2.0 ** -35 * p.max(-1)) + np.abs(wl) * 2.0 ** -22 + 2.0 ** -20
        assert (np.abs(lse[s] - wl) <= lt).all(), (s, float((np.abs(lse[s] - wl) / lt).max()))


def with_channels(S, Hq, D, dt, peak, seed=0):
    """Normal queries with one element of each head at `peak`, in turn of either sign."""
    q = randn((S, Hq, D), dt, seed)
    rng = np.random.default_rng(seed)
    for s in range(S):
        for h in range(Hq):
            q[s, h, rng.integers(D)] = peak * (-1) ** h
    return q


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("peak", [30.0, 100.0, 300.0, 3000.0])
def test_queries_with_a_large_channel(peak, D, dt):
    # one token: the denominator's logarithm is the score itself
    t = Batch([int(peak), D], [1] * 24, 2, D, 16, dt)
    check(t, with_channels(24, 8, D, dt, peak), 1 / math.sqrt(D))
    # minima far from zero
    t = Batch([int(peak), D], [1] * 24, 2, D, 16, dt)
    t.kp[..., t.D // 32:] += np.float16(20)
    t.cache = b.Q4Cache(dev(t.kc), dev(t.vc), dev(t.kp), dev(t.vp), DT[dt])
    check(t, with_channels(24, 8, D, dt, peak), 1 / math.sqrt(D))
# ------------------------------------------------------------------------------ weights
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("Hk,G,D,B", [(1, 1, 64, 8), (2, 4, 128, 16), (1, 8, 128, 32), (2, 3, 64, 32), (1, 12, 128, 16)])
@pytest.mark.parametrize("std", [0.01, 1.0])
def test_weights_keep_their_bits(std, Hk, G, D, B, dt):
    # nearly equal weights: their own rounding is what an output would show
    t = Batch([G, D, B], [20, 33, 1, 700, 5], Hk, D, B, dt)
    for num_ctas in (0, 3):
        check(t, randn((5, Hk * G, D), dt, 1, std), 1 / math.sqrt(D), num_ctas=num_ctas)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("peak", [30.0, 300.0])
def test_contexts_of_queries_with_a_large_channel(peak, D):
    t = Batch([int(peak), D], [700, 33, 64], 2, D, 16)
    check(t, with_channels(3, 8, D, t.dt, peak), 0.01)
# ---------------------------------------------------------------------------- V scales
@pytest.mark.parametrize("num_ctas", [0, 1])
@pytest.mark.parametrize("D,top", [(64, 0.3), (64, 5000.0), (128, 300.0), (128, 60000.0)])
def test_light_tokens_beside_a_large_scale(D, top, num_ctas):
    # one token 2^18 to 2^22 above 131071 others, which hold about a tenth of the softmax together
    L, NG = 131072, D // 32
    t = Batch([D, int(top)], [L], 1, D, 32)
    rng = np.random.default_rng(1)
    t.kp[..., :NG] = 0
    x = -rng.uniform(18, 22, L) * math.log(2) / (D * 0.125)
    x[200] = 0                                        # (of the first warp where there are 16)
    t.kp[t.tab[0, : L // 32], 0, :, NG:] = x.reshape(-1, 32, 1).astype(np.float16)
    t.vp[t.tab[0, 3], 0, 0, 5] = top                  # a V scale of group 0, token 101
    t.cache = b.Q4Cache(dev(t.kc), dev(t.vc), dev(t.kp), dev(t.vp), DT[t.dt])
    check(t, torch.ones(1, 2, D, dtype=DT[t.dt]), 0.125, num_ctas=num_ctas)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scales", [(1e-6, 1e-6), (1e-4, 1e-4), (1e-4, 1000.0), (1000.0, 1e-4), (60000.0, 1e-6)])
def test_tiny_and_mixed_scales(scales, D):
    # even and odd groups of different orders, with minima of their own order
    NG = D // 32
    t = Batch(3, [300, 17], 2, D, 16)
    rng = np.random.default_rng(2)
    for g in range(NG):
        s = rng.uniform(0.3, 1.0, t.vp[:, :, g].shape) * scales[g % 2]
        live = ~np.isnan(t.vp[:, :, g])
        t.vp[:, :, g][live] = s[live].astype(np.float16)
        t.vp[:, :, NG + g][live] = (-7.5 * np.minimum(s, 8000))[live].astype(np.float16)
    t.cache = b.Q4Cache(dev(t.kc), dev(t.vc), dev(t.kp), dev(t.vp), DT[t.dt])
    for std in (0.01, 1.0):
        check(t, randn((2, 8, D), t.dt, 4, std), 1 / math.sqrt(D))


def test_scales_that_grow_from_tiny_to_large():
    t = Batch(7, [640], 1, 64, 16)
    for i, blk in enumerate(t.tab[0, :40]):
        t.vp[blk] = (t.vp[blk].astype(np.float64) * 2.0 ** (i - 22)).clip(-60000, 60000).astype(np.float16)
    t.cache = b.Q4Cache(dev(t.kc), dev(t.vc), dev(t.kp), dev(t.vp), DT[t.dt])
    for c in (1, 3):
        check(t, randn((1, 3, 64), t.dt, 0, 2.0), 0.125, num_ctas=c)


# -------------------------------------------------------------------------- long sums
@pytest.mark.parametrize("G", [1, 5])
@pytest.mark.parametrize("D", [64, 128])
def test_long_sums_are_not_cut_to_one_side(D, G):
    """Nearly equal weights over n = 8192 tokens a warp: the codes' share of an output and the minima's
    are some 2 and cancel, so a sum that is cut towards zero at each step would show (7e-5 here). The
    tolerance, in units u = 2^-23 of the mean |m| or scale s:
      - sums of minima, scales and weights in fp32, two additions a subtile to nearest, N = n / 16 each:
        errors of either sign with a deviation of u / sqrt(12) of the sum so far, sqrt(N / 3) u / sqrt(12)
        in all; three sums, 16 warps, six deviations: 0.44 sqrt(N) u
      - their products within a half, cut at most four times: 4 u
      - codes around zero: n steps of up to 7.5 s, 4.7 s rms of either sign, wander to 6 times
        4.7 s sqrt(n), of which each of n / 8 cuts takes up to u: (n / 8) 28 s / sqrt(n) u of the mean."""
    L, NG = 131072, D // 32
    n = L // 16
    t = Batch(5, [L], 1, D, 32)
    q = randn((1, G, D), t.dt, 3, 0.01)
    k, v = O.q4_rows(t.tab[0], L, t.kc, t.vc, t.kp, t.vp)
    want, _, _ = O.attend(q[0].double().numpy(), k, v, 0.09)
    par = np.abs(t.vp[t.tab[0, : L // 32]].astype(np.float64)).mean((0, 1, 3))
    s, m = np.repeat(par[:NG], 32), np.repeat(par[NG:], 32)
    u = 2.0 ** -23
    tol = u * ((0.44 * math.sqrt(n / 16) + 4) * m + n / 8 * 28 * s / math.sqrt(n)) + np.abs(want) * 2.0 ** -19
    out = b.decode_attention_q4(q.cuda(), t.cache, dev(t.tab), dev(t.lens), 0.09, out_dtype=torch.float32, num_ctas=1)
    err = np.abs(out[0].double().cpu().numpy() - want)
    assert b.get_error() == 0
    assert (err <= tol).all(), (float((err / tol).max()), float(err.max()))
