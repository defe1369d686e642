"""Weights of the decode over selected blocks, 16-bit caches, against 64 bits.

Tolerance of an output sum p_t v_t: a score's sums of D exact products in fp32 are off by less than
(D / 8 + 8) 2^-23 of |scale| sum |q k|, its exponent z (log2 units) by 2^-21 |z|, the exponential by
2^-21. A weight enters the product as two numbers of the cache's type: kept to 2^-22 (fp16; at least to
2^-25 where the largest is at 2^10 or above, 2^-35 of it) or 2^-17 (bf16, two times eight bits and the
signs), and the denominator sums what enters. Sums over tokens: a warp adds its own, 16 at a time,
and up to 64 additions join the warps' pieces: (n / 16 + 64) 2^-23 for n tokens a warp, the
denominator's the same."""
import math

import numpy as np
import pytest
import torch

from oracle import step_ops as O
from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def check(q, k, v, scale, dt, B, S=1):
    """One context of L tokens, all blocks selected, S times. q [G][D], k and v [L][D], fp32 of the type's values."""
    L, D = k.shape
    n = -(-L // B)
    pools = [torch.full((n * B, D), math.nan) for _ in range(2)]
    for p, x in zip(pools, (k, v)):
        p[:L] = x
    order = torch.from_numpy(np.random.default_rng(0).permutation(n))
    pools = [p.view(n, 1, B, D)[order].to(DT[dt]).cuda() for p in pools]
    tab = torch.argsort(order).to(torch.int32).repeat(S, 1).cuda()
    lens = torch.full((S,), L, dtype=torch.int32, device="cuda")
    means = torch.zeros(n, 1, D, dtype=DT[dt], device="cuda")
    out = b.decode_attention_sparse(q.to(DT[dt]).repeat(S, 1, 1).cuda(), *pools, means, tab, lens, scale, n, out_dtype=torch.float32)
    assert b.get_error() == 0
    out = out.double().cpu().numpy()
    # tokens a warp has of a context: an even share of all subtiles of 16, a context's start counted as two
    warps = 10 * torch.cuda.get_device_properties(0).multi_processor_count
    share = min(L, 16 * (S * -(-len(q) // 8) * (-(-L // 16) + 2) // warps + 4))
    sums = (share / 16 + 64) * 2.0 ** -23
    q, k, v = (x.double().numpy() for x in (q, k, v))
    want, wl, p = O.attend(q, k[None], v[None], scale)
    size = abs(scale) * np.abs(q) @ np.abs(k).T
    z = np.abs(wl)[:, None] + np.abs(np.log2(np.maximum(p, 1e-300)))
    weight = size * (D / 8 + 8) * 2.0 ** -23 + (z + 1) * 2.0 ** -21 + (2.0 ** -22 if dt == "f16" else 2.0 ** -17)
    for h in range(len(q)):
        move = np.abs(v - want[h])
        tol = 2 * (p[h] * weight[h]) @ move + 2 * sums * (p[h] @ np.abs(v)) + np.abs(want[h]) * 2.0 ** -24
        if dt == "f16":
            tol += L * 2.0 ** -35 * p[h].max() * move.max(0)
        err = np.abs(out[:, h] - want[h])
        assert (err <= tol).all(), (h, float((err / tol).max()), float(err.max()))


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D,G", [(64, 3), (128, 8), (128, 12)])
def test_many_light_tokens(D, G, dt):
    # one token 2^25 above 65000 others: together 2^-9 of the softmax; contexts enough for warps of 4000 to 8000 tokens
    L, S = 65001, 186 if G <= 8 else 93
    rng = np.random.default_rng(D)
    x = -rng.uniform(25.05, 25.3, L) * math.log(2) / (D * 0.125)
    x[40000] = 0
    k = torch.from_numpy(x)[:, None].repeat(1, D).float().to(DT[dt]).float()
    v = torch.from_numpy(1 + 0.1 * rng.normal(size=(L, D))).float().to(DT[dt]).float()
    v[40000] = -1
    check(torch.ones(G, D), k, v, 0.125, dt, 32, S)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("std", [0.01, 1.0])
@pytest.mark.parametrize("L,D,B", [(1, 64, 8), (20, 128, 16), (333, 64, 32), (2000, 128, 8)])
def test_weights_keep_their_bits(L, D, B, std, dt):
    g = torch.Generator().manual_seed(L)
    q, k, v = (torch.randn(n, D, generator=g).to(DT[dt]).float() for n in (5, L, L))
    check((q * std).to(DT[dt]).float(), k, v, 1 / math.sqrt(D), dt, B)
