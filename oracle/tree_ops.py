"""Plain implementations of the calls that verify drafted tokens (include/pkv_tree.h), in 64 bits, on the CPU or
wherever the tensors lie. Test infrastructure only."""
import math

import numpy as np
import torch


def ancestors(parents):
    """bool [n][n]: token j is i or above it."""
    a = np.zeros((len(parents), len(parents)), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            a[i] = a[p]
        a[i, i] = True
    return a


def words(a, W):
    """int64 [n][W] of the truth values [n][m]."""
    m = np.zeros((a.shape[0], W), np.uint64)
    for j in range(a.shape[1]):
        m[:, j // 64] |= a[:, j].astype(np.uint64) << np.uint64(j % 64)
    return m.view(np.int64)


def accept(parents, tokens, targets):
    """(path, next token) of one sequence."""
    holds, depth, best = [], [], -1
    for i, p in enumerate(parents):
        holds.append(p < 0 or (holds[p] and tokens[i] == targets[p]))
        depth.append(0 if p < 0 else depth[p] + 1)
        if holds[i] and (best < 0 or depth[i] > depth[best]):
            best = i
    path, i = [], best
    while i >= 0:
        path.insert(0, i)
        i = parents[i]
    return path, (int(targets[best]) if best >= 0 else -1)


def rows_of(pool, table, L):
    """K or V rows [Hk][L][D] of a context, in 64 bits; a block outside the pool reads as zeros."""
    NB, Hk, B, D = pool.shape
    ids = table[: -(-L // B)].long()
    ok = (ids >= 0) & (ids < NB)
    x = pool[ids.clamp(0, NB - 1)].double()
    x[~ok] = 0
    return x.transpose(0, 1).reshape(Hk, -1, D)[:, :L]


def attend(q, k, v, sees, scale):
    """q [n][Hq][D], k and v [Hk][L][D], sees [n][L]: (out [n][Hq][D], log2 denominators [n][Hq], the largest
    sum |q k| scale of a seen place, the largest seen |v|). What is not seen is not looked at."""
    n, Hq, D = q.shape
    Hk = k.shape[0]
    out = torch.zeros(n, Hq, D, dtype=torch.float64, device=q.device)
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device=q.device)
    Z = V = 0.0
    for i in range(n):
        t = torch.nonzero(sees[i])[:, 0]
        if len(t) == 0:
            continue
        kk, vv, qq = k[:, t], v[:, t], q[i].double().view(Hk, -1, D)
        z = torch.einsum("hgd,htd->hgt", qq, kk) * scale
        out[i] = torch.einsum("hgt,htd->hgd", torch.softmax(z, -1), vv).reshape(Hq, D)
        lse[i] = (torch.logsumexp(z, -1) / math.log(2)).reshape(Hq)
        Z = max(Z, float(torch.einsum("hgd,htd->hgt", qq.abs(), kk.abs()).max()) * abs(scale))
        V = max(V, float(vv.abs().max()))
    return out, lse, Z, V
