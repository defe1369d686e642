"""Block-sparse decode on the GPU: means and selections exactly as defined (the order of the fp32
additions is part of the definition), the attention over the selection within the decode's own
tolerance (2e-3 for 16-bit caches, 1e-5 for fp32) of 64 bits."""
import math

import numpy as np
import pytest
import torch

from oracle import step_ops as O
from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def randn(shape, dt, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dt])


def rounder(dt):
    return lambda x: torch.from_numpy(x).to(DT[dt])


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("D", [64, 128])
def test_means_exact(D, B, dt):
    NB, Hk = 9, 3
    k = randn((NB, Hk, B, D), dt, 1)
    k[4] = math.nan                                   # never asked for
    means = torch.full((NB, Hk, D), 9.0, dtype=DT[dt], device="cuda")
    slots = np.array([2 * B + B - 1, -1, 5, 7 * B + B - 1, 4 * B + B - 2, 8 * B + B - 1, -B])
    b.block_means(dev(slots), k.cuda(), means)
    assert b.get_error() == 0
    want = torch.full((NB, Hk, D), 9.0, dtype=DT[dt])
    for blk in (2, 7, 8):
        want[blk] = O.block_mean(k[blk].float().numpy(), rounder(dt))
    assert torch.equal(means.cpu(), want)
    b.block_means(dev(np.array([NB * B + B - 1])), k.cuda(), means)
    assert b.get_error() == b.DEVERR_SLOT and torch.equal(means.cpu(), want)


class Batch:
    def __init__(self, seed, lens, Hk, D, B, dt, ties=False):
        rng = np.random.default_rng(seed)
        lens = np.asarray(lens, np.int32)
        n = -(-lens // B)
        M = int(n.max()) + 1
        NB = int(n.sum()) + 2
        self.tab = np.full((len(lens), M), -1, np.int32)
        self.tab[np.arange(M)[None, :] < n[:, None]] = rng.permutation(NB)[: int(n.sum())]
        self.k, self.v = (randn((NB, Hk, B, D), dt, int(rng.integers(1 << 30))) for _ in range(2))
        self.means = O.block_mean(self.k.float().numpy(), rounder(dt))
        if ties:                                      # few different means: many equal scores
            self.means = self.means[torch.from_numpy(rng.integers(0, 3, NB))].contiguous()
        for s, L in enumerate(lens):                  # rows behind the last token hold NaN
            if L % B:
                for p in (self.k, self.v):
                    p[self.tab[s, n[s] - 1], :, L % B:] = math.nan
                self.means[self.tab[s, n[s] - 1]] = math.nan
        self.lens, self.n, self.B, self.D, self.Hk, self.dt = lens, n, B, D, Hk, dt

    def selection(self, q, s, h, top, first, last):
        G = q.shape[1] // self.Hk
        blk = self.tab[s, : self.n[s]].astype(np.int64)
        sc = O.block_scores(q[s, h * G: (h + 1) * G].float().numpy(), self.means[torch.from_numpy(blk), h].float().numpy())
        return O.select(sc, int(self.n[s]), top, first, last)

    def check(self, G, top, first=1, last=1, seed=0, attention=True):
        S, W = len(self.lens), top + first + last
        q = randn((S, G * self.Hk, self.D), self.dt, seed)
        args = (dev(self.tab), dev(self.lens))
        kp, vp, km = self.k.cuda(), self.v.cuda(), self.means.cuda()
        st, sl = b.select_blocks(q.cuda(), kp, km, *args, top, first, last)
        assert b.get_error() == 0
        out = None
        if attention:
            st2, sl2 = torch.full_like(st, 77), torch.full_like(sl, 77)
            ws = b.alloc_sparse_workspace(kp, S, G * self.Hk, self.tab.shape[1])
            out = b.decode_attention_sparse(q.cuda(), kp, vp, km, *args, 1 / math.sqrt(self.D), top, first, last,
                                            out_dtype=torch.float32, sel_tables=st2, sel_lens=sl2, workspace=ws)
            assert b.get_error() == 0
            assert torch.equal(st, st2) and torch.equal(sl, sl2)
            assert not ws[: 4096 * (16 if self.dt == "f32" else 4)].any()     # arrival counters back at zero
            out = out.double().cpu().numpy()
        st, sl = st.cpu().numpy(), sl.cpu().numpy()
        tol = 1e-5 if self.dt == "f32" else 2e-3
        for s, L in enumerate(self.lens):
            for h in range(self.Hk):
                sel = self.selection(q, s, h, top, first, last) if L else []
                want = [int(self.tab[s, j]) * self.Hk + h for j in sel]
                assert st[s, h].tolist() == want + [-1] * (W - len(want)), (s, h)
                have = (len(sel) - 1) * self.B + int(L) - (int(self.n[s]) - 1) * self.B if L else 0
                assert sl[s, h] == have
                if not attention:
                    continue
                o = out[s, h * G: (h + 1) * G]
                if not L:
                    assert not o.any()
                    continue
                idx = torch.from_numpy(self.tab[s, sel].astype(np.int64))
                k, v = (p[idx, h].double().reshape(-1, self.D)[:have].numpy()[None] for p in (self.k, self.v))
                ref, _, _ = O.attend(q[s, h * G: (h + 1) * G].double().numpy(), k, v, 1 / math.sqrt(self.D))
                assert np.abs(o - ref).max() <= tol


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G", [(1, 1), (2, 2), (3, 3), (2, 4), (1, 5), (1, 8), (2, 12), (1, 17)])
def test_sparse_head_groups(Hk, G, D, dt):
    Batch([Hk, G], [400, 0, 1, 33, 160], Hk, D, 8, dt).check(G, 6, 1, 2)


@pytest.mark.parametrize("top,first,last", [(0, 0, 1), (0, 2, 3), (1, 0, 1), (5, 3, 2), (49, 0, 1), (50, 1, 1),
                                            (200, 0, 1), (3, 60, 1), (3, 0, 70)])
@pytest.mark.parametrize("B", [8, 16, 32])
def test_sparse_selections(top, first, last, B):
    # 50 blocks, full and not
    Batch([top, first, B], [50 * B, 50 * B - 3, 49 * B + 1, B, 1], 2, 64, B, "bf16").check(4, top, first, last)


@pytest.mark.parametrize("top", [1, 7, 40])
def test_ties_go_to_the_lower_block(top):
    Batch(top, [16 * 80, 16 * 79 + 5], 2, 64, 16, "f16", ties=True).check(2, top, 2, 3)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_long_selections(dt):
    # 600 to 20000 blocks: several keys a thread, several passes
    Batch(1, [8 * 600], 1, 64, 8, dt).check(4, 100, 1, 4)
    Batch(2, [8 * 9001 - 1, 8 * 20000], 1, 64, 8, dt).check(2, 1000, 4, 4, attention=dt == "bf16")
    Batch(3, [8 * 20011], 1, 64, 8, dt, ties=True).check(1, 9999, 0, 1, attention=False)


@pytest.mark.parametrize("S,Hk,hi", [(1, 2, 60), (19, 8, 60), (3, 2, 300), (38, 8, 300), (1, 1, 1023), (2, 1, 1024),
                                     (39, 8, 300), (305, 1, 1100), (5, 1, 1100), (160, 1, 1100), (305, 1, 16384), (305, 1, 16385)])
def test_selection_forms(S, Hk, hi):
    """Rows for less and more than one, two and four CTAs an SM, short and long; more than 256
    candidates and fewer."""
    rng = np.random.default_rng(S)
    lens = rng.integers(1, 8 * (min(hi, 1100) - 1), S)
    lens[0] = 8 * (hi - 1)                           # table columns: hi
    Batch(40, lens, Hk, 64, 8, "bf16").check(2, 30, attention=False)
    if S == 38:
        Batch(41, lens, Hk, 64, 8, "bf16", ties=True).check(2, 30, attention=False)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G", [(1, 1), (3, 2), (2, 4), (1, 5), (2, 8), (1, 12)])
def test_spread_selections(Hk, G, D, dt):
    """Long rows, few of them: scores from all over the GPU."""
    Batch(43, [8 * 1500 - 3, 0, 8 * 1030, 5, 8 * 70 + 1], Hk, D, 8, dt).check(G, 25, 2, 3)


@pytest.mark.parametrize("S", [256, 257, 300])
def test_sparse_many_rows(S):
    """2048 rows are one launch of the decode, more are several."""
    lens = np.random.default_rng(0).integers(0, 60, S)
    Batch(42, lens, 8, 64, 8, "f16").check(3, 2)


def test_nan_infinite_and_zero_means():
    t = Batch(4, [16 * 30], 1, 64, 16, "bf16")
    for j, x in ((3, math.nan), (9, math.inf), (10, -math.inf), (20, 0.0), (21, -0.0)):
        t.means[t.tab[0, j]] = x
    for top in (1, 2, 3, 5, 28):
        t.check(3, top, 0, 1, attention=False)


def test_bad_ids_and_lengths_are_flagged():
    t = Batch(5, [16 * 10, 16 * 10], 2, 64, 16, "bf16")
    q = randn((2, 4, 64), "bf16", 0).cuda()
    tab = t.tab.copy()
    tab[0, 0] = len(t.k)                             # always listed
    tab[1, 9] = -4
    st, sl = b.select_blocks(q, t.k.cuda(), t.means.cuda(), dev(tab), dev(t.lens), 3, 1, 1)
    assert b.get_error() == b.DEVERR_BLOCK_ID
    assert st[0, 0, 0] == -1 and st[1, 1, 4] == -1 and (st[0, :, 1:] >= 0).all() and (sl == 80).all()
    lens = t.lens.copy()
    lens[0], lens[1] = -1, 10000
    st, sl = b.select_blocks(q, t.k.cuda(), t.means.cuda(), dev(t.tab), dev(lens), 3, 1, 1)
    assert b.get_error() & b.DEVERR_CONTEXT
    assert (sl[0] == 0).all() and (st[0] == -1).all()


def test_sparse_graph_and_other_stream():
    t = Batch(6, [16 * 40, 16 * 25 + 3], 2, 128, 16, "bf16")
    q = randn((2, 8, 128), "bf16", 0).cuda()
    kp, vp, km = t.k.cuda(), t.v.cuda(), t.means.cuda()
    out = torch.zeros_like(q)
    ws = b.alloc_sparse_workspace(kp, 2, 8, t.tab.shape[1])
    call = b.prepared_decode_attention_sparse(q, kp, vp, km, dev(t.tab), dev(t.lens), 0.09, 6, 1, 2, out=out, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    q.neg_()
    g.replay()
    assert torch.equal(out, b.decode_attention_sparse(q, kp, vp, km, dev(t.tab), dev(t.lens), 0.09, 6, 1, 2))


def test_sparse_two_streams_at_once():
    runs = []
    for seed, lens, Hk in ((7, [16 * 700, 16 * 250 + 3], 2), (8, list(range(16, 16 * 90, 70)), 8)):
        t = Batch(seed, lens, Hk, 128, 16, "bf16")
        q = randn((len(lens), 4 * Hk, 128), "bf16", 0).cuda()
        pools = (t.k.cuda(), t.v.cuda(), t.means.cuda())
        args = (q, *pools, dev(t.tab), dev(t.lens), 0.09, 6, 1, 2)
        want = b.decode_attention_sparse(*args)
        outs = [torch.zeros_like(q) for _ in range(20)]
        ws = b.alloc_sparse_workspace(pools[0], len(lens), 4 * Hk, t.tab.shape[1])
        runs.append((torch.cuda.Stream(), want, outs,
                     [b.prepared_decode_attention_sparse(*args, out=o, workspace=ws) for o in outs]))
    torch.cuda.synchronize()
    for i in range(20):
        for st, _, _, calls in runs:
            calls[i](st)
    torch.cuda.synchronize()
    for _, want, outs, _ in runs:
        for o in outs:
            assert torch.equal(o, want)


@pytest.mark.parametrize("S", [18, 20])
def test_sparse_pool_past_32_bits(S):
    """Chunks and means at both ends of a pool of more than 2^32 bytes; 18 sequences of 8 heads are
    fewer rows than SMs, 20 more: the selection's two forms."""
    Hk, B, D, NB, n = 8, 32, 128, 70000, 13
    assert NB * Hk * B * D * 2 > 1 << 32
    t = Batch(9, [B * n - 5] * S, Hk, D, B, "bf16")
    args = (1 / math.sqrt(D), 4, 1, 2)
    q = randn((S, 4 * Hk, D), "bf16", 3).cuda()
    small = [x.cuda() for x in (t.k, t.v, t.means)]
    lens = dev(t.lens)
    want = b.decode_attention_sparse(q, *small, dev(t.tab), lens, *args)
    place = np.arange(len(t.k)) * 3
    place = np.where(np.arange(len(t.k)) % 2 == 0, place, NB - 1 - place)
    at = torch.from_numpy(place).cuda()
    big = [torch.empty(NB, *x.shape[1:], dtype=x.dtype, device="cuda") for x in small]
    for x, y in zip(big, small):
        x[at] = y
    tab = np.where(t.tab >= 0, place[t.tab], -1).astype(np.int32)
    assert torch.equal(want, b.decode_attention_sparse(q, *big, dev(tab), lens, *args))
    # the means of the same blocks, from their slots
    full = place[t.tab[:, : n - 1].ravel()].astype(np.int64)
    big[2].zero_()
    b.block_means(dev(full * B + B - 1), big[0], big[2])
    assert torch.equal(big[2][torch.from_numpy(full).cuda()], small[2][torch.from_numpy(t.tab[:, : n - 1].ravel().astype(np.int64)).cuda()])
    assert b.get_error() == 0
