"""The 4-bit cache on the GPU: codes and parameters bit for bit, gathered values exactly, and the
decode attention against 64 bits.

Tolerance of one output element o = sum p_t v_t: a weight p_t is off by
  - its rounding to fp16, half a step, 2^-11 relative (the denominator sums the rounded weights, so
    this moves the average around: sum p_t |v_t - o| 2^-11);
  - the error of its exponent. A score sums D exact products and NG scaled partial sums in fp32:
    below (D / 8 + 8) 2^-23 of scale sum |q| (|s c| + |m|) for any order within the matrix
    instructions, plus the exponential, 2^-21;
and a weight times a V scale is kept to 2^-22, its sums over the tokens to (L / 16 + 16) 2^-23 of
sum p_t (|s c| + |m|). Then half a step of the output's type. fp16 weights below 2^-14 of what they
are scaled to (the largest is brought to at least 2^5) are off by at most 2^-25, 2^-30 of the
largest weight each: L 2^-30 of the largest |v - o|."""
import math

import numpy as np
import pytest
import torch

from oracle import step_ops as O
from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def randn(shape, dt, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(DT[dt])


def cache_arrays(c):
    return [t.cpu().numpy() for t in (c.k_codes, c.v_codes, c.k_params, c.v_params)]


# ------------------------------------------------------------------------------ store
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hk,D,B", [(1, 1, 64, 8), (1, 8, 128, 16), (67, 3, 64, 16), (300, 8, 128, 32),
                                      (129, 5, 128, 8), (5000, 8, 128, 16), (9001, 5, 64, 32)])
def test_append_bits_and_gather(T, Hk, D, B, dt):
    rng = np.random.default_rng([T, B])
    k, v = randn((T, Hk, D), dt, 0), randn((T, Hk, D), dt, 1, 3.0)
    k[0, 0, :32] = 0.75                              # a constant group: scale 0
    v[-1, -1, 32:] = 0
    k[0, -1, 33] *= 1000
    NB = -(-T // B) + 2
    slots = rng.permutation(NB * B)[:T]
    slots[rng.random(T) < 0.1] = -1
    slots[0] = 3
    slots[1:][slots[1:] == 3] = -1
    c = b.Q4Cache.empty(NB, Hk, B, D, DT[dt])
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xA5)
    want = O.q4_append(k.float().numpy(), v.float().numpy(), slots, *cache_arrays(c))
    b.append_q4(k.cuda(), v.cuda(), dev(slots), c)
    assert b.get_error() == 0
    for g, w in zip(cache_arrays(c), want):
        np.testing.assert_array_equal(g.view(np.uint8), w.view(np.uint8))
    # every row, some twice, some none
    ask = np.concatenate([slots, slots[:1], [-1, NB * B - 1]])
    for od in (torch.float32, torch.float16, torch.bfloat16):
        ko, vo = b.gather_q4(dev(ask), c, out_dtype=od)
        for i, s in enumerate(ask):
            if s < 0:
                assert not ko[i].any() and not vo[i].any()
        live = np.flatnonzero(ask >= 0)
        NG = D // 32
        for o, codes, par, rows in ((ko, want[0], want[2], True), (vo, want[1], want[3].swapaxes(2, 3), False)):
            blk, off = ask[live] // B, ask[live] % B
            p = par[blk, :, off]
            x = O.q4_values(O.q4_unpack(codes[blk, :, off], rows), p[..., :NG], p[..., NG:])
            # s c is exact in fp32 and the sum is rounded once, then to the output's type
            x = torch.from_numpy(x.astype(np.float32)).to(od)
            assert torch.equal(o.cpu()[live], x)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_append_extremes(dt):
    D, Hk = 64, 2
    k = torch.zeros(6, Hk, D, dtype=DT[dt])
    k[0, 0, 0], k[0, 1, 40] = math.inf, -math.inf
    k[1, 0, 5] = math.nan
    k[2, 0, :2] = torch.tensor([6e4, -6e4])
    k[3, 0, :32] = torch.finfo(DT[dt]).tiny * torch.arange(32)
    k[4, 0, 1] = -0.0
    if dt == "bf16":
        k[5, 0, :3] = torch.tensor([3e38, -3e38, 1e30])
    c = b.Q4Cache.empty(1, Hk, 8, D, DT[dt])
    slots = np.arange(6)
    want = O.q4_append(k.float().numpy(), k.float().numpy(), slots, *cache_arrays(c))
    b.append_q4(k.cuda(), k.cuda(), dev(slots), c)
    got = cache_arrays(c)
    for i in (0, 1):
        np.testing.assert_array_equal(got[i], want[i])
    for i in (2, 3):
        np.testing.assert_array_equal(np.isnan(got[i]), np.isnan(want[i]))
        ok = ~np.isnan(want[i])
        assert (got[i][ok] == want[i][ok]).all()
    assert np.isnan(got[2]).sum() == 6 and b.get_error() == 0


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("low", [0.0, -8.0, 512.0, 1000.0])
def test_append_halves(dt, low):
    """Quotients on a half, and one step of the rows' type to either side of it."""
    t = low + 2.0 * torch.arange(16, dtype=torch.float64)
    halves = (t[:15] + 1).to(DT[dt])
    step = torch.tensor([torch.finfo(DT[dt]).eps]).to(torch.float64) * halves.double().abs()
    rows = []
    for d in (0, -1, 1, -0.5, 0.5):
        x = torch.zeros(32, dtype=torch.float64)
        x[:16], x[16:31], x[31] = t, halves.double() + d * step, low
        rows.append(x.to(DT[dt]))
    k = torch.stack(rows * 8)[:, None, :].repeat(1, 3, 4)
    c = b.Q4Cache.empty(6, 3, 8, 128, DT[dt])
    slots = np.random.default_rng(0).permutation(48)[: len(k)]
    want = O.q4_append(k.float().numpy(), -k.float().numpy(), slots, *cache_arrays(c))
    b.append_q4(k.cuda(), -k.cuda(), dev(slots), c)
    assert b.get_error() == 0
    for g, w in zip(cache_arrays(c), want):
        np.testing.assert_array_equal(g.view(np.uint8), w.view(np.uint8))
    if low == 0 or dt == "f16":                      # (the type holds every one of these halves)
        assert (want[2][slots[0] // 8, 0, slots[0] % 8, :4] == 2).all()
        codes = O.q4_unpack(want[0][slots[0] // 8, 0, slots[0] % 8], True).reshape(4, 32)[0]
        assert codes[:16].tolist() == list(range(16))
        assert codes[16:31].tolist() == [2 * ((i + 1) // 2) for i in range(15)]


def test_pool_past_32_bits():
    """Codes and parameters whose byte offsets pass 2^32: both ends of the pool."""
    Hk, B, D, NB = 8, 32, 128, 270000                # codes 4.4 GB each, element offsets past 2^32
    assert NB * Hk * B * (D // 2) > 1 << 32
    c = b.Q4Cache.empty(NB, Hk, B, D, torch.bfloat16)
    ids = np.array([NB - 1, 0, NB - 2, 1, NB // 2], np.int32)
    L = 5 * B - 3
    k, v = randn((L, Hk, D), "bf16", 0), randn((L, Hk, D), "bf16", 1)
    pos = np.arange(L)
    slots = ids[pos // B].astype(np.int64) * B + pos % B
    small = b.Q4Cache.empty(5, Hk, B, D, torch.bfloat16)
    for cache, at in ((c, slots), (small, pos)):
        b.append_q4(k.cuda(), v.cuda(), dev(at), cache)
    q = randn((1, 32, D), "bf16", 2).cuda()
    lens = dev(np.array([L], np.int32))
    out = b.decode_attention_q4(q, c, dev(ids[None]), lens, 0.09)
    assert torch.equal(out, b.decode_attention_q4(q, small, dev(np.arange(5, dtype=np.int32)[None]), lens, 0.09))
    for x, y in zip(b.gather_q4(dev(slots), c), b.gather_q4(dev(pos), small)):
        assert torch.equal(x, y)
    b.block_copy_q4([[NB - 1, 2]], c)
    ids[0] = 2
    assert torch.equal(out, b.decode_attention_q4(q, c, dev(ids[None]), lens, 0.09))
    assert b.get_error() == 0

def test_bad_slots_are_flagged_and_skipped():
    c = b.Q4Cache.empty(2, 2, 8, 64, torch.float16)
    x = randn((3, 2, 64), "f16", 0).cuda()
    b.append_q4(x, x, dev(np.array([16, 1 << 40, 2])), c)
    assert b.get_error() == b.DEVERR_SLOT
    assert int((c.k_params[..., 0] != 0).sum()) == 2
    ko, vo = b.gather_q4(dev(np.array([16, 2, -9])), c)
    assert b.get_error() == b.DEVERR_SLOT
    assert not ko[0].any() and not vo[2].any() and ko[1].any()


def test_block_copy():
    c = b.Q4Cache.empty(5, 3, 16, 128, torch.bfloat16)
    for t in (c.k_codes, c.v_codes):
        t.random_(0, 256)
    for t in (c.k_params, c.v_params):
        t.normal_()
    before = [t.clone() for t in (c.k_codes, c.v_codes, c.k_params, c.v_params)]
    b.block_copy_q4([[0, 3], [1, 4]], c)
    for t, w in zip((c.k_codes, c.v_codes, c.k_params, c.v_params), before):
        assert torch.equal(t[3], w[0]) and torch.equal(t[4], w[1]) and torch.equal(t[:3], w[:3])


# ----------------------------------------------------------------------------- decode
class Batch:
    """Random 4-bit cache and tables; what no context holds is NaN."""

    def __init__(self, seed, lens, Hk, D, B, dt="bf16", big=1.0, off=0.0):
        rng = np.random.default_rng(seed)
        NG = D // 32
        lens = np.asarray(lens, np.int32)
        n = -(-lens // B)
        M = int(n.max()) + 2
        NB = int(n.sum()) + 3
        perm = rng.permutation(NB)[: int(n.sum())]
        self.tab = np.full((len(lens), M), -1, np.int32)
        self.tab[np.arange(M)[None, :] < n[:, None]] = perm
        used = np.zeros(NB, np.int64)
        used[self.tab[self.tab >= 0]] = np.clip(lens[:, None] - np.arange(M) * B, 0, B)[self.tab >= 0]
        dead = np.arange(B)[None, :] >= used[:, None]
        self.kc, self.vc = (rng.integers(0, 256, (NB, Hk, B, D // 2), dtype=np.uint8) for _ in range(2))
        par = []
        for g in (1.0, big):
            s = rng.uniform(0.1, 0.4, (NB, Hk, B, NG)) * g
            m = -7.5 * s + rng.normal(0, 0.3, s.shape) * g + off * g
            p = np.concatenate([s, m], -1).astype(np.float16)
            p[np.broadcast_to(dead[:, None, :], p.shape[:3])] = np.nan
            par.append(p)
        self.kp, self.vp = par[0], np.ascontiguousarray(par[1].swapaxes(2, 3))
        self.lens, self.B, self.D, self.Hk, self.dt = lens, B, D, Hk, dt
        self.cache = b.Q4Cache(dev(self.kc), dev(self.vc), dev(self.kp), dev(self.vp), DT[dt])

    def expect(self, q, scale, s):
        """(out, tolerance without the output's rounding, log2 denominators) of sequence s."""
        L = int(self.lens[s])
        k, v = O.q4_rows(self.tab[s], L, self.kc, self.vc, self.kp, self.vp)
        qs = q[s].double().numpy()
        out, lse, p = O.attend(qs, k, v, scale)
        G, NG = qs.shape[0] // self.Hk, self.D // 32
        # |s c| + |m| of every element
        blk = self.tab[s, : -(-L // self.B)].astype(np.int64)
        size = []
        for par in (self.kp[blk], self.vp[blk].swapaxes(2, 3)):
            a = 15 * np.abs(par[..., :NG].astype(np.float64)) + np.abs(par[..., NG:].astype(np.float64))
            a = np.repeat(a, 32, -1).transpose(1, 0, 2, 3).reshape(self.Hk, -1, self.D)[:, :L]
            size.append(np.repeat(a, G, 0))
        score_err = abs(scale) * np.einsum("hd,hld->hl", np.abs(qs), size[0]) * (self.D / 8 + 8) * 2.0 ** -23
        move = np.abs(np.repeat(v, G, 0) - out[:, None])
        tol = 2 * np.einsum("hl,hld->hd", p * (2.0 ** -11 + score_err + 2.0 ** -21), move)
        tol += np.einsum("hl,hld->hd", p, size[1]) * (2.0 ** -22 + (L / 16 + 16) * 2.0 ** -23)
        tol += L * 2.0 ** -30 * move.max(1)
        return out, tol, lse, score_err.max(1)

    def check(self, Hq, scale=None, seed=0, qstd=1.0, out_dtype=torch.float32, **kw):
        scale = 1 / math.sqrt(self.D) if scale is None else scale
        S = len(self.lens)
        q = randn((S, Hq, self.D), self.dt, seed, qstd)
        lse = torch.full((S, Hq), 7.0, device="cuda")
        ws = kw.pop("workspace", None)
        if ws is None:
            ws = b.alloc_q4_workspace(self.cache, Hq, kw.get("num_ctas", 0))
        out = b.decode_attention_q4(q.cuda(), self.cache, dev(self.tab), dev(self.lens), scale, out_dtype=out_dtype,
                                    lse_out=lse, workspace=ws, **kw)
        assert b.get_error() == 0
        assert not ws[: 4096 * 4].any()              # arrival counters back at zero
        got = out.double().cpu().numpy()
        for s in range(S):
            if self.lens[s] == 0:
                assert not got[s].any() and (lse[s] == -math.inf).all()
                continue
            want, tol, wl, se = self.expect(q, scale, s)
            tol = tol + np.abs(want) * torch.finfo(out_dtype).eps / 2 + (2.0 ** -25 if out_dtype == torch.float16 else 0)
            err = np.abs(got[s] - want)
            assert (err <= tol).all(), (s, float((err / tol).max()), float(err.max()))
            # denominator: weights to 2^-11 each, scores as above, fp32 sums; in log2 units
            lt = 1.5 * (2.0 ** -11 + se + (self.lens[s] / 16 + 16) * 2.0 ** -23) + np.abs(wl) * 2.0 ** -22 + 2.0 ** -20
            assert (np.abs(lse[s].double().cpu().numpy() - wl) <= lt).all()
        return out


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("L", [1, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 250, 511])
def test_decode_lengths(L, B, D):
    Batch([L, B], [L], 1, D, B).check(4)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk,G", [(1, 1), (3, 1), (2, 2), (2, 3), (1, 4), (2, 5), (1, 8), (2, 9), (1, 16), (1, 20)])
def test_decode_head_groups(Hk, G, D):
    Batch([Hk, G], [130, 0, 1, 77, 16], Hk, D, 16, "f16").check(Hk * G)


@pytest.mark.parametrize("num_ctas", [1, 2, 3, 7, 40, 152, 600])
@pytest.mark.parametrize("G", [4, 8])
def test_decode_splits(num_ctas, G):
    # units cut between warps, between CTAs, over many CTAs, and not at all
    Batch(num_ctas, [900, 3, 0, 1700, 40, 16, 5000, 0, 333], 2, 128, 16).check(2 * G, num_ctas=num_ctas)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_decode_types(dt, out_dtype):
    Batch(3, [100, 1, 700], 2, 128, 16, dt).check(8, out_dtype=out_dtype)


def test_decode_trailing_and_leading_empty_contexts():
    Batch(4, [0, 0, 5, 0, 90, 0, 0], 2, 64, 8).check(4)
    Batch(4, [0, 0, 0], 1, 64, 8).check(1)


@pytest.mark.parametrize("big,off", [(1e-3, 0.0), (40.0, 0.0), (900.0, 30.0), (1.0, 50.0)])
def test_decode_v_ranges(big, off):
    # V scales from tiny to near the end of fp16, minima far from zero
    Batch(5, [400, 33], 2, 128, 16, big=big, off=off).check(8)


@pytest.mark.parametrize("qstd,scale", [(0.0, None), (1e-20, None), (30.0, None), (300.0, 1.0), (1.0, -0.5), (1.0, 0.0)])
def test_decode_score_ranges(qstd, scale):
    # from equal weights to one token taking all
    Batch(6, [600, 20], 1, 128, 16).check(4, scale=scale, qstd=qstd)


def test_decode_growing_scales_and_scores():
    # the reference exponent and the bound on V scales move all along the context
    t = Batch(7, [640], 1, 64, 16)
    order = t.tab[0, :40]
    for i, blk in enumerate(order):
        t.vp[blk] *= np.float16(1.25 ** (i - 10) if i < 30 else 0.01)
        t.kp[blk] *= np.float16(0.05 * i)
    t.cache = b.Q4Cache(dev(t.kc), dev(t.vc), dev(t.kp), dev(t.vp), DT[t.dt])
    for c in (1, 3):
        t.check(3, num_ctas=c, qstd=2.0)


def test_decode_zero_scales():
    # constant groups: every value is the minimum
    t = Batch(8, [50], 2, 64, 8)
    t.kp[..., :2] *= 0
    t.vp[:, :, :2] *= 0
    t.cache = b.Q4Cache(dev(t.kc), dev(t.vc), dev(t.kp), dev(t.vp), DT[t.dt])
    t.check(4)


def test_decode_long_context():
    Batch(9, [131072 - 5], 1, 128, 32).check(8)
    Batch(9, [60000, 17], 2, 64, 8, "f16").check(2, num_ctas=2)


def test_decode_many_sequences():
    # more than one launch
    lens = np.random.default_rng(0).integers(0, 40, 1100)
    Batch(10, lens, 1, 64, 8).check(2)


def test_decode_nan_rows_show_and_dead_rows_do_not():
    t = Batch(11, [60, 60], 2, 64, 16)               # unused rows hold NaN already
    blk = t.tab[0, 2]
    t.vp[blk, 1, 0, 3] = np.nan                      # group 0 of token 35, head 1
    t.cache = b.Q4Cache(dev(t.kc), dev(t.vc), dev(t.kp), dev(t.vp), DT[t.dt])
    q = randn((2, 4, 64), t.dt, 0).cuda()
    out = b.decode_attention_q4(q, t.cache, dev(t.tab), dev(t.lens), 0.1).isnan().cpu()
    want = torch.zeros(2, 4, 64, dtype=torch.bool)
    want[0, 2:, :32] = True
    assert torch.equal(out, want)
    t.kp[blk, 0, 3, 1] = np.nan                      # a NaN score takes the whole head
    t.cache = b.Q4Cache(dev(t.kc), dev(t.vc), dev(t.kp), dev(t.vp), DT[t.dt])
    out = b.decode_attention_q4(q, t.cache, dev(t.tab), dev(t.lens), 0.1).isnan().cpu()
    want[0, :2] = True
    assert torch.equal(out, want)


def test_decode_bad_ids_and_lengths():
    t = Batch(12, [40, 70, 30], 1, 64, 16)
    q = randn((3, 2, 64), t.dt, 0).cuda()
    # a block id outside the pool reads as zeros
    tab = t.tab.copy()
    tab[1, 2] = len(t.kc)
    out = b.decode_attention_q4(q, t.cache, dev(tab), dev(t.lens), 0.1, out_dtype=torch.float32)
    assert b.get_error() == b.DEVERR_BLOCK_ID
    k, v = O.q4_rows(t.tab[1], 70, t.kc, t.vc, t.kp, t.vp)
    k[:, 32:48] = v[:, 32:48] = 0
    want, _, _ = O.attend(q[1].double().cpu().numpy(), k, v, 0.1)
    assert np.abs(out[1].cpu().numpy() - want).max() <= 2.0 ** -9 * np.abs(v).max()
    # lengths out of range: clamped, flagged
    lens = t.lens.copy()
    lens[0] = -4
    out = b.decode_attention_q4(q, t.cache, dev(t.tab), dev(lens), 0.1)
    assert b.get_error() == b.DEVERR_CONTEXT
    assert not out[0].any() and out[1].any()


def test_decode_other_stream_graph_and_shared_workspace():
    t, u = Batch(13, [300, 900, 45], 2, 128, 16), Batch(14, [2000, 31], 2, 128, 16)
    ws = b.alloc_q4_workspace(t.cache, 8)
    s = torch.cuda.Stream()
    outs, graphs, calls = [], [], []                 # a graph does not keep its call's tensors alive
    for x in (t, u):
        q = randn((len(x.lens), 8, 128), x.dt, 5).cuda()
        out = torch.zeros_like(q)
        call = b.prepared_decode_attention_q4(q, x.cache, dev(x.tab), dev(x.lens), 0.09, out=out, workspace=ws)
        s.wait_stream(torch.cuda.current_stream())
        call(s)
        s.synchronize()
        want = out.clone()
        out.zero_()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
            call()
        outs.append((out, want))
        graphs.append(g)
        calls.append(call)
    for _ in range(3):                               # two graphs, one workspace, one stream
        for g, (out, want) in zip(graphs, outs):
            out.zero_()
            g.replay()
            assert torch.equal(out, want)
    assert not ws[: 4096 * 4].any()


def test_decode_repeats_bitwise_and_tables_ready_changes_nothing():
    t = Batch(15, [3000, 10, 777, 0], 2, 128, 16)
    a = t.check(8)
    for kw in (dict(), dict(tables_ready=True)):
        assert torch.equal(t.check(8, **kw), a)


def test_decode_over_a_selection_of_one_head_blocks():
    # the head view: each (sequence, kv head) reads its own blocks
    t = Batch(16, [96, 96], 2, 64, 16)
    q = randn((2, 4, 64), t.dt, 0)
    tab = np.empty((2, 2, 3), np.int32)
    for s in range(2):
        for h in range(2):
            tab[s, h] = t.tab[s, [0, 2 + h, 5]] * 2 + h
    lens = np.full((2, 2), 48, np.int32)
    out = b.decode_attention_q4(q.cuda().view(4, 2, 64), t.cache.head_view(), dev(tab.reshape(4, 3)),
                                dev(lens.reshape(4)), 0.1, out_dtype=torch.float32).view(2, 4, 64).cpu()
    for s in range(2):
        k, v = O.q4_rows(t.tab[s], 96, t.kc, t.vc, t.kp, t.vp)
        for h in range(2):
            rows = np.concatenate([np.arange(16), np.arange(16) + 16 * (2 + h), np.arange(16) + 80])
            want, _, _ = O.attend(q[s, 2 * h: 2 * h + 2].double().numpy(), k[h: h + 1, rows], v[h: h + 1, rows], 0.1)
            assert np.abs(out[s, 2 * h: 2 * h + 2].numpy() - want).max() <= 2.0 ** -10 * np.abs(v).max()


def test_decode_two_streams_at_once():
    t, u = Batch(23, [4000, 900, 45], 2, 128, 16), Batch(24, [7000, 31], 2, 128, 16)
    runs = []
    for x in (t, u):
        q = randn((len(x.lens), 8, 128), x.dt, 5).cuda()
        want = b.decode_attention_q4(q, x.cache, dev(x.tab), dev(x.lens), 0.09)
        outs = [torch.zeros_like(q) for _ in range(20)]
        ws = b.alloc_q4_workspace(x.cache, 8)        # one for each stream
        runs.append((torch.cuda.Stream(), want, outs, [b.prepared_decode_attention_q4(
            q, x.cache, dev(x.tab), dev(x.lens), 0.09, out=o, workspace=ws) for o in outs]))
    torch.cuda.synchronize()
    for i in range(20):
        for st, _, _, calls in runs:
            calls[i](st)
    torch.cuda.synchronize()
    for _, want, outs, _ in runs:
        for o in outs:
            assert torch.equal(o, want)
