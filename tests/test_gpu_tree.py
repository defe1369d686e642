"""Tree attention on the GPU against 64 bits: types, head layouts, lengths, splits, masks, what masks hide, refusals
by the device, streams and graphs.

Tolerance of an output element, with Z the largest scale * sum |q_d k_d| and V the largest |v| among what the row
sees, L its context. Products of 16-bit values are exact in fp32, and a sum of D <= 128 of them is off by at most
2^-23 of sum |q k| a step: a score by D 2^-23 Z <= 2^-16 Z, which moves softmax weights by as much, numerator and
denominator, so the output by 2 2^-16 Z * 2 V / 2 (the weights' mean moves within [-V, V]). Weights enter the second product with 16 bits
or more (off by 2^-16 at most), 2^x is off by 2^-22, a weight's exponent by 2^-23 times its size (at most ~2^7 for a
weight that counts: 2^-16); the second sum takes L / 16 + 16 steps of 2^-23 and rescalings of 2^-23 each. Together
below V (2^-15 Z + 2^-15 + (L / 8 + 64) 2^-22), then half a step of the output's type. fp32: sums of D products,
2^-24 of sum |q k| each step and product: within the same bound."""
import math

import numpy as np
import pytest
import torch

from oracle import tree_ops as O
from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def randn(shape, dt, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(DT[dt]).cuda()


def parents_of(rng, n, wide):
    return np.array([-1 if i == 0 else (int(rng.integers(0, i)) if rng.random() < wide else i - 1) for i in range(n)],
                    np.int32)


class Batch:
    """A batch of contexts of P tokens with n drafted ones behind."""

    def __init__(self, P, n, G=4, Hk=2, D=128, B=16, dt="bf16", seed=0, wide=0.5, words=None, spare_rows=0, std=1.0):
        rng = np.random.default_rng(seed)
        self.P, self.n = np.asarray(P), np.asarray(n)
        self.lens = self.P + self.n
        S = len(self.lens)
        self.Hq, self.Hk, self.D, self.B, self.dt = G * Hk, Hk, D, B, dt
        self.offs = np.concatenate([[0], np.cumsum(self.n)]).astype(np.int32)
        T = int(self.offs[-1]) + spare_rows
        blocks = -(-self.lens // B)
        self.M = int(blocks.max(initial=0)) + 1
        self.NB = int(blocks.sum()) + 2
        perm = rng.permutation(self.NB)
        self.tab = np.full((S, self.M), -1, np.int32)
        self.tab[np.arange(self.M)[None, :] < blocks[:, None]] = perm[: int(blocks.sum())]
        self.parents = np.concatenate([parents_of(rng, m, wide) for m in self.n] + [np.zeros(spare_rows, np.int32)]).astype(np.int32)
        self.W = words or max(1, -(-int(self.n.max(initial=1)) // 64))
        self.masks = np.zeros((T, self.W), np.int64)
        for s in range(S):
            self.masks[self.rows(s)] = O.words(O.ancestors(self.parents[self.rows(s)]), self.W)
        self.q = randn((T, self.Hq, D), dt, seed + 1, std)
        self.k, self.v = (randn((self.NB, Hk, B, D), dt, seed + i) for i in (2, 3))
        dead = np.ones((self.NB, B), bool)               # what no context holds
        for s in range(S):
            for j in range(blocks[s]):
                dead[self.tab[s, j], : max(0, min(B, self.lens[s] - j * B))] = False
        for p in (self.k, self.v):
            p.masked_fill_(dev(dead)[:, None, :, None], math.nan)
        self.scale = 1 / math.sqrt(D)

    def rows(self, s):
        return slice(int(self.offs[s]), int(self.offs[s + 1]))

    def place(self, s, j):
        """Block and offset of the j-th drafted token."""
        at = int(self.P[s]) + j
        return int(self.tab[s, at // self.B]), at % self.B

    def args(self, masks=True):
        return (self.q, self.k, self.v, dev(self.tab), dev(self.lens, torch.int32), dev(self.offs),
                dev(self.masks) if masks else None, self.scale)

    def run(self, masks=True, out_dtype=torch.float32, max_tree=None, fill=None, **kw):
        out = torch.full(self.q.shape, 77.0 if fill is None else fill, dtype=out_dtype, device="cuda")
        b.decode_attention_tree(*self.args(masks), max_tree=max_tree or max(1, int(self.n.max(initial=1))), out=out, **kw)
        return out

    def sees(self, s, masks=True):
        n, P = int(self.n[s]), int(self.P[s])
        seen = np.zeros((n, P + n), bool)
        seen[:, :P] = True
        if masks:
            w = self.masks[self.rows(s)].view(np.uint64)
            seen[:, P:] = np.array([[w[i, j // 64] >> np.uint64(j % 64) & np.uint64(1) for j in range(n)] for i in range(n)], bool).reshape(n, n)
        else:
            seen[:, P:] = np.tril(np.ones((n, n), bool))
        return seen

    def check(self, out, masks=True, lse=None, only=None):
        for s in range(len(self.lens)) if only is None else only:
            n, L = int(self.n[s]), int(self.lens[s])
            if n == 0:
                continue
            tab = dev(self.tab[s])
            k, v = O.rows_of(self.k, tab, L), O.rows_of(self.v, tab, L)
            seen = dev(self.sees(s, masks))
            want, wl, Z, V = O.attend(self.q[self.rows(s)], k, v, seen, self.scale)
            tol = V * (2.0 ** -15 * Z + 2.0 ** -15 + (L / 8 + 64) * 2.0 ** -22) + want.abs() * torch.finfo(out.dtype).eps / 2
            if out.dtype == torch.float16:
                tol = tol + 2.0 ** -25
            got = out[self.rows(s)].double()
            bad = ~((got - want).abs() <= tol)
            assert not bad.any(), (s, int(bad.sum()), torch.nonzero(bad)[:4].tolist(), float((got - want).abs().max()))
            if lse is not None:
                g = lse[self.rows(s)].double()
                none = torch.isinf(wl)
                assert torch.equal(torch.isinf(g) & (g < 0), none)
                # a score's error in units of log2, and the sum's
                assert ((g - wl).abs()[~none] <= 2.0 ** -15 * Z + 2.0 ** -15 + (L / 8 + 64) * 2.0 ** -22).all()


SHAPES = [
    dict(P=[0], n=[1]), dict(P=[5], n=[3], G=1, Hk=1), dict(P=[127], n=[1], G=8, Hk=1), dict(P=[100, 0, 300], n=[7, 5, 16]),
    dict(P=[1000], n=[33], G=4, Hk=3), dict(P=[130, 17, 64, 1], n=[64, 1, 0, 40], G=5, Hk=2),
    dict(P=[700, 90], n=[100, 250], G=2, Hk=1), dict(P=[33], n=[256], G=3, Hk=1), dict(P=[260], n=[20], G=12, Hk=1),
    dict(P=[3000, 40, 1100], n=[12, 13, 60], G=4, Hk=2),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_matches_64_bits(shape, D, dt):
    for B in (8, 16, 32):
        x = Batch(D=D, B=B, dt=dt, seed=shape, **SHAPES[shape])
        lse = torch.full(x.q.shape[:2], 5.0, device="cuda")
        x.check(x.run(lse_out=lse), lse=lse)
    x.check(x.run(masks=False), masks=False)
    x.check(x.run(out_dtype=DT[dt]))
    assert b.get_error() == 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("ctas", [1, 2, 3, 7, 40, 151, 600])
def test_any_split(ctas, dt):
    x = Batch([3000, 1, 777, 128, 0, 250], [17, 5, 40, 128, 9, 0], G=4, Hk=2, dt=dt, seed=ctas)
    ref = x.run(num_ctas=ctas)
    x.check(ref)
    for _ in range(3):                                    # equal inputs give equal bits
        assert torch.equal(x.run(num_ctas=ctas), ref)
    assert b.get_error() == 0


def test_bound_far_above_the_tokens_and_wide_masks():
    x = Batch([400, 30], [5, 9], G=4, Hk=2, words=4)
    x.check(x.run(max_tree=256))
    y = Batch([400, 30], [5, 9], G=40, Hk=1, dt="f16", words=2)
    y.check(y.run(max_tree=100))
    assert b.get_error() == 0


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_rows_that_see_nothing_and_any_masks(dt):
    rng = np.random.default_rng(3)
    x = Batch([0, 0, 500, 200], [6, 70, 30, 1], G=4, Hk=2, dt=dt)
    x.masks = rng.integers(-(1 << 63), 1 << 63, x.masks.shape, dtype=np.int64)      # bits past n say nothing
    x.masks[[0, 3]] = 0                                   # no context before and nothing shown
    x.masks[80] = 0                                       # the context alone
    lse = torch.zeros(x.q.shape[:2], device="cuda")
    for ctas in (0, 1, 5):
        out = x.run(lse_out=lse, num_ctas=ctas)
        x.check(out, lse=lse)
        assert (out[[0, 3]] == 0).all()


@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [128, 64])
def test_hidden_infinities_and_nans_reach_nobody(D, dt, what):
    # drafted tokens with such K and V, seen by themselves alone
    for P, n, G in (([0, 300, 90], [5, 40, 20], 4), ([100], [130], 2)):
        x = Batch(P, n, G=G, D=D, dt=dt, wide=1.0)
        bad = []
        for s in range(len(P)):
            for j in range(1, x.n[s], 3):
                row = int(x.offs[s]) + j
                bad.append(row)
                blk, off = x.place(s, j)
                x.k[blk, :, off] = what
                x.v[blk, :, off] = what
                for i in range(x.n[s]):
                    if i != j:
                        x.masks[int(x.offs[s]) + i, j // 64] &= ~np.int64(np.uint64(1 << (j % 64)).view(np.int64))
        out = x.run()
        good = np.setdiff1d(np.arange(x.q.shape[0]), bad)
        assert torch.isfinite(out[good]).all()
        for s in range(len(P)):
            seen = dev(x.sees(s))
            tab = dev(x.tab[s])
            k, v = O.rows_of(x.k, tab, int(x.lens[s])), O.rows_of(x.v, tab, int(x.lens[s]))
            local = [r - int(x.offs[s]) for r in good if x.offs[s] <= r < x.offs[s + 1]]
            want, _, Z, V = O.attend(x.q[x.rows(s)][local], k, v, seen[local], x.scale)
            tol = V * (2.0 ** -15 * Z + 2.0 ** -15 + (int(x.lens[s]) / 8 + 64) * 2.0 ** -22)
            assert ((out[x.rows(s)][local].double() - want).abs() <= tol).all()
    # seen V, not K: infinities reach exactly the rows that see them
    x = Batch([200], [30], G=4, D=D, dt=dt, wide=0.5)
    blk, off = x.place(0, 4)
    x.v[blk, :, off] = what
    out, seen = x.run(), x.sees(0)[:, 200 + 4]
    assert torch.isfinite(out[~seen]).all() and not torch.isfinite(out[seen]).any()
    if not math.isnan(what):
        assert (out[seen] == what).all()


def test_large_scores_and_growing_maxima():
    # maxima that rise and fall from tile to tile, weights that vanish
    for dt in ("bf16", "f16", "f32"):
        x = Batch([2000, 515], [16, 40], dt=dt, std=8.0)
        x.scale = 0.5
        for ctas in (0, 1):
            out = x.run(num_ctas=ctas)
            for s in range(2):
                tab = dev(x.tab[s])
                k, v = O.rows_of(x.k, tab, int(x.lens[s])), O.rows_of(x.v, tab, int(x.lens[s]))
                want, _, Z, V = O.attend(x.q[x.rows(s)], k, v, dev(x.sees(s)), x.scale)
                assert ((out[x.rows(s)].double() - want).abs() <= V * (2.0 ** -15 * Z + 2.0 ** -15 + 400 * 2.0 ** -22)).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_behind_the_last_sequence_stay(dt):
    x = Batch([40, 600], [3, 20], dt=dt, spare_rows=50)
    x.q[23:] = math.nan
    lse = torch.full(x.q.shape[:2], 3.0, device="cuda")
    out = x.run(lse_out=lse)
    x.check(out, lse=lse)
    assert (out[23:] == 77).all() and (lse[23:] == 3).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_bad_lengths_and_offsets_leave_sequences_out(dt):
    x = Batch([40, 600, 10, 33], [3, 20, 4, 9], dt=dt)
    q, k, v, tab, lens, offs, masks, scale = x.args()
    for change, bit in (((1, -1), b.DEVERR_CONTEXT), ((1, x.M * x.B + 1), b.DEVERR_CONTEXT), ((2, 3), b.DEVERR_TOKENS)):
        l2 = lens.clone()
        l2[change[0]] = change[1]
        out = torch.full(x.q.shape, 77.0, device="cuda")
        b.decode_attention_tree(q, k, v, tab, l2, offs, masks, scale, max_tree=20, out=out)
        assert b.get_error() == bit
        assert (out[x.rows(change[0])] == 77).all()
        x.check(out, only=[s for s in range(4) if s != change[0]])
    out = torch.full(x.q.shape, 77.0, device="cuda")     # more tokens than the bound
    b.decode_attention_tree(q, k, v, tab, lens, offs, masks, scale, max_tree=19, out=out)
    assert b.get_error() == b.DEVERR_TOKENS and (out[x.rows(1)] == 77).all()
    x.check(out, only=[0, 2, 3])
    for bad in ([0, 3, 2, 27, 36], [-1, 3, 23, 27, 36], [0, 3, 23, 27, 1 << 30], [0, 3, 23, 27, 37]):
        o2 = dev(np.array(bad, np.int32))
        b.decode_attention_tree(q, k, v, tab, lens, o2, masks, scale, max_tree=64, out=out)
        assert b.get_error() & b.DEVERR_TOKENS


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_bad_block_ids_read_as_zeros(dt):
    x = Batch([300, 50], [10, 6], dt=dt)
    good = x.tab.copy()
    x.tab[0, 3], x.tab[1, 0] = -5, x.NB
    out = x.run()
    assert b.get_error() == b.DEVERR_BLOCK_ID
    x.check(out)
    x.tab = good
    x.check(x.run())
    assert b.get_error() == 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_more_sequences_than_one_launch(dt):
    rng = np.random.default_rng(5)
    n = rng.integers(0, 5, 2500)
    x = Batch(rng.integers(0, 60, 2500), n, G=2, Hk=1, D=64, dt=dt)
    out = x.run()
    x.check(out, only=list(range(0, 2500, 97)) + [1023, 1024, 1025, 2047, 2048, 2499])
    assert b.get_error() == 0
    z = Batch([10, 20], [0, 0], dt=dt, spare_rows=4)
    assert (z.run(max_tree=4) == 77).all()


def test_pools_past_4_gb():
    # rows whose byte offsets pass 32 bits
    NB, Hk, B, D = 140000, 8, 16, 128
    k, v = (torch.empty(NB, Hk, B, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = [NB - 1, 7, NB - 3, 70001, 131072, 65535]
    x = Batch([80], [9], Hk=Hk, B=B, D=D)
    for src, dst in zip(x.tab[0], ids):
        k[dst], v[dst] = x.k[src], x.v[src]
    blocks = -(-89 // B)
    x.tab[0, :blocks] = ids[:blocks]
    x.k, x.v, x.NB = k, v, NB
    x.check(x.run())
    assert b.get_error() == 0


def test_streams_graphs_and_two_calls_at_once():
    xs = [Batch([900, 77], [20, 64], seed=1), Batch([50, 2000, 1], [3, 10, 30], G=8, Hk=1, dt="f16", seed=2)]
    refs = [x.run() for x in xs]
    outs = [torch.zeros_like(r) for r in refs]
    calls = [b.prepared_decode_attention_tree(*x.args(), max_tree=int(x.n.max()), out=o) for x, o in zip(xs, outs)]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        for c, st in zip(calls, sides):
            c(st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for o, r in zip(outs, refs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    for o in outs:
        o.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, r) for o, r in zip(outs, refs))
    # a one-shot call on another stream makes what it needs there
    st = torch.cuda.Stream()
    x = xs[0]
    out = b.decode_attention_tree(*x.args(), max_tree=64, out_dtype=torch.float32, stream=st)
    st.synchronize()
    assert torch.equal(out, refs[0])
    assert b.get_error() == 0


@pytest.mark.parametrize("scale", [-0.11, 0.0, 1.3])
@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
def test_any_scale(dt, scale):
    x = Batch([300, 0, 65], [12, 40, 1], dt=dt, seed=7)
    x.scale = scale
    lse = torch.zeros(x.q.shape[:2], device="cuda")
    for ctas in (0, 2):
        x.check(x.run(lse_out=lse, num_ctas=ctas), lse=lse)
    assert b.get_error() == 0


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_many_rows_a_kv_head(dt):
    x = Batch([100], [256], G=41, Hk=1, D=64, dt=dt, seed=3)          # 41 chunks of 256 rows
    x.check(x.run())
    y = Batch([700, 3], [9, 14], G=16, Hk=2, dt=dt, seed=4)           # 129..256 rows, and fewer
    for ctas in (0, 3):
        y.check(y.run(num_ctas=ctas))
    assert b.get_error() == 0


@pytest.mark.parametrize("G", [4, 20])
def test_a_wait_that_runs_out(G):
    # the first copy's arrival is withheld: the call ends, says so, and leaves nothing behind
    x = Batch([900, 40], [12, 7], G=G, dt="bf16", seed=9)
    ref = x.run()
    b.set_wait_fault(2_000_000, 1)
    x.run()
    status, word = b.get_error_status()
    b.set_wait_fault(0, 0)
    assert status == -5 and word & b.DEVERR_TIMEOUT
    assert torch.equal(x.run(), ref)
    b.set_wait_fault(2_000_000, 0)                         # the limit alone changes nothing
    assert torch.equal(x.run(), ref)
    b.set_wait_fault(0, 0)
    assert b.get_error() == 0


def test_back_to_back_steps_on_one_cache():
    # each call's rows are written by the call before it on the stream
    x = Batch([500, 64], [16, 5], seed=4)
    q, k, v, tab, lens, offs, masks, scale = x.args()
    slots = dev(np.concatenate([[x.place(s, j)[0] * x.B + x.place(s, j)[1] for j in range(x.n[s])] for s in range(2)]).astype(np.int64))
    new = [randn((21, x.Hk, x.D), "bf16", 50 + i) for i in range(6)]
    out = torch.empty(x.q.shape, device="cuda")
    call = b.prepared_decode_attention_tree(q, k, v, tab, lens, offs, masks, scale, max_tree=16, out=out)
    for i in range(0, 6, 2):
        b.append(new[i], new[i + 1], slots, k, v)
        call()
        x.check(out)


COUNTERS = 32768                       # bytes of counters, at the workspace's start


def test_one_workspace_for_calls_of_all_shapes():
    # the counters' region is one size, whatever the call, and every call leaves it zero
    xs = [(Batch([900, 40, 0], [12, 7, 1], G=4, dt="bf16", seed=1), 0), (Batch([700, 90], [30, 60], G=8, Hk=1, dt="f16", seed=2), 3),
          (Batch([500, 3], [9, 4], G=4, dt="f32", seed=3), 0), (Batch([3000], [16], G=20, D=64, dt="bf16", seed=4), 600)]
    ws = torch.zeros(max(b.tree_workspace_bytes(x.k, x.Hq, int(x.n.max()), c) for x, c in xs), dtype=torch.uint8, device="cuda")
    refs = [x.run(num_ctas=c) for x, c in xs]
    for _ in range(3):
        for (x, c), ref in zip(xs, refs):
            assert torch.equal(x.run(num_ctas=c, workspace=ws), ref)
            assert not ws[:COUNTERS].any()
    # two captured graphs of one workspace, replayed in turn
    outs, graphs = [torch.zeros_like(r) for r in refs[:2]], []
    for (x, c), o in zip(xs, outs):
        call = b.prepared_decode_attention_tree(*x.args(), max_tree=int(x.n.max()), out=o, workspace=ws, num_ctas=c)
        graphs.append((torch.cuda.CUDAGraph(), call))
        with torch.cuda.graph(graphs[-1][0]):
            call()
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g, _call in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(outs, refs))
    assert not ws[:COUNTERS].any() and b.get_error() == 0


@pytest.mark.parametrize("G", [4, 20])
def test_workspace_of_a_call_whose_wait_ran_out(G):
    x = Batch([900, 40], [12, 7], G=G, dt="f16", seed=9)
    ws = b.alloc_tree_workspace(x.k, x.Hq, 12)
    ref = x.run()
    b.set_wait_fault(2_000_000, 1)
    x.run(workspace=ws)
    status, word = b.get_error_status()
    b.set_wait_fault(0, 0)
    assert status == -5 and word & b.DEVERR_TIMEOUT
    ws[:COUNTERS].zero_()                                  # as the interface asks for
    for _ in range(2):
        assert torch.equal(x.run(workspace=ws), ref)
        assert not ws[:COUNTERS].any()


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("D", [128, 64])
@pytest.mark.parametrize("ctas", [1, 2, 5])
def test_large_and_small_units_by_turns(ctas, D, dt):
    # units of two row tiles and of one follow each other in a worker's share: one group runs ahead of the other
    rng = np.random.default_rng(ctas)
    n = np.where(np.arange(90) % 3 == 0, rng.integers(33, 65, 90), rng.integers(1, 9, 90))
    P = rng.integers(0, 200, 90)
    P[1::9] = 1500
    for B in (8, 32):
        x = Batch(P, n, G=4, Hk=1, D=D, B=B, dt=dt, seed=ctas)
        ref = x.run(num_ctas=ctas)
        x.check(ref)
        assert torch.equal(x.run(num_ctas=ctas), ref)
    assert b.get_error() == 0


class WideTable(Batch):
    """The same with tables far wider than the contexts: units may have two row tiles."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        spare = 4608 // self.B
        self.M += spare
        self.tab = np.pad(self.tab, ((0, 0), (0, spare)), constant_values=-1)


@pytest.mark.parametrize("what, args", [(test_matches_64_bits, (s, D, dt)) for s in (5, 6, 7, 8) for D in (64, 128) for dt in ("f16", "bf16")]
                         + [(test_any_split, (c, "bf16")) for c in (1, 3, 40, 151, 600)]
                         + [(test_bound_far_above_the_tokens_and_wide_masks, ())]
                         + [(test_rows_that_see_nothing_and_any_masks, (dt,)) for dt in ("f16", "bf16")]
                         + [(test_hidden_infinities_and_nans_reach_nobody, (D, dt, w)) for D, dt, w in
                            ((128, "f16", math.inf), (128, "bf16", math.nan), (64, "bf16", -math.inf), (64, "f16", math.nan))]
                         + [(test_large_scores_and_growing_maxima, ()), (test_bad_block_ids_read_as_zeros, ("f16",)),
                            (test_any_scale, ("bf16", -0.11)), (test_a_wait_that_runs_out, (20,)),
                            (test_workspace_of_a_call_whose_wait_ran_out, (20,)), (test_one_workspace_for_calls_of_all_shapes, ())]
                         + [(test_many_rows_a_kv_head, (dt,)) for dt in ("f16", "bf16")]
                         + [(test_large_and_small_units_by_turns, (c, D, "bf16")) for c in (1, 2, 5) for D in (64, 128)])
def test_wide_tables(monkeypatch, what, args):
    monkeypatch.setitem(globals(), "Batch", WideTable)
    what(*args)


def test_one_workspace_for_any_width_of_table():
    for x in (Batch([700, 90], [40, 60], G=4), WideTable([700, 90], [40, 60], G=4)):
        ws = b.alloc_tree_workspace(x.k, x.Hq, 60)
        for _ in range(2):
            x.check(x.run(workspace=ws))
    assert not ws[:COUNTERS].any() and b.get_error() == 0
