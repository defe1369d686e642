"""Device block tables on the GPU against the plain implementation: every output, in place and out
of place, one CTA and many, refusals that change nothing, and a serving loop with the host block
manager beside it."""
import numpy as np
import pytest
import torch

from oracle import step_ops as O
from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


class State:
    def __init__(self, rng, S, M, B, lens, spare=50, NB=None):
        n = -(-np.asarray(lens) // B)
        NB = NB or int(n.sum()) + spare
        perm = rng.permutation(NB).astype(np.int32)
        self.tab = np.full((S, M), -1, np.int32)
        self.tab[np.arange(M)[None, :] < n[:, None]] = perm[: int(n.sum())]
        self.lens = np.asarray(lens, np.int32)
        self.nf = NB - int(n.sum())
        self.free = np.full(NB, -7, np.int32)
        self.free[: self.nf] = perm[int(n.sum()):]
        self.B, self.M, self.NB = B, M, NB

    def device(self):
        return dev(self.tab), dev(self.lens), dev(self.free), dev(np.array([self.nf], np.int32))


def run_append(st, add, max_tokens, in_place=False):
    tab, lens, free, nf = st.device()
    S = len(st.lens)
    slots = torch.full((max_tokens,), 99, dtype=torch.int64, device="cuda")
    pos = torch.full((max_tokens,), 99, dtype=torch.int32, device="cuda")
    offs = torch.full((S + 1,), 99, dtype=torch.int32, device="cuda")
    ws = b.alloc_tables_workspace()
    lo = lens if in_place else torch.full_like(lens, 99)
    no = nf if in_place else torch.full_like(nf, 99)
    b.tables_append(tab, lens, dev(np.asarray(add, np.int32)), free, nf, st.B, slots, pos, offs, ws,
                    context_lens_out=lo, num_free_out=no)
    err = b.get_error()
    assert not ws.any()
    if not in_place:
        assert (lens.cpu().numpy() == st.lens).all() and int(nf) == st.nf
    assert (free.cpu().numpy() == st.free).all()
    return err, [x.cpu().numpy() for x in (tab, lo, no, slots, pos, offs)]


def check_append(st, add, max_tokens, in_place=False):
    err, got = run_append(st, add, max_tokens, in_place)
    tab, lens, nf, slots, pos, offs = O.tables_append(st.tab, st.lens, np.asarray(add, np.int32), st.free, st.nf,
                                                      st.B, max_tokens)
    assert err == 0
    for g, w in zip(got, (tab, lens, [nf], slots, pos, offs)):
        np.testing.assert_array_equal(g, w)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("S,hi,add_hi", [(1, 0, 1), (1, 100, 300), (3, 40, 0), (64, 500, 1), (513, 90, 40),
                                         (1300, 30, 9), (40, 0, 3000)])
def test_append_matches_oracle(S, hi, add_hi, B, in_place):
    rng = np.random.default_rng([S, hi, add_hi, B])
    lens, add = rng.integers(0, hi + 1, S), rng.integers(0, add_hi + 1, S)
    if S == 64:
        add[:] = 1
        lens[:4] = 0, B - 1, B, 2 * B - 1          # around a block's end
    M = (hi + add_hi) // B + 2
    st = State(rng, S, M, B, lens, spare=int((-(-(lens + add) // B)).sum()) + 1)
    check_append(st, add, int(add.sum()) + int(rng.integers(0, 70)), in_place)


@pytest.mark.parametrize("shift", [0, 1])
def test_append_many_ctas_and_unaligned_buffers(shift):
    # token buffers that begin 8 (4) bytes past a 16-byte boundary
    rng = np.random.default_rng(9)
    S, B, M = 700, 16, 30
    lens, add = rng.integers(0, 200, S), rng.integers(0, 60, S)
    st = State(rng, S, M, B, lens, spare=4000)
    T = int(add.sum()) + 7
    tab, ln, free, nf = st.device()
    slots = torch.full((T + 2,), 99, dtype=torch.int64, device="cuda")
    pos = torch.full((T + 2,), 99, dtype=torch.int32, device="cuda")
    offs = torch.empty(S + 1, dtype=torch.int32, device="cuda")
    v = slice(shift, shift + T)
    for _ in range(2):                               # twice in place: the second continues from the first
        b.tables_append(tab, ln, dev(add.astype(np.int32)), free, nf, B, slots[v], pos[v], offs, b.alloc_tables_workspace())
        assert b.get_error() == 0
        st.tab, st.lens, st.nf, ws, wp, wo = O.tables_append(st.tab, st.lens, add.astype(np.int32), st.free, st.nf, B, T)
        np.testing.assert_array_equal(slots[v].cpu().numpy(), ws)
        np.testing.assert_array_equal(pos[v].cpu().numpy(), wp)
        np.testing.assert_array_equal(offs.cpu().numpy(), wo)
        np.testing.assert_array_equal(ln.cpu().numpy(), st.lens)
        assert int(nf) == st.nf
        assert (slots[:shift] == 99).all() and (slots[shift + T:] == 99).all() and (pos[shift + T:] == 99).all()


def test_append_exact_fits():
    rng = np.random.default_rng(0)
    # every free block, every table entry and every token entry used
    st = State(rng, 2, 4, 8, [3, 8], spare=6)
    check_append(st, [29, 24], 53)


def test_append_no_requests_and_no_tokens():
    rng = np.random.default_rng(0)
    st = State(rng, 2, 4, 8, [3, 8])
    check_append(st, [0, 0], 0)
    check_append(st, [0, 0], 9)
    z = State(rng, 0, 4, 8, np.zeros(0, np.int64))
    check_append(z, np.zeros(0), 5)


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("what,bit", [("blocks", b.DEVERR_NO_BLOCKS), ("tokens", b.DEVERR_TOKENS),
                                      ("negative", b.DEVERR_TOKENS), ("row", b.DEVERR_CONTEXT),
                                      ("length", b.DEVERR_CONTEXT), ("free", b.DEVERR_NO_BLOCKS)])
def test_append_refused_changes_nothing(what, bit, many):
    rng = np.random.default_rng(1)
    S = 200
    lens, add = rng.integers(0, 60, S), rng.integers(1, 30, S)
    st = State(rng, S, 24, 8, lens, spare=2000)
    if many:
        add *= 4                                     # more tokens than one CTA's share: many CTAs
    T = int(add.sum()) + 5
    if what == "blocks":
        st.nf = 3
    elif what == "tokens":
        T = int(add.sum()) - 1
    elif what == "negative":
        add[77] = -1
    elif what == "row":
        add[77] = 193
    elif what == "length":
        st.lens[5] = -2
    else:
        st.nf = st.NB + 1
    for in_place in (False, True):
        err, (tab, lo, no, slots, pos, offs) = run_append(st, add, T, in_place)
        assert err & bit
        np.testing.assert_array_equal(tab, st.tab)
        np.testing.assert_array_equal(lo, st.lens)
        assert no[0] == st.nf
        assert (slots == -1).all() and not pos.any() and not offs.any()


def test_append_bad_block_ids_give_no_slot():
    rng = np.random.default_rng(2)
    st = State(rng, 3, 6, 8, [5, 8, 12], spare=10)
    st.tab[0, 0] = st.NB                         # the block token 5 of request 0 falls into
    st.free[st.nf - 1] = -3                      # the first block taken
    err, (tab, lo, no, slots, pos, offs) = run_append(st, [4, 1, 1], 8)
    assert err == b.DEVERR_BLOCK_ID
    want = O.tables_append(st.tab, st.lens, np.array([4, 1, 1], np.int32), st.free, st.nf, 8, 8)
    bad = (want[3] < 0) | (want[3] >= st.NB * 8)
    assert bad[:4].all() and not bad[4:6].any()
    np.testing.assert_array_equal(slots, np.where(bad, -1, want[3]))
    np.testing.assert_array_equal(lo, want[1])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("S,hi", [(1, 7), (5, 0), (64, 3000), (1500, 100)])
def test_release_matches_oracle(S, hi, in_place):
    rng = np.random.default_rng([S, hi])
    st = State(rng, S, hi // 16 + 1, 16, rng.integers(0, hi + 1, S))
    for share in (0.0, 0.3, 1.0):
        rel = rng.random(S) < share
        tab, lens, free, nf = st.device()
        ws = b.alloc_tables_workspace()
        lo = lens if in_place else torch.full_like(lens, 99)
        no = nf if in_place else torch.full_like(nf, 99)
        flags = dev(rel) if share else dev(rel.astype(np.uint8))
        b.tables_release(tab, lens, flags, free, nf, 16, ws, context_lens_out=lo, num_free_out=no)
        assert b.get_error() == 0 and not ws.any()
        wl, wf, wn = O.tables_release(st.tab, st.lens, rel, st.free, st.nf, 16)
        np.testing.assert_array_equal(lo.cpu().numpy(), wl)
        np.testing.assert_array_equal(free.cpu().numpy(), wf)
        assert int(no) == wn
        np.testing.assert_array_equal(tab.cpu().numpy(), st.tab)


def test_release_refused_changes_nothing():
    rng = np.random.default_rng(3)
    st = State(rng, 4, 8, 16, [100, 5, 60, 128])
    for nf, lens, bit in ((st.NB - 3, st.lens, b.DEVERR_NO_BLOCKS), (st.nf, st.lens - 6, b.DEVERR_CONTEXT),
                          (-1, st.lens, b.DEVERR_NO_BLOCKS)):
        tab, _, free, _ = st.device()
        n, ln, ws = dev(np.array([nf], np.int32)), dev(lens.astype(np.int32)), b.alloc_tables_workspace()
        b.tables_release(tab, ln, dev(np.ones(4, bool)), free, n, 16, ws)
        assert b.get_error() & bit
        assert int(n) == nf and (ln.cpu().numpy() == lens).all()
        np.testing.assert_array_equal(free.cpu().numpy(), st.free)


def test_loop_agrees_with_the_block_manager_and_replays_as_a_graph():
    rng = np.random.default_rng(5)
    NB, B, S, M, T = 300, 16, 12, 20, 700
    bm = b.BlockManager(NB, B)
    for s in range(S):
        bm.add_sequence(s)
    tab = torch.full((S, M), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(S, dtype=torch.int32, device="cuda")
    free, nf = dev(np.arange(NB, dtype=np.int32)[::-1]), dev(np.array([NB], np.int32))
    rel, add = torch.zeros(S, dtype=torch.bool, device="cuda"), torch.zeros_like(lens)
    slots = torch.empty(T, dtype=torch.int64, device="cuda")
    pos = torch.empty(T, dtype=torch.int32, device="cuda")
    offs = torch.empty(S + 1, dtype=torch.int32, device="cuda")
    ws = b.alloc_tables_workspace()
    calls = (b.prepared_tables_release(tab, lens, rel, free, nf, B, ws),
             b.prepared_tables_append(tab, lens, add, free, nf, B, slots, pos, offs, ws))
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for c in calls:                          # nothing to do yet: warms the kernels up
            c()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for c in calls:
            c()
    host = np.zeros(S, np.int64)
    for step in range(25):
        r = (rng.random(S) < 0.1) & (host > 0)
        host[r] = 0
        a = np.where(r, 0, np.minimum(rng.integers(0, 50, S), M * B - host))
        for s in np.flatnonzero(r):
            bm.free_sequence(int(s))
            bm.add_sequence(int(s))
        need = (-(-(host + a) // B) - -(-host // B)).sum()
        if need > bm.num_free():
            a[:] = 0
        host += a
        rel.copy_(torch.from_numpy(r))
        add.copy_(torch.from_numpy(a))
        graph.replay()
        want, _ = bm.append_batch(range(S), a.tolist())
        assert slots[: int(a.sum())].tolist() == want.tolist()
        assert (slots[int(a.sum()):] == -1).all()
        wt, wl = bm.block_tables(range(S), M)
        assert lens.tolist() == wl.tolist()
        live = torch.arange(M)[None, :] < ((wl + B - 1) // B)[:, None]
        assert (tab.cpu()[live] == wt[live]).all()
        assert int(nf) == bm.num_free()
    assert b.get_error() == 0
