"""Plans, acceptance, committed rows and truncated tables of drafted tokens on the GPU, exact against the plain
implementation; and a whole step of them, captured and replayed."""
import math

import numpy as np
import pytest
import torch

from oracle import step_ops as SO
from oracle import tree_ops as O
from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def trees(rng, n, wide, roots=0.0):
    out = []
    for m in n:
        p = [-1 if i == 0 or rng.random() < roots else (int(rng.integers(0, i)) if rng.random() < wide else i - 1) for i in range(m)]
        out.append(np.array(p, np.int32))
    return out


def flat(xs):
    return np.concatenate([np.zeros(0, np.int32)] + list(xs)).astype(np.int32)


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int32)


# -------------------------------------------------------------------------------------- plan
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("wide,roots", [(0.0, 0.0), (0.5, 0.0), (1.0, 0.1)])
def test_plan(W, wide, roots):
    rng = np.random.default_rng([W, int(10 * wide)])
    n = np.concatenate([[0, 1, 2, 64 * W], rng.integers(0, 64 * W + 1, 60)])
    ps, offs = trees(rng, n, wide, roots), offsets(n)
    lens = n + rng.integers(0, 5000, len(n))
    deltas = rng.integers(-100, 100, len(n))
    T = int(offs[-1]) + 9
    for axes, use in ((1, False), (3, True)):
        masks = torch.full((T, W), 77, dtype=torch.int64, device="cuda")
        pos = torch.full((axes, T), 77, **I32)
        b.tree_plan(dev(np.concatenate([flat(ps), np.full(9, 1 << 20, np.int32)])), dev(offs), dev(lens, torch.int32), masks, pos,
                    position_deltas=dev(deltas, torch.int32) if use else None)
        assert b.get_error() == 0
        m, p = masks.cpu().numpy(), pos.cpu().numpy()
        for s, parents in enumerate(ps):
            a = O.ancestors(parents)
            r = slice(offs[s], offs[s + 1])
            np.testing.assert_array_equal(m[r], O.words(a, W))
            want = lens[s] - n[s] + (deltas[s] if use else 0) + a.sum(1) - 1
            for k in range(axes):
                np.testing.assert_array_equal(p[k, r], want)
        assert (m[offs[-1]:] == 77).all() and (p[:, offs[-1]:] == 77).all()


def test_plan_of_chains_and_of_one_output():
    n = np.array([5, 0, 130])
    offs, lens = dev(offsets(n)), dev(n + 7, torch.int32)
    masks, pos = torch.zeros(135, 4, dtype=torch.int64, device="cuda"), torch.zeros(135, **I32)
    b.tree_plan(None, offs, lens, masks, pos)
    m2, p2 = torch.zeros_like(masks), torch.zeros_like(pos)
    chain = dev(flat([np.arange(k) - 1 for k in n]))
    b.tree_plan(chain, offs, lens, masks=m2)
    b.tree_plan(chain, offs, lens, positions=p2)
    assert torch.equal(masks, m2) and torch.equal(pos, p2)
    assert pos.tolist() == list(range(7, 12)) + list(range(7, 137))
    assert b.get_error() == 0


def test_plan_flags_what_is_wrong():
    offs, lens = dev(np.array([0, 3, 6], np.int32)), dev(np.array([5, 9], np.int32))
    masks, pos = torch.full((6, 1), 7, dtype=torch.int64, device="cuda"), torch.full((6,), 7, **I32)
    b.tree_plan(dev(np.array([-1, 1, -2, -1, 0, 3], np.int32)), offs, lens, masks, pos)
    assert b.get_error() == b.DEVERR_TREE
    assert masks[:, 0].tolist() == [1, 2, 4, 1, 3, 4] and pos.tolist() == [2, 2, 2, 6, 7, 6]
    masks.fill_(7)
    for l, o, bit in (([2, 9], [0, 3, 6], b.DEVERR_TOKENS), ([-1, 9], [0, 3, 6], b.DEVERR_CONTEXT),
                      ([5, 9], [4, 3, 6], b.DEVERR_TOKENS)):
        masks.fill_(7)
        b.tree_plan(None, dev(np.array(o, np.int32)), dev(np.array(l, np.int32)), masks)
        assert b.get_error() == bit
        assert masks[:, 0].tolist() == [7, 7, 7, 1, 3, 7]
    masks = torch.full((70, 1), 7, dtype=torch.int64, device="cuda")
    b.tree_plan(None, dev(np.array([0, 65, 70], np.int32)), dev(np.array([90, 9], np.int32)), masks)
    assert b.get_error() == b.DEVERR_TOKENS and (masks[:65] == 7).all() and masks[65:, 0].tolist() == [1, 3, 7, 15, 31]


# ------------------------------------------------------------------------------------ accept
@pytest.mark.parametrize("most", [1, 16, 64, 65, 200, 256])
@pytest.mark.parametrize("right,wide,roots", [(0.0, 0.5, 0.0), (0.8, 0.3, 0.0), (1.0, 1.0, 0.2), (0.9, 0.0, 0.0)])
def test_accept(most, right, wide, roots):
    rng = np.random.default_rng([most, int(10 * right)])
    n = np.concatenate([[0, 1, most], rng.integers(0, most + 1, 40)])
    ps, offs = trees(rng, n, wide, roots), offsets(n)
    T = int(offs[-1]) + 5
    few = rng.integers(2, 9)                              # tokens that repeat: several children may hold
    tokens, targets = (rng.integers(0, few, T).astype(np.int32) for _ in range(2))
    for s, parents in enumerate(ps):
        for i, p in enumerate(parents):
            if p >= 0 and rng.random() < right:
                tokens[offs[s] + i] = targets[offs[s] + p]
    lens = n + rng.integers(0, 1000, len(n))
    path = torch.full((T,), 77, **I32)
    got = b.tree_accept(dev(np.concatenate([flat(ps), np.zeros(5, np.int32)])), dev(tokens), dev(targets), dev(offs),
                        dev(lens, torch.int32), max_tree=most, path=path)
    assert b.get_error() == 0
    path, counts, nxt, out = (t.cpu().numpy() for t in got)
    for s, parents in enumerate(ps):
        r = slice(offs[s], offs[s + 1])
        want, answer = O.accept(parents, tokens[r], targets[r])
        assert path[r].tolist() == want + [-1] * (n[s] - len(want)), s
        assert counts[s] == len(want) and nxt[s] == answer and out[s] == lens[s] - n[s] + len(want)
    assert (path[offs[-1]:] == 77).all()


def test_accept_chains_in_place_and_bad_input():
    n = np.array([3, 4])
    offs = dev(offsets(n))
    lens = dev(np.array([10, 4], np.int32))
    tokens = dev(np.array([5, 6, 7, 1, 2, 3, 4], np.int32))
    targets = dev(np.array([6, 9, 9, 2, 3, 4, 8], np.int32))
    path, counts, nxt, out = b.tree_accept(None, tokens, targets, offs, lens, max_tree=4, context_lens_out=lens)
    assert path.tolist() == [0, 1, -1, 0, 1, 2, 3] and counts.tolist() == [2, 4] and nxt.tolist() == [9, 8]
    assert lens.tolist() == [9, 4] and b.get_error() == 0
    # a bad parent does not hold, nor what hangs on it; a bad sequence has nothing
    lens = dev(np.array([10, 2], np.int32))
    path = torch.full((7,), 77, **I32)
    p = dev(np.array([-1, 1, 1, -1, 0, 1, 2], np.int32))
    path, counts, nxt, out = b.tree_accept(p, tokens, targets, offs, lens, max_tree=4, path=path)
    assert b.get_error() == b.DEVERR_TREE | b.DEVERR_TOKENS
    assert path.tolist() == [0, -1, -1, 77, 77, 77, 77] and counts.tolist() == [1, 0]
    assert nxt.tolist() == [6, -1] and out.tolist() == [8, 2]


# ------------------------------------------------------------------------------------ commit
@pytest.mark.parametrize("dt", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hk", [1, 3, 40])
def test_commit(Hk, D, dt):
    for B in (8, 16, 32):
        rng = np.random.default_rng([Hk, D, B])
        n = np.concatenate([[0, 1, 256, 17], rng.integers(0, 65, 12)])
        P = rng.integers(0, 100, len(n))
        lens = P + n
        blocks = -(-lens // B)
        NB, M = int(blocks.sum()) + 2, int(blocks.max()) + 1
        tab = np.full((len(n), M), -1, np.int32)
        tab[np.arange(M)[None, :] < blocks[:, None]] = rng.permutation(NB)[: int(blocks.sum())]
        offs = offsets(n)
        path, counts = np.full(int(offs[-1]), -1, np.int32), np.zeros(len(n), np.int32)
        for s, m in enumerate(n):
            some = np.sort(rng.permutation(m)[: rng.integers(0, m + 1)]) if s % 3 else np.arange(m)[m % 2:]
            counts[s] = len(some)
            path[offs[s]: offs[s] + len(some)] = some
        k, v = (torch.randn(NB, Hk, B, D, generator=torch.Generator().manual_seed(i)).to(dt) for i in (1, 2))
        kd, vd = k.cuda(), v.cuda()
        b.tree_commit(dev(path), dev(counts), dev(offs), dev(lens, torch.int32), dev(tab), kd, vd, max_tree=256)
        assert b.get_error() == 0
        for x in (k, v):
            old = x.clone()
            for s in range(len(n)):
                for i in range(counts[s]):
                    a, z = P[s] + path[offs[s] + i], P[s] + i
                    x[tab[s, z // B], :, z % B] = old[tab[s, a // B], :, a % B]
        assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)


def test_commit_refuses_bad_paths_and_blocks():
    B, tab = 8, np.array([[0, 1], [2, 3]], np.int32)
    k0 = torch.arange(6 * 2 * B * 64, dtype=torch.float32).reshape(6, 2, B, 64)
    offs, lens = dev(np.array([0, 6, 12], np.int32)), dev(np.array([10, 12], np.int32))

    def go(path, counts, tab=tab, offs=offs, lens=lens, most=6):
        k = k0.clone().cuda()
        b.tree_commit(dev(np.array(path, np.int32)), dev(np.array(counts, np.int32)), offs, lens, dev(tab), k, k.clone(), max_tree=most)
        return b.get_error(), k.cpu()

    row = lambda x, s, at: x[tab[s][at // B], :, at % B]  # noqa: E731
    # the second step of sequence 0 goes down: the first is moved, nothing more; sequence 1 as asked
    err, k = go([2, 1, 4, 5, 0, 0, 0, 3, 5, 0, 0, 0], [4, 3])
    assert err == b.DEVERR_TREE
    assert torch.equal(row(k, 0, 4), row(k0, 0, 6)) and torch.equal(row(k, 0, 5), row(k0, 0, 5)) and torch.equal(row(k, 0, 6), row(k0, 0, 6))
    assert torch.equal(row(k, 1, 7), row(k0, 1, 9)) and torch.equal(row(k, 1, 8), row(k0, 1, 11))
    for path, counts, bit in (([0, 6] + [0] * 10, [2, 0], b.DEVERR_TREE), ([-1, 2] + [0] * 10, [2, 0], b.DEVERR_TREE),
                              ([0] * 12, [7, 0], b.DEVERR_TOKENS), ([0] * 12, [-1, 0], b.DEVERR_TOKENS)):
        err, k = go(path, counts)
        assert err == bit and torch.equal(k, k0)
    err, k = go([1, 2] + [0] * 10, [2, 0], tab=np.array([[99, 1], [2, 3]], np.int32))
    assert err == b.DEVERR_BLOCK_ID and torch.equal(k, k0)
    err, k = go([1, 2] + [0] * 10, [2, 0], lens=dev(np.array([17, 12], np.int32)))
    assert err == b.DEVERR_CONTEXT and torch.equal(k, k0)
    err, k = go([1, 2] + [0] * 10, [2, 0], most=5)
    assert err == b.DEVERR_TOKENS and torch.equal(k, k0)


# ---------------------------------------------------------------------------------- truncate
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("S,hi,cut", [(1, 90, 90), (5, 300, 20), (513, 60, 60), (1300, 300, 300), (64, 500, 0)])
def test_truncate(S, hi, cut, B, in_place):
    rng = np.random.default_rng([S, hi, B])
    lens = rng.integers(0, hi + 1, S)
    kept = np.maximum(0, lens - rng.integers(0, cut + 1, S))
    blocks = -(-lens // B)
    M, NB = int(blocks.max()) + 1, int(blocks.sum()) + 7
    perm = rng.permutation(NB).astype(np.int32)
    tab = np.full((S, M), -1, np.int32)
    tab[np.arange(M)[None, :] < blocks[:, None]] = perm[:-7]
    free = np.full(NB, -7, np.int32)
    free[:7] = perm[-7:]
    want = list(perm[-7:])
    for s in range(S):
        want += tab[s, -(-kept[s] // B): blocks[s]].tolist()
    ld, fd, nd, ws = dev(lens, torch.int32), dev(free), dev(np.array([7], np.int32)), b.alloc_tables_workspace()
    lo, no = (ld, nd) if in_place else (torch.full_like(ld, 99), torch.full_like(nd, 99))
    b.tables_truncate(dev(tab), ld, dev(kept, torch.int32), fd, nd, B, ws, context_lens_out=lo, num_free_out=no)
    assert b.get_error() == 0 and not ws.any()
    assert lo.tolist() == kept.tolist() and int(no) == len(want) and fd[: len(want)].tolist() == want
    assert (fd[len(want):] == -7).all()
    if not in_place:
        assert ld.tolist() == lens.tolist() and int(nd) == 7


def test_truncate_refuses_as_a_whole():
    tab, free = dev(np.array([[0, 1], [2, 3]], np.int32)), dev(np.array([5, 4, -1, -1, -1, -1], np.int32))
    lens, nf, ws = dev(np.array([9, 16], np.int32)), dev(np.array([2], np.int32)), b.alloc_tables_workspace()
    for kept, nfree, bit in (([9, 17], 2, b.DEVERR_CONTEXT), ([-1, 3], 2, b.DEVERR_CONTEXT), ([0, 0], 3, b.DEVERR_NO_BLOCKS)):
        nf.fill_(nfree)
        b.tables_truncate(tab, lens, dev(np.array(kept, np.int32)), free, nf, 8, ws)
        assert b.get_error() == bit and lens.tolist() == [9, 16] and int(nf) == nfree
        assert free.tolist() == [5, 4, -1, -1, -1, -1]
    with pytest.raises(b.PkvError):
        b.tables_truncate(tab, lens, lens, free, nf, 8, ws)


# ------------------------------------------------------------------------------- a whole step
def test_graph_of_a_whole_verifying_step():
    """Tables, plan, rotation on three axes with append, tree attention, acceptance, commit, truncation, over and over
    as one graph; the host only writes the step's inputs."""
    S, Hq, Hk, D, B, M, NB, N = 4, 8, 2, 64, 8, 14, 64, 12
    T = 60 * S
    bf = torch.bfloat16
    rng = np.random.default_rng(1)
    scale = 1 / math.sqrt(D)
    sections = (8, 12, 12)
    plan = b.RopeAxesPlan(sections, order="cycled")
    axis, w, amp = SO.axes_frequencies(sections, "cycled", "shared", 10000.0)
    tab, lens = torch.full((S, M), -1, **I32), torch.zeros(S, **I32)
    full, kept = torch.zeros(S, **I32), torch.zeros(S, **I32)
    free, nf, add = torch.arange(NB - 1, -1, -1, **I32), torch.tensor([NB], **I32), torch.zeros(S, **I32)
    slots, pos, offs = torch.empty(T, dtype=torch.int64, device="cuda"), torch.zeros(3, T, **I32), torch.empty(S + 1, **I32)
    parents, tokens, targets, deltas = torch.zeros(T, **I32), torch.zeros(T, **I32), torch.zeros(T, **I32), torch.zeros(S, **I32)
    masks = torch.zeros(T, 1, dtype=torch.int64, device="cuda")
    qkv = torch.zeros(T, (Hq + 2 * Hk) * D, dtype=bf, device="cuda")
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
    kp, vp = (torch.zeros(NB, Hk, B, D, dtype=bf, device="cuda") for _ in range(2))
    qo, out = torch.empty(T, Hq, D, dtype=bf, device="cuda"), torch.empty(T, Hq, D, device="cuda")
    path, counts, nxt = torch.full((T,), -1, **I32), torch.zeros(S, **I32), torch.zeros(S, **I32)
    tws, ws = b.alloc_tables_workspace(), b.alloc_tree_workspace(kp, Hq, 60)

    def step():
        b.tables_append(tab, lens, add, free, nf, B, slots, pos[0], offs, tws, context_lens_out=full)
        b.tree_plan(parents, offs, full, masks, pos, position_deltas=deltas)
        b.rope_axes_append(q, k, v, pos, slots, plan, kp, vp, q_out=qo)
        b.decode_attention_tree(qo, kp, vp, tab, full, offs, masks, scale, max_tree=60, out=out, workspace=ws)
        b.tree_accept(parents, tokens, targets, offs, full, 60, path, counts, nxt, kept)
        b.tree_commit(path, counts, offs, full, tab, kp, vp, max_tree=60)
        b.tables_truncate(tab, full, kept, free, nf, B, tws, context_lens_out=lens)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert b.get_error() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    hist = [[np.zeros((0, Hk, D))] * 2 for _ in range(S)]         # kept keys (turned) and values, 64 bits
    for it in range(10):
        n = rng.integers(1, N + 1, S) if it else np.array([60, 33, 50, 20])       # prompts first, as chains
        n = np.minimum(n, M * B - np.array([len(h[0]) for h in hist]))
        ps = trees(rng, n, 0.0 if it == 0 else 0.5)
        o, total = offsets(n), int(n.sum())
        tk, tg = rng.permutation(1000)[:T].astype(np.int32), (1000 + rng.permutation(1000)[:T]).astype(np.int32)
        for s, p in enumerate(ps):
            for i in range(1, n[s]):
                if it == 0 or rng.random() < 0.7:
                    tg[o[s] + p[i]] = tk[o[s] + i]
        dl = rng.integers(-20, 20, S)
        for t, x in ((add, n), (tokens, tk), (targets, tg), (deltas, dl)):
            t.copy_(torch.from_numpy(x.astype(np.int32)))
        parents[:total].copy_(torch.from_numpy(flat(ps)))
        qkv.copy_(torch.randn(qkv.shape, generator=torch.Generator().manual_seed(it)).to(bf))
        graph.replay()
        assert b.get_error() == 0
        rows = [x[:total].double().cpu().numpy() for x in (q, k, v)]
        where = np.concatenate([len(hist[s][0]) + dl[s] + O.ancestors(ps[s]).sum(1) - 1 for s in range(S)])
        assert pos.cpu().numpy()[:, :total].tolist() == [where.tolist()] * 3
        turned = [SO.rope(x, where, w, amp, "half")[0] for x in rows[:2]]
        for s in range(S):
            r = slice(o[s], o[s + 1])
            kk, vv = (torch.from_numpy(np.concatenate([h, x[r]])).transpose(0, 1) for h, x in zip(hist[s], (turned[1], rows[2])))
            L0 = len(hist[s][0])
            seen = np.ones((n[s], L0 + n[s]), bool)
            seen[:, L0:] = O.ancestors(ps[s])
            want, _, Z, V = O.attend(torch.from_numpy(turned[0][r]), kk, vv, torch.from_numpy(seen), scale)
            # turned q and k are rounded to bf16 (2^-8 each): scores move by 2^-7 Z, weights by as much, and
            # their mean by that of V
            got = out[r].double().cpu()
            assert ((got - want).abs() <= V * (2 * 2.0 ** -8 * Z * 1.01 + 2.0 ** -12)).all()
            want_path, answer = O.accept(ps[s], tk[r], tg[r])
            assert path[r].tolist() == want_path + [-1] * (n[s] - len(want_path))
            assert int(counts[s]) == len(want_path) and int(nxt[s]) == answer
            hist[s] = [np.concatenate([h, x[r][want_path]]) for h, x in zip(hist[s], (turned[1], rows[2]))]
            tabs = tab[s].cpu()
            for pool, h in ((kp, hist[s][0]), (vp, hist[s][1])):
                held = O.rows_of(pool.cpu(), tabs, len(h)).transpose(0, 1).numpy()
                # bf16 has 8 bits of a value: a number m 2^e, 1 <= m < 2, lies in steps of 2^(e - 7), so half a step
                # is 2^(e - 8) <= 2^-8 of it; the turn adds 2^-21 of |x_a| + |x_b| (test_gpu_rope.py)
                assert (np.abs(held - h) <= 2.0 ** -8 * np.abs(h) + 2.0 ** -19 * np.abs(h).max()).all()
        assert lens.tolist() == [len(h[0]) for h in hist]
        held = tab.cpu()[torch.arange(M)[None, :] < ((lens.cpu() + B - 1) // B)[:, None]]
        rest = free[: int(nf)].cpu()
        assert sorted(held.tolist() + rest.tolist()) == list(range(NB))


FIRST_CALL = """
import torch
from paged_kv_cache_47_gb300 import binding as b
i32 = dict(dtype=torch.int32, device="cuda")
for dt in (torch.float32, torch.float16, torch.bfloat16):
    q, k = torch.randn(6, 8, 64, device="cuda").to(dt), torch.randn(6, 2, 64, device="cuda").to(dt)
    kp, vp = (torch.randn(8, 2, 16, 64, device="cuda").to(dt) for _ in range(2))
    tab, lens, offs = torch.arange(4, **i32).view(2, 2), torch.tensor([20, 3], **i32), torch.tensor([0, 4, 6], **i32)
    par, tok = torch.tensor([-1, 0, 0, 1, -1, 0], **i32), torch.arange(6, **i32)
    masks, pos = torch.zeros(6, 1, dtype=torch.int64, device="cuda"), torch.zeros(2, 6, **i32)
    path, cnt, nxt, kept = torch.zeros(6, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros(2, **i32)
    free, nf = torch.tensor([7, 6, 5, 4, 0, 0, 0, 0], **i32), torch.tensor([4], **i32)
    slots = torch.arange(16, 22, device="cuda")
    calls = [b.prepared_tree_plan(par, offs, lens, masks, pos),
             b.prepared_rope_axes_append(q, k, k, pos, slots, b.RopeAxesPlan((16, 16)), kp, vp),
             b.prepared_rope_axes(q, k, pos, b.RopeAxesPlan((16, 16))),
             b.prepared_decode_attention_tree(q, kp, vp, tab, lens, offs, masks, 0.1, max_tree=4),
             b.prepared_tree_accept(par, tok, tok + 1, offs, lens, path, cnt, nxt, kept, max_tree=4),
             b.prepared_tree_commit(path, cnt, offs, lens, tab, kp.clone(), vp.clone(), max_tree=4),
             b.prepared_tables_truncate(tab, lens, kept, free, nf, 16, b.alloc_tables_workspace(),
                                        context_lens_out=lens.clone(), num_free_out=nf.clone())]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for call in calls:
            call()
    g.replay()
    torch.cuda.synchronize()
    assert b.get_error() == 0
    a = [t.clone() for t in (masks, pos, path, cnt, nxt, kept, free, calls[3].out)]
    for call in calls:
        call()
    assert all(torch.equal(x, y) for x, y in zip(a, (masks, pos, path, cnt, nxt, kept, free, calls[3].out)))
print("captured")
"""


def test_first_calls_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "captured", r.stderr[-2000:]
