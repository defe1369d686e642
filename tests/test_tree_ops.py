"""CPU checks of the calls that verify drafted tokens and of rotation over several axes: exports, refusals before
anything is enqueued, the plan's numbers, pins of the plain implementations."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from oracle import step_ops as SO
from oracle import tree_ops as O
from paged_kv_cache_47_gb300 import binding as b
from paged_kv_cache_47_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
REF = ctypes.byref
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    build.build()
    return b._ops_lib()


def test_exports_every_declared_symbol(L):
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB], capture_output=True, text=True, check=True).stdout
    exported = set(re.findall(r" T (pkv_\w+)", out))
    for h in ("pkv_tree.h", "pkv_tables.h", "pkv_rope.h"):
        src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h)).read(), flags=re.S)
        names = set(re.findall(r"\b(pkv_[a-z_0-9]+)\s*\(", src))
        assert names and names <= exported, (h, names - exported)


def _desc(nb=8, bs=16, hk=2, d=64, dt=b.PKV_BF16):
    return b.CacheDesc(nb, bs, hk, d, dt)


def _plan(L, S=2, T=8, par=16, offs=16, lens=16, dl=16, masks=16, W=1, pos=16, A=1):
    return L.pkv_tree_plan(S, T, par, offs, lens, dl, masks, W, pos, A, None)


def _accept(L, S=2, T=8, N=4, par=16, tok=16, tgt=16, offs=16, lens=16, path=16, cnt=16, nxt=16, lo=16):
    return L.pkv_tree_accept(S, T, N, par, tok, tgt, offs, lens, path, cnt, nxt, lo, None)


def _commit(L, desc=None, S=2, T=8, N=4, path=16, cnt=16, offs=16, lens=16, tab=16, M=4, kp=16, vp=16):
    return L.pkv_tree_commit(REF(desc or _desc()), S, T, N, path, cnt, offs, lens, tab, M, kp, vp, None)


def _attend(L, desc=None, q=16, T=8, Hq=4, kp=16, vp=16, tab=16, S=2, M=4, lens=16, offs=16, masks=16, W=1, N=4, scale=1.0,
            out=32, odt=2, ws=32, wsb=BIG, ctas=None, lse=None):
    o = b.TreeOptions(ctas or 0, 0, lse)
    return L.pkv_decode_attention_tree(REF(desc or _desc()), q, T, Hq, kp, vp, tab, S, M, lens, offs, masks, W, N, scale,
                                       out, odt, ws, wsb, None, REF(o) if ctas or lse else None)


def _truncate(L, NB=64, B=16, S=2, kept=32, tab=16, M=8, lens=16, lo=16, free=16, nf=16, nfo=16, ws=16):
    return L.pkv_tables_truncate(NB, B, S, kept, tab, M, lens, lo, free, nf, nfo, ws, None)


def test_tree_calls_reject_bad_arguments(L):
    for call in (_plan, _accept, _commit, _attend):
        assert call(L, S=-1) == -1
        assert call(L, T=-1) == -1
        assert call(L, S=0) == 0
        assert call(L, offs=None) == -1
        assert call(L, lens=None) == -1
        assert call(L, offs=18) == -1
        assert call(L, lens=17) == -1
    for call in (_accept, _commit, _attend):
        for n in (0, -3, 257):
            assert call(L, N=n) == -1
    for call in (_plan, _commit, _attend):
        assert call(L, T=0) == 0
    for call in (_commit, _attend):
        for bad, want in ((_desc(d=96), -2), (_desc(bs=12), -2), (_desc(nb=0), -1), (_desc(hk=0), -1), (_desc(dt=3), -2)):
            assert call(L, desc=bad) == want
        assert call(L, M=0) == -1
        assert call(L, M=1 << 28) == -2
        for kw in (dict(tab=None), dict(kp=None), dict(vp=None), dict(tab=6), dict(kp=24), dict(vp=8)):
            assert call(L, **kw) == -1, kw
    for kw in (dict(W=0), dict(W=5), dict(A=0), dict(A=5), dict(par=18), dict(dl=18), dict(masks=12), dict(pos=18)):
        assert _plan(L, **kw) == -1, kw
    for kw in (dict(tok=None), dict(tgt=None), dict(path=None), dict(cnt=None), dict(nxt=None), dict(lo=None), dict(par=18),
               dict(tok=18), dict(path=18), dict(cnt=18), dict(nxt=18), dict(lo=18)):
        assert _accept(L, **kw) == -1, kw
    for kw in (dict(path=None), dict(cnt=None), dict(path=18), dict(cnt=18)):
        assert _commit(L, **kw) == -1, kw
    for kw in (dict(Hq=3), dict(Hq=0), dict(q=None), dict(out=None), dict(q=24), dict(out=18), dict(masks=12), dict(W=0), dict(W=5),
               dict(N=65), dict(scale=math.nan), dict(scale=math.inf), dict(ctas=-1), dict(ctas=4097), dict(lse=18)):
        assert _attend(L, **kw) == -1, kw
    assert _attend(L, odt=3) == -2
    assert _attend(L, Hq=2 * 4097) == -2
    assert _attend(L, desc=_desc(nb=1 << 30), ctas=2) == -2                  # 2^31 (block, head) chunks
    assert _attend(L, ctas=2, ws=None) == -6
    need = L.pkv_decode_tree_workspace_bytes(REF(_desc()), 4, 4, 2)
    assert need > 0 and _attend(L, ctas=2, wsb=need - 1) == -6
    assert _attend(L, ctas=2, ws=8) == -1
    assert L.pkv_decode_tree_workspace_bytes(REF(_desc()), 3, 4, 2) == 0
    assert L.pkv_decode_tree_workspace_bytes(REF(_desc()), 4, 0, 2) == 0
    assert L.pkv_decode_tree_workspace_bytes(REF(_desc()), 4, 4, 4097) == 0


def test_truncate_rejects_bad_arguments(L):
    for kw, want in ((dict(B=12), -2), (dict(NB=0), -1), (dict(S=-1), -1), (dict(M=0), -1), (dict(M=1 << 28), -2),
                     (dict(tab=None), -1), (dict(kept=None), -1), (dict(lens=None), -1), (dict(free=None), -1),
                     (dict(nfo=None), -1), (dict(ws=None), -6), (dict(lens=18), -1), (dict(kept=18), -1),
                     (dict(kept=16), -1)):                                   # kept_lens is also an output
        assert _truncate(L, **kw) == want, kw


def _axes(L, plan=None, dt=b.PKV_BF16, D=64, pos=16, ps=8, T=2, q=16, qs=256, Hq=4, qo=16, qos=256, k=16, ks=128, Hk=2,
          ko=32, kos=128):
    return L.pkv_rope_axes(dt, D, REF(plan or b.RopeAxesPlan((8, 8)).c), pos, ps, T, q, qs, Hq, qo, qos, k, ks, Hk, ko, kos, None)


def _axes_append(L, plan=None, desc=None, pos=16, ps=8, slots=16, T=2, q=16, qs=256, Hq=4, qo=16, qos=256, k=16, ks=128,
                 v=16, vs=128, kp=16, vp=16):
    return L.pkv_rope_axes_append(REF(desc or _desc()), REF(plan or b.RopeAxesPlan((8, 8)).c), pos, ps, slots, T, q, qs, Hq,
                                  qo, qos, k, ks, v, vs, kp, vp, None)


def test_rope_axes_rejects_bad_arguments(L):
    bad_axis = b.RopeAxesPlan((8, 8)).c
    bad_axis.axis[3] = 2
    for call in (_axes, _axes_append):
        assert call(L, plan=b._RopeAxesPlan()) == -1
        assert call(L, plan=bad_axis) == -1
        assert call(L, plan=b.RopeAxesPlan((40, 24)).c) == -1                # wider than the head
        for kw in (dict(pos=None), dict(pos=18), dict(ps=-1), dict(T=-1), dict(q=None), dict(q=24), dict(qs=252), dict(qs=264)):
            assert call(L, **kw) == -1, kw
        assert call(L, T=0) == 0
        assert call(L, T=1 << 30) == -2
    assert L.pkv_rope_axes(2, 64, None, 16, 8, 2, 16, 256, 4, 16, 256, 16, 128, 2, 32, 128, None) == -1
    assert _axes_append(L, slots=None) == -1 and _axes_append(L, kp=8) == -1 and _axes_append(L, vs=64) == -1
    for kw in (dict(sections=(0, 8)), dict(sections=(60, 5)), dict(sections=(8, -8, 8)), dict(sections=(8,), base=1.0),
               dict(sections=(1, 8), frequencies="own", scaling="base", factor=2.0)):
        with pytest.raises(b.PkvError):
            b.RopeAxesPlan(**kw)
    with pytest.raises(ValueError, match="axes"):
        b.RopeAxesPlan((2,) * 5)
    d = b.RopeAxesDesc()
    p = b._RopeAxesPlan()
    d.rope = b.RopeDesc(32, 0, 0, 0, 1e4, 1, 0, 0, 0, 0, 0)
    d.num_axes, d.sections[0] = 1, 15
    assert L.pkv_rope_axes_plan_init(REF(d), REF(p)) == -1                   # 15 pairs of 16
    d.sections[0], d.order = 16, 2
    assert L.pkv_rope_axes_plan_init(REF(d), REF(p)) == -1
    d.order, d.frequencies = 0, -1
    assert L.pkv_rope_axes_plan_init(REF(d), REF(p)) == -1
    d.frequencies = 0
    assert L.pkv_rope_axes_plan_init(REF(d), REF(p)) == 0
    assert L.pkv_rope_axes_plan_init(None, REF(p)) == -1 and L.pkv_rope_axes_plan_init(REF(d), None) == -1


@pytest.mark.parametrize("kw", [
    dict(sections=(16, 24, 24)), dict(sections=(24, 20, 20), order="cycled"), dict(sections=(1, 2, 3, 4), order="cycled"),
    dict(sections=(8, 12, 12), frequencies="own"), dict(sections=(9, 3), order="cycled", frequencies="own", base=5e5),
    dict(sections=(6, 10), frequencies="own", scaling="yarn", factor=16.0, original_len=4096)])
def test_rope_axes_plan_numbers(L, kw):
    args = dict(kw)
    axis, w, amp = SO.axes_frequencies(args.pop("sections"), args.pop("order", "sections"), args.pop("frequencies", "shared"),
                                       args.pop("base", 10000.0), **args)
    p = b.RopeAxesPlan(**kw).c
    assert list(p.axis[: len(axis)]) == axis.tolist() and p.num_axes == len(kw["sections"])
    assert p.plan.rotary_dim == 2 * len(w) and p.plan.amplitude == np.float32(amp)
    for i, f in enumerate(w):
        turns = f / (2 * math.pi)
        d = abs(p.plan.turns[i] / 2.0 ** 64 - turns % 1.0)
        assert min(d, 1 - d) <= 16 * 2.0 ** -53 * turns + 2.0 ** -62


def test_axes_oracle_pins():
    axis, w, _ = SO.axes_frequencies((3, 1, 2), "cycled", "shared", 10000.0)
    assert axis.tolist() == [0, 1, 2, 0, 2, 0]
    assert SO.axes_frequencies((3, 1, 2), "sections", "own", 10000.0)[0].tolist() == [0, 0, 0, 1, 2, 2]
    assert np.allclose(SO.axes_frequencies((3, 1, 2), "sections", "own", 10000.0)[1],
                       [1, 1e4 ** (-1 / 3), 1e4 ** (-2 / 3), 1, 1, 1e-2])
    assert np.allclose(w, 1e4 ** (-np.arange(6) / 6))


def test_tree_oracle_pins():
    p = [-1, 0, 0, 1, 3]
    a = O.ancestors(p)
    assert a.astype(int).tolist() == [[1, 0, 0, 0, 0], [1, 1, 0, 0, 0], [1, 0, 1, 0, 0], [1, 1, 0, 1, 0], [1, 1, 0, 1, 1]]
    assert O.words(a, 1)[:, 0].tolist() == [1, 3, 5, 11, 27]
    assert O.words(np.ones((1, 65), bool), 2).tolist() == [[-1, 1]]
    # 0 answers 7: token 1 holds; 1 answers 9: token 3 does not; token 2 holds too, but is as deep and later
    assert O.accept(p, [5, 7, 7, 8, 9], [7, 9, 1, 9, 2]) == ([0, 1], 9)
    assert O.accept(p, [5, 7, 7, 9, 9], [7, 9, 1, 9, 2]) == ([0, 1, 3, 4], 2)
    assert O.accept([], [], []) == ([], -1)
    q = torch.zeros(1, 2, 64)
    k, v = torch.zeros(1, 3, 64).double(), torch.arange(3.0).double()[None, :, None].expand(1, 3, 64)
    out, lse, Z, V = O.attend(q, k, v, torch.tensor([[True, False, True]]), 1.0)
    assert (out == 1).all() and (lse == 1).all() and Z == 0 and V == 2


def test_binding_refuses_what_is_not_on_the_gpu_or_does_not_fit():
    i32 = dict(dtype=torch.int32)
    lens, offs, par = torch.zeros(2, **i32), torch.zeros(3, **i32), torch.zeros(5, **i32)
    masks, pos = torch.zeros(5, 1, dtype=torch.int64), torch.zeros(5, **i32)
    with pytest.raises(ValueError, match="GPU"):
        b.tree_plan(par, offs, lens, masks, pos)
    with pytest.raises(ValueError, match="neither"):
        b.tree_plan(par, offs, lens)
    with pytest.raises(ValueError, match="masks"):
        b.tree_plan(par, offs, lens, torch.zeros(5, 5, dtype=torch.int64))
    with pytest.raises(ValueError, match="token_offsets"):
        b.tree_plan(par, offs[:2], lens, masks)
    with pytest.raises(ValueError, match="GPU"):
        b.tree_accept(par, par, par, offs, lens, max_tree=4)
    with pytest.raises(ValueError, match="counts"):
        b.tree_commit(par, par, offs, lens, torch.zeros(2, 3, **i32), torch.zeros(2, 1, 16, 64), torch.zeros(2, 1, 16, 64), 4)
    with pytest.raises(ValueError, match="positions"):
        b.rope_axes(torch.zeros(5, 2, 64), torch.zeros(5, 1, 64), torch.zeros(3, 5, **i32), b.RopeAxesPlan((8, 8)))
    with pytest.raises(ValueError, match="contiguous"):
        b.rope_axes(torch.zeros(5, 2, 64), torch.zeros(5, 1, 64), torch.zeros(5, 2, **i32).t(), b.RopeAxesPlan((8, 8)))
