"""CPU checks of the step operators (device tables, rotary positions, the 4-bit cache, block
selection): exports, refusals before anything is enqueued, the rotary plan's numbers, the 4-bit
decode's split, and pins of the plain implementations the GPU tests compare with."""
import ctypes
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from oracle import step_ops as O
from paged_kv_cache_47_gb300 import binding as b
from paged_kv_cache_47_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
REF = ctypes.byref
BIG = 1 << 30


@pytest.fixture(scope="module")
def L():
    build.build()
    return b._ops_lib()


def test_exports_every_declared_symbol(L):
    out = subprocess.run(["nm", "-D", "--defined-only", build.LIB], capture_output=True, text=True,
                         check=True).stdout
    exported = set(re.findall(r" T (pkv_\w+)", out))
    for h in ("pkv_tables.h", "pkv_rope.h", "pkv_q4.h", "pkv_sparse.h"):
        src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", h)).read(), flags=re.S)
        names = set(re.findall(r"\b(pkv_[a-z_0-9]+)\s*\(", src))
        assert names and names <= exported, (h, names - exported)


# ----------------------------------------------------------------------------- refusals
def _append(L, NB=64, B=16, S=2, add=16, tab=16, M=8, lens=16, lens_out=16, free=16, nf=16, nfo=16,
            slots=16, pos=16, T=8, offs=16, ws=16):
    return L.pkv_tables_append(NB, B, S, add, tab, M, lens, lens_out, free, nf, nfo, slots, pos, T, offs,
                               ws, None)


def _release(L, NB=64, B=16, S=2, rel=16, tab=16, M=8, lens=16, lens_out=16, free=16, nf=16, nfo=16, ws=16):
    return L.pkv_tables_release(NB, B, S, rel, tab, M, lens, lens_out, free, nf, nfo, ws, None)


def test_tables_reject_bad_arguments(L):
    for call in (_append, _release):
        assert call(L, B=12) == -2
        assert call(L, NB=0) == -1
        assert call(L, S=-1) == -1
        assert call(L, M=0) == -1
        assert call(L, M=1 << 28) == -2            # a row of 2^32 tokens
        assert call(L, tab=None) == -1
        assert call(L, lens=None) == -1
        assert call(L, free=None) == -1
        assert call(L, nfo=None) == -1
        assert call(L, ws=None) == -6
        assert call(L, lens=18) == -1              # misaligned
    assert _append(L, T=-1) == -1
    assert _append(L, slots=None) == -1
    assert _append(L, slots=20) == -1
    assert _append(L, offs=None) == -1
    assert _release(L, rel=None) == -1


def _desc(nb=8, bs=16, hk=2, d=64, dt=b.PKV_BF16):
    return b.CacheDesc(nb, bs, hk, d, dt)


def _plan(rd=64, **kw):
    return b.RopePlan(rd, **kw).c


def _rope(L, dt=b.PKV_BF16, D=64, plan=None, pos=16, T=2, q=16, qs=256, Hq=4, qo=16, qos=256, k=16, ks=128,
          Hk=2, ko=32, kos=128):
    return L.pkv_rope(dt, D, REF(plan or _plan()), pos, T, q, qs, Hq, qo, qos, k, ks, Hk, ko, kos, None)


def _rope_append(L, desc=None, plan=None, pos=16, slots=16, T=2, q=16, qs=256, Hq=4, qo=16, qos=256, k=16,
                 ks=128, v=16, vs=128, kp=16, vp=16):
    return L.pkv_rope_append(REF(desc or _desc()), REF(plan or _plan()), pos, slots, T, q, qs, Hq, qo, qos, k,
                             ks, v, vs, kp, vp, None)


def test_rope_rejects_bad_arguments(L):
    assert _rope(L, dt=3) == -2
    assert _rope(L, D=96) == -2
    assert _rope(L, plan=_plan(128)) == -1                 # wider than the head
    assert _rope(L, plan=b._RopePlan()) == -1              # not a plan
    assert _rope(L, T=-1) == -1
    assert _rope(L, T=1 << 30) == -2
    assert _rope(L, T=0) == 0
    assert _rope(L, Hq=0, Hk=0, q=None, k=None) == 0
    assert _rope(L, pos=None) == -1
    assert _rope(L, q=None) == -1
    assert _rope(L, q=24) == -1                            # misaligned
    assert _rope(L, qs=252) == -1                          # stride below the heads
    assert _rope(L, qs=260) == -1                          # stride not of 16 bytes
    assert _rope(L, qs=264) == -1                          # in place with two strides
    assert _rope_append(L, desc=_desc(d=96)) == -2
    assert _rope_append(L, T=0) == 0
    assert _rope_append(L, slots=None) == -1
    assert _rope_append(L, slots=20) == -1
    assert _rope_append(L, kp=None) == -1
    assert _rope_append(L, vp=8) == -1
    assert _rope_append(L, vs=64) == -1
    assert _rope_append(L, qos=264) == -1
    for kw in (dict(rotary_dim=3), dict(rotary_dim=130), dict(rotary_dim=0), dict(base=1.0), dict(base=math.inf),
               dict(scaling="linear", factor=0.0), dict(scaling="bands", factor=2.0),
               dict(scaling="bands", factor=2.0, original_len=8, low_freq_factor=4.0),
               dict(scaling="yarn", factor=2.0, original_len=8, beta_fast=0.5),
               dict(scaling="base", factor=2.0, rotary_dim=2), dict(scaling="base", factor=1e-9, base=2.0)):
        with pytest.raises(b.PkvError):
            b.RopePlan(**{"rotary_dim": 64, **kw})


def _q4desc(nb=8, bs=16, hk=2, d=128, act=b.PKV_BF16):
    return b.Q4CacheDesc(nb, bs, hk, d, act)


def _pools(kc=16, vc=16, kp=16, vp=16):
    return b.Q4Pools(kc, vc, kp, vp)


def _q4decode(L, desc=None, pools=None, S=1, Hq=4, q=16, bt=16, M=4, lens=16, scale=1.0, out=16, odt=2, ws=16,
              wsb=BIG, opts=None):
    return L.pkv_decode_attention_q4(REF(desc or _q4desc()), q, S, Hq, REF(pools or _pools()), bt, M, lens, scale,
                                     out, odt, ws, wsb, None, REF(opts) if opts is not None else None)


def test_q4_rejects_bad_arguments(L):
    for bad, want in ((_q4desc(act=b.PKV_F32), -2), (_q4desc(d=96), -2), (_q4desc(bs=12), -2), (_q4desc(nb=0), -1),
                      (_q4desc(hk=0), -1)):
        assert _q4decode(L, bad) == want
        assert L.pkv_append_q4(REF(bad), 16, 16, 16, 1, REF(_pools()), None) == want
        assert L.pkv_gather_q4(REF(bad), REF(_pools()), 16, 1, 16, 16, 2, None) == want
    assert _q4decode(L, Hq=3) == -1
    assert _q4decode(L, S=-1) == -1
    assert _q4decode(L, S=0) == 0
    assert _q4decode(L, odt=3) == -2
    assert _q4decode(L, M=0) == -1
    assert _q4decode(L, scale=math.nan) == -1
    assert _q4decode(L, q=None) == -1
    assert _q4decode(L, q=24) == -1
    assert _q4decode(L, out=18) == -1
    assert _q4decode(L, M=1 << 28) == -2
    for p in (_pools(kc=None), _pools(vp=8)):
        assert _q4decode(L, pools=p) == -1
    o = b.DecodeOptions()
    o.num_ctas = 2
    assert _q4decode(L, opts=o, ws=None) == -6
    assert _q4decode(L, opts=o, wsb=4096 * 4 + 2 * 2 * 2 * 129 * 4 - 1) == -6
    assert _q4decode(L, opts=o, ws=8) == -1
    for field, value, want in (("consumer", 1, -2), ("consumer", 3, -1), ("num_ctas", -1, -1), ("num_ctas", 4097, -1),
                               ("pending_tail", -1, -1), ("pending_tail", 1, -1)):
        o = b.DecodeOptions()
        setattr(o, field, value)
        assert _q4decode(L, opts=o) == want, field
    d = _q4desc()
    assert L.pkv_append_q4(REF(d), 16, 16, 16, -1, REF(_pools()), None) == -1
    assert L.pkv_append_q4(REF(d), 16, 16, 16, 0, REF(_pools()), None) == 0
    assert L.pkv_append_q4(REF(d), 16, None, 16, 1, REF(_pools()), None) == -1
    assert L.pkv_append_q4(REF(d), 16, 24, 16, 1, REF(_pools()), None) == -1
    assert L.pkv_gather_q4(REF(d), REF(_pools()), 16, 1, 16, 16, 4, None) == -2
    assert L.pkv_gather_q4(REF(d), REF(_pools()), 12, 1, 16, 16, 2, None) == -1
    p = torch.tensor([[0, 8]], dtype=torch.int64)
    assert L.pkv_block_copy_q4(REF(d), p.data_ptr(), 1, REF(_pools()), None) == -1
    assert L.pkv_block_copy_q4(REF(d), p.data_ptr(), -1, REF(_pools()), None) == -1
    assert L.pkv_block_copy_q4(REF(d), p.data_ptr(), 0, REF(_pools()), None) == 0


def test_q4_workspace_formula(L):
    # 4096 arrival counters, then C CTAs x 2 pieces x heads x (D outputs + 1 denominator)
    assert L.pkv_decode_q4_workspace_bytes(REF(_q4desc(hk=8)), 32, 10) == 4096 * 4 + 10 * 2 * 4 * 129 * 4
    assert L.pkv_decode_q4_workspace_bytes(REF(_q4desc(hk=1, d=64)), 12, 3) == 4096 * 4 + 3 * 2 * 8 * 65 * 4
    # more than 4 heads at head size 128: and 16 warps' pieces a CTA
    assert L.pkv_decode_q4_workspace_bytes(REF(_q4desc(hk=1)), 8, 3) == 4096 * 4 + 3 * 8 * (2 * 129 + 16 * 128) * 4
    assert L.pkv_decode_q4_workspace_bytes(REF(_q4desc()), 3, 10) == 0
    assert L.pkv_decode_q4_workspace_bytes(REF(_q4desc()), 4, 4097) == 0


def _select(L, desc=None, sel=(1, 0, 1), q=16, S=1, Hq=4, means=16, bt=16, M=4, lens=16, st=16, sl=16, ws=16,
            wsb=BIG):
    return L.pkv_select_blocks(REF(desc or _desc()), q, S, Hq, means, bt, M, lens,
                               REF(b.SparseSelect(*sel)) if sel else None, st, sl, ws, wsb, None)


def _sparse(L, desc=None, sel=(1, 0, 1), q=16, S=1, Hq=4, kp=16, vp=16, means=16, bt=16, M=4, lens=16, scale=1.0,
            st=16, sl=16, out=16, odt=2, ws=16, wsb=BIG):
    return L.pkv_decode_attention_sparse(REF(desc or _desc()), q, S, Hq, kp, vp, means, bt, M, lens, scale,
                                         REF(b.SparseSelect(*sel)) if sel else None, st, sl, out, odt, ws, wsb,
                                         None)


def test_sparse_rejects_bad_arguments(L):
    assert L.pkv_block_means(REF(_desc(bs=12)), 16, 1, 16, 16, None) == -2
    assert L.pkv_block_means(REF(_desc()), 16, -1, 16, 16, None) == -1
    assert L.pkv_block_means(REF(_desc()), 16, 0, 16, 16, None) == 0
    assert L.pkv_block_means(REF(_desc()), None, 1, 16, 16, None) == -1
    assert L.pkv_block_means(REF(_desc()), 16, 1, 16, 24, None) == -1
    assert _select(L, sel=None) == -1
    for sel in ((-1, 0, 1), (1, -1, 1), (1, 0, 0)):
        assert _select(L, sel=sel) == -1
    assert _select(L, sel=(1 << 30, 0, 1)) == -2
    assert _select(L, wsb=15) == -6                # 1 x 2 x 4 scores
    assert _select(L, ws=None) == -6
    assert _select(L, ws=8) == -1
    assert _select(L, S=0) == 0
    assert _sparse(L, S=0) == 0
    assert _sparse(L, odt=3) == -2
    assert _sparse(L, scale=math.inf) == -1
    assert _sparse(L, kp=None) == -1
    assert _sparse(L, vp=8) == -1
    for call in (_select, _sparse):
        assert call(L, desc=_desc(d=96)) == -2
        assert call(L, Hq=3) == -1
        assert call(L, S=-1) == -1
        assert call(L, M=0) == -1
        assert call(L, desc=_desc(nb=1 << 30)) == -2      # 2^31 (block, head) chunks
    assert L.pkv_select_workspace_bytes(REF(_desc()), 3, 5) == 3 * 2 * 8 * 4
    assert L.pkv_select_workspace_bytes(REF(_desc()), -1, 5) == 0


def test_binding_refuses_what_is_not_on_the_gpu_or_not_contiguous():
    i32 = dict(dtype=torch.int32)
    tab, lens, one = torch.zeros(2, 4, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    ws = torch.zeros(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        b.tables_release(tab, lens, torch.zeros(2, dtype=torch.bool), torch.zeros(8, **i32), one, 16, ws)
    with pytest.raises(ValueError, match="contiguous"):
        b.tables_release(tab.t().contiguous().t(), lens, torch.zeros(2, dtype=torch.bool), torch.zeros(8, **i32),
                         one, 16, ws)
    q, pool = torch.zeros(3, 4, 64), torch.zeros(2, 2, 16, 64)
    pos, slots = torch.zeros(3, **i32), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="GPU"):
        b.rope_append(q, q[:, :2], q[:, 2:], pos, slots, b.RopePlan(64), pool, pool)
    with pytest.raises(ValueError, match="contiguous"):
        b.rope(q.transpose(1, 2).contiguous().transpose(1, 2), q, pos, b.RopePlan(64))
    with pytest.raises(ValueError, match="k_params"):
        b.Q4Cache(*[torch.zeros(2, 2, 16, 64, dtype=torch.uint8)] * 2, *[torch.zeros(2, 2, 16, 4).half()] * 2,
                  torch.float16)
    c = b.Q4Cache.empty(2, 2, 16, 128, torch.float16, device="cpu")
    with pytest.raises(ValueError, match="GPU"):
        b.append_q4(torch.zeros(1, 2, 128).half(), torch.zeros(1, 2, 128).half(), slots[:1], c)


# --------------------------------------------------------------------------------- plan
@pytest.mark.parametrize("kw", [
    dict(rotary_dim=128), dict(rotary_dim=20, base=500000.0),
    dict(rotary_dim=64, scaling="linear", factor=4.0), dict(rotary_dim=64, scaling="linear", factor=0.01),
    dict(rotary_dim=96, scaling="base", factor=8.0),
    dict(rotary_dim=128, base=500000.0, scaling="bands", factor=8.0, original_len=8192),
    dict(rotary_dim=128, scaling="yarn", factor=16.0, original_len=4096),
    dict(rotary_dim=128, scaling="yarn", factor=16.0, original_len=4096, attention_factor=0.7)])
def test_rope_plan_numbers(L, kw):
    w, amp = O.rope_frequencies(**{"base": 10000.0, **kw})
    p = b.RopePlan(**kw).c
    assert p.rotary_dim == kw["rotary_dim"] and p.amplitude == np.float32(amp)
    for i, f in enumerate(w):
        turns = f / (2 * math.pi)
        got = p.turns[i] / 2.0 ** 64
        d = abs(got - turns % 1.0)
        # a few roundings of 2^-53 each in pow, the scaling and the division
        assert min(d, 1 - d) <= 16 * 2.0 ** -53 * turns + 2.0 ** -62
    assert not any(p.turns[i] for i in range(len(w), 64))


# ------------------------------------------------------------------------------- oracle
def test_q4_oracle_pins():
    # -1, 0, 14: minimum -1, scale 1, codes 0, 1, 15
    x = np.zeros((1, 64), np.float32)
    x[0, :3] = -1, 0, 14
    c, s, m = O.q4_quantize(x)
    assert s[0, 0] == 1 and m[0, 0] == -1 and list(c[0, :4]) == [0, 1, 15, 1]
    assert s[0, 1] == 0 and m[0, 1] == 0 and not c[0, 32:].any()
    assert (O.q4_values(c, s, m)[0] == x[0]).all()
    # a half step goes to the even code: 0.5 -> 0, 1.5 -> 2
    x[0, 3:5] = -0.5, 0.5
    assert list(O.q4_quantize(x)[0][0, 3:5]) == [0, 2]
    x[0, 5] = np.inf
    c, s, m = O.q4_quantize(x)
    assert np.isnan(s[0, 0]) and np.isnan(m[0, 0]) and not c[0, :32].any() and m[0, 1] == 0
    rng = np.random.default_rng(0)
    for D in (64, 128):
        c = rng.integers(0, 16, (3, D)).astype(np.uint8)
        for rows in (True, False):
            assert (O.q4_unpack(O.q4_pack(c, rows), rows) == c).all()
    # K: element 33 of 128 (group 1, place 1) is nibble 1 of word 1; V: nibble 1 of half-word 1
    one = np.zeros((1, 128), np.uint8)
    one[0, 33] = 5
    assert O.q4_pack(one, True).view(np.uint32)[0, 1] == 0x50
    assert O.q4_pack(one, False).view(np.uint16)[0, 1] == 0x50


def test_tables_oracle_agrees_with_the_block_manager():
    rng = np.random.default_rng(3)
    NB, B, S, M = 40, 8, 5, 9
    bm = b.BlockManager(NB, B)
    tab, lens = np.full((S, M), -1, np.int32), np.zeros(S, np.int32)
    free, nf = np.arange(NB, dtype=np.int32)[::-1].copy(), NB
    for s in range(S):
        bm.add_sequence(s)
    for step in range(30):
        rel = rng.random(S) < 0.15
        for s in np.flatnonzero(rel):
            bm.free_sequence(int(s))
            bm.add_sequence(int(s))
        lens, free, nf = O.tables_release(tab, lens, rel, free, nf, B)
        add = rng.integers(0, 9, S).astype(np.int32)
        add = np.minimum(add, M * B - lens)
        got = O.tables_append(tab, lens, add, free, nf, B, 64)
        if got is None:
            break
        tab, lens, nf, slots, pos, offs = got
        want, _ = bm.append_batch(range(S), add.tolist())
        assert slots[: add.sum()].tolist() == want.tolist()
        wt, wl = bm.block_tables(range(S), M)
        assert wl.tolist() == lens.tolist()
        for s in range(S):
            n = -(-int(lens[s]) // B)
            assert tab[s, :n].tolist() == wt[s, :n].tolist()
        assert nf == bm.num_free()
    assert step > 3


def test_select_oracle_pins():
    score = np.array([9, 1, 5, 5, 5, 0, 9], np.float32)
    assert O.select(score, 7, 2, 1, 1) == [0, 2, 3, 6]       # ties go to the lower block
    assert O.select(score, 7, 0, 1, 2) == [0, 5, 6]
    assert O.select(score, 7, 9, 0, 1) == list(range(7))
    assert O.select(score, 2, 1, 3, 4) == [0, 1]
    q = np.ones((2, 64), np.float32)
    q[1] = -1
    m = np.stack([np.full(64, 0.5), np.full(64, -2.0)]).astype(np.float32)
    assert O.block_scores(q, m).tolist() == [32.0, 128.0]


def test_warp_split_replay(tmp_path):
    exe = tmp_path / "warp_split_check"
    subprocess.run(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "paged_kv_cache_47_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "warp_split_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "OK", r.stdout
