"""The step operators together, as a serving loop calls them: device tables, rotary append, then
decode over the 16-bit cache, over the selected blocks of it, and over a 4-bit cache; captured into
one CUDA graph and replayed step after step with no host decision in between."""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import step_ops as O
from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu


def test_graph_of_a_whole_serving_step():
    S, Hq, Hk, D, B, M, NB, T = 5, 8, 2, 64, 8, 12, 64, 360
    bf, i32 = torch.bfloat16, dict(dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(0)
    scale = 1 / math.sqrt(D)
    kw = dict(rotary_dim=D, base=10000.0)
    plan = b.RopePlan(**kw)
    tab, lens = torch.full((S, M), -1, **i32), torch.zeros(S, **i32)
    free, nf = torch.arange(NB - 1, -1, -1, **i32), torch.tensor([NB], **i32)
    done, add = torch.zeros(S, dtype=torch.bool, device="cuda"), torch.zeros(S, **i32)
    slots, pos, offs = torch.empty(T, dtype=torch.int64, device="cuda"), torch.empty(T, **i32), torch.empty(S + 1, **i32)
    qkv = torch.zeros(T, (Hq + 2 * Hk) * D, dtype=bf, device="cuda")
    q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
    kp, vp = (torch.zeros(NB, Hk, B, D, dtype=bf, device="cuda") for _ in range(2))
    km = torch.zeros(NB, Hk, D, dtype=bf, device="cuda")
    cache = b.Q4Cache.empty(NB, Hk, B, D, bf)
    qo, k4, v4 = (torch.empty(T, h, D, dtype=bf, device="cuda") for h in (Hq, Hk, Hk))
    q4o = torch.empty_like(qo)
    last, ql = torch.empty(S, dtype=torch.int64, device="cuda"), torch.empty(S, Hq, D, dtype=bf, device="cuda")
    out, out_s, out_4 = (torch.empty(S, Hq, D, dtype=torch.float32, device="cuda") for _ in range(3))
    tws = b.alloc_tables_workspace()
    ws, ws_s, ws_4 = (b.alloc_workspace(kp, Hq), b.alloc_sparse_workspace(kp, S, Hq, M), b.alloc_q4_workspace(cache, Hq))
    sel = torch.empty(S, Hk, 6, **i32), torch.empty(S, Hk, **i32)

    def step():
        b.tables_release(tab, lens, done, free, nf, B, tws)
        b.tables_append(tab, lens, add, free, nf, B, slots, pos, offs, tws)
        b.rope_append(q, k, v, pos, slots, plan, kp, vp, q_out=qo)
        b.block_means(slots, kp, km)
        b.rope(q, k, pos, plan, q_out=q4o, k_out=k4)
        v4.copy_(v)
        b.append_q4(k4, v4, slots, cache)
        # each request's newest token asks (requests without new tokens ask with another's: not looked at)
        torch.sub(offs[1:], 1, out=last).clamp_(min=0)
        torch.index_select(qo, 0, last, out=ql)
        b.decode_attention(ql, kp, vp, tab, lens, scale, out=out, workspace=ws)
        b.decode_attention_sparse(ql, kp, vp, km, tab, lens, scale, 3, 1, 2, out=out_s, sel_tables=sel[0],
                                  sel_lens=sel[1], workspace=ws_s)
        b.decode_attention_q4(ql, cache, tab, lens, scale, out=out_4, workspace=ws_4)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert b.get_error() == 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()

    w, amp = O.rope_frequencies(**kw)
    hist = [[np.zeros((0, Hk, D))] * 2 for _ in range(S)]            # turned keys and values, 64 bits
    for it in range(12):
        fin = np.array([it % 5 == 4 and s == it % 3 for s in range(S)])
        for s in np.flatnonzero(fin):
            hist[s] = [np.zeros((0, Hk, D))] * 2
        grow = np.array([rng.integers(20, 71) if not len(hist[s][0]) else rng.integers(0, 3) for s in range(S)])
        grow = np.minimum(grow, M * B - np.array([len(h[0]) for h in hist]))
        grow[fin] = 0
        done.copy_(torch.from_numpy(fin))
        add.copy_(torch.from_numpy(grow.astype(np.int32)))
        qkv.copy_(torch.randn(T, qkv.shape[1], generator=torch.Generator().manual_seed(it)).to(bf))
        graph.replay()
        assert b.get_error() == 0
        n = int(grow.sum())
        rows = [x.double().cpu().numpy() for x in (q, k, v)]
        p = pos.cpu().numpy()
        assert (slots[n:] == -1).all()
        tk = O.rope(rows[1][:n], p[:n], w, amp, "half")[0]
        at = 0
        for s in range(S):
            m = int(grow[s])
            assert p[at: at + m].tolist() == list(range(len(hist[s][0]), len(hist[s][0]) + m))
            hist[s] = [np.concatenate([h, x[at: at + m]]) for h, x in zip(hist[s], (tk, rows[2]))]
            at += m
        assert lens.tolist() == [len(h[0]) for h in hist]
        held = tab.cpu()[torch.arange(M)[None, :] < ((lens.cpu() + B - 1) // B)[:, None]]
        assert len(set(held.tolist())) == len(held) == NB - int(nf)
        at = 0
        for s in range(S):
            m = int(grow[s])
            at += m
            if m == 0:
                continue
            qs = ql[s].double().cpu().numpy()
            kk, vv = (h.transpose(1, 0, 2) for h in hist[s])
            want = O.attend(qs, kk, vv, scale)[0]
            # turned keys are rounded to bf16 (2^-8): scores move by 2^-8 scale sum |q k| at most,
            # and weights by as much, twice (numerator and denominator), of |v - o|
            z = scale * np.einsum("hd,hld->hl", np.abs(qs), np.abs(np.repeat(kk, Hq // Hk, 0))).max()
            spread = 2 * np.abs(vv).max()
            tol = 2 * 2.0 ** -8 * z * spread + 2e-3
            assert np.abs(out[s].cpu().numpy() - want).max() <= tol
            L = len(hist[s][0])
            if -(-L // B) <= 6:                       # all blocks selected: the same attention
                assert np.abs(out_s[s].cpu().numpy() - out[s].cpu().numpy()).max() <= 4e-3
            # the 4-bit cache against the attention over its own values
            arrays = [t.cpu().numpy() for t in (cache.k_codes, cache.v_codes, cache.k_params, cache.v_params)]
            k8, v8 = O.q4_rows(tab[s].cpu().numpy(), L, *arrays)
            want4 = O.attend(qs, k8, v8, scale)[0]
            assert np.abs(out_4[s].cpu().numpy() - want4).max() <= 2.0 ** -9 * 2 * np.abs(v8).max()
            # and each cached element is within a step of the rounded row (scale / 2, parameters to 2^-11)
            got = np.abs(k8 - kk)
            step_k = (kk.max(-1) - kk.min(-1)).max() / 15
            assert got.max() <= 0.5 * step_k + 2.0 ** -8 * np.abs(kk).max() + 16 * 2.0 ** -11 * np.abs(kk).max()
    assert max(len(h[0]) for h in hist) > 6 * B      # selections left blocks out


FIRST_CALL = """
import torch
from paged_kv_cache_47_gb300 import binding as b
i32 = dict(dtype=torch.int32, device="cuda")
q, k = torch.randn(4, 8, 64, device="cuda").half(), torch.randn(4, 2, 64, device="cuda").half()
pos, slots = torch.arange(4, **i32), torch.arange(4, device="cuda")
kp, vp = (torch.zeros(8, 2, 16, 64, device="cuda").half() for _ in range(2))
km = torch.zeros(8, 2, 64, device="cuda").half()
tab, lens = torch.arange(4, **i32).view(4, 1), torch.full((4,), 1, **i32)
free, nf, one = torch.arange(8, **i32), torch.tensor([4], **i32), torch.ones(4, **i32)
sl, ps, of = torch.zeros(8, dtype=torch.int64, device="cuda"), torch.zeros(8, **i32), torch.zeros(5, **i32)
c = b.Q4Cache.empty(8, 2, 16, 64, torch.float16)
calls = [b.prepared_tables_release(tab, lens, torch.zeros(4, dtype=torch.bool, device="cuda"), free, nf, 16,
                                   b.alloc_tables_workspace(), context_lens_out=one.clone(), num_free_out=nf.clone()),
         b.prepared_tables_append(tab, lens, one, free, nf, 16, sl, ps, of, b.alloc_tables_workspace(),
                                  context_lens_out=one.clone(), num_free_out=nf.clone()),
         b.prepared_rope_append(q, k, k, pos, slots, b.RopePlan(64), kp, vp),
         b.prepared_append_q4(k, k, slots, c), b.prepared_gather_q4(slots, c), b.prepared_block_means(slots, kp, km),
         b.prepared_decode_attention_q4(q, c, tab, lens, 0.1),
         b.prepared_decode_attention_sparse(q, kp, vp, km, tab, lens, 0.1, 1, 0, 1)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for call in calls:
        call()
g.replay()
torch.cuda.synchronize()
assert b.get_error() == 0
a = [x.out.clone() for x in calls[6:]] + list(t.clone() for t in calls[4].out) + [sl.clone()]
for call in calls:
    call()
assert all(torch.equal(x, y) for x, y in zip(a, [x.out for x in calls[6:]] + list(calls[4].out) + [sl]))
print("captured")
"""


def test_first_calls_of_a_process_can_be_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "captured", r.stderr[-2000:]
