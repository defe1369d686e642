"""Rotary positions of several axes on the GPU against the formula in 64 bits; tolerances as for one axis
(test_gpu_rope.py): 2^-21 of |x_a| + |x_b|, then half a step of the output's type."""
import numpy as np
import pytest
import torch

from oracle import step_ops as O
from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def randn(shape, dt, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DT[dt])


def close(got, x, pos, kw):
    """got against x turned; CPU tensors [T][H][D], positions [axes][T]."""
    args = {k: v for k, v in kw.items() if k not in ("layout", "sections", "order", "frequencies")}
    axis, w, amp = O.axes_frequencies(kw["sections"], kw.get("order", "sections"), kw.get("frequencies", "shared"),
                                      args.pop("base", 10000.0), **args)
    want, size = O.rope(x.double().numpy(), pos.numpy().T[:, axis], w, amp, kw.get("layout", "half"))
    rd = 2 * len(w)
    tol = size * amp * 2.0 ** -21 + np.abs(want) * torch.finfo(x.dtype).eps / 2
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    bad = np.abs(got.double().numpy() - want)[..., :rd] > tol[..., :rd]
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3])
    assert torch.equal(got[..., rd:], x[..., rd:])


PLANS = [
    dict(sections=(16, 8, 8)), dict(sections=(8, 12, 12), order="cycled"), dict(sections=(1, 30, 1), order="cycled"),
    dict(sections=(8, 12, 12), frequencies="own", layout="interleaved"), dict(sections=(5, 5), layout="interleaved"),
    dict(sections=(10,)), dict(sections=(4, 4, 4, 4), order="cycled", frequencies="own", base=500000.0),
    dict(sections=(8, 8, 8, 8), scaling="bands", factor=8.0, original_len=8192),
    dict(sections=(6, 4, 6), order="cycled", frequencies="own", scaling="yarn", factor=16.0, original_len=4096),
    dict(sections=(7, 2, 3), frequencies="own", scaling="base", factor=4.0),
    dict(sections=(3, 4, 9), scaling="linear", factor=0.25),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("plan", range(len(PLANS)))
def test_matches_formula(plan, D, dt):
    kw = PLANS[plan]
    p = b.RopeAxesPlan(**kw)
    A = len(kw["sections"])
    for T, Hq, Hk in ((1, 1, 1), (3, 8, 2), (700, 4, 1)):
        q, k = randn((T, Hq, D), dt, T), randn((T, Hk, D), dt, T + 1)
        pos = torch.from_numpy(np.random.default_rng(T).integers(-5, 1 << 20, (A, T)).astype(np.int32))
        qo, ko = b.rope_axes(q.cuda(), k.cuda(), pos.cuda(), p)
        close(qo.cpu(), q, pos, kw)
        close(ko.cpu(), k, pos, kw)


def test_full_heads_strides_in_place_and_append():
    kw = dict(sections=(16, 24, 24))
    p = b.RopeAxesPlan(**kw)
    T, Hq, Hk, D, B, NB = 33, 8, 2, 128, 16, 9
    for dt in ("bf16", "f32"):
        qkv = randn((T, (Hq + 2 * Hk) * D), dt, 5).cuda()
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
        wide = torch.from_numpy(np.random.default_rng(0).integers(0, 9000, (3, T + 7)).astype(np.int32)).cuda()
        pos = wide[:, 2: 2 + T]                          # axes further apart than the tokens
        slots = torch.randperm(NB * B, generator=torch.Generator().manual_seed(1))[:T].cuda()
        slots[4] = -1
        kp, vp = (torch.zeros(NB, Hk, B, D, dtype=DT[dt], device="cuda") for _ in range(2))
        before = qkv.clone()
        qo = b.rope_axes_append(q, k, v, pos, slots, p, kp, vp)
        assert b.get_error() == 0 and torch.equal(qkv, before)
        close(qo.cpu(), q.cpu().contiguous(), pos.cpu(), kw)
        keep = [i for i in range(T) if i != 4]
        sl = slots[keep]
        got_k, got_v = kp[sl // B, :, sl % B], vp[sl // B, :, sl % B]
        close(got_k.cpu(), k.cpu()[keep], pos.cpu()[:, keep], kw)
        assert torch.equal(got_v, v[keep])
        b.rope_axes(q, k, pos, p, q_out=q, k_out=k)      # in place
        assert torch.equal(q, qo) and torch.equal(k[keep], got_k)
        assert int((kp.abs().sum(-1) > 0).sum()) == (T - 1) * Hk


def test_one_axis_equals_rope():
    q, k = randn((50, 4, 128), "bf16", 1).cuda(), randn((50, 2, 128), "bf16", 2).cuda()
    pos = torch.arange(50, dtype=torch.int32, device="cuda") * 977
    for layout in ("half", "interleaved"):
        a = b.rope(q, k, pos, b.RopePlan(96, layout=layout))
        z = b.rope_axes(q, k, pos[None], b.RopeAxesPlan((48,), layout=layout))
        same = b.rope_axes(q, k, pos[None].expand(3, -1), b.RopeAxesPlan((10, 20, 18), layout=layout, order="cycled"))
        assert all(torch.equal(x, y) and torch.equal(x, w) for x, y, w in zip(a, z, same))
