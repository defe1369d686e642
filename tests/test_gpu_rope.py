"""Rotary positions on the GPU against the formula in 64 bits, element by element.

Tolerance of one element y = x_a c - x_b s (n = |x_a| + |x_b|, A the amplitude): cosine and sine
are fp32 values off by at most 2^-22 A (angle rounded to fp32 in half turns, at most pi 2^-25;
sincospif within 2 ulp of values up to 1, 2^-23; times the amplitude, 2^-24), and the two products
and their sum add less than 2^-23 of n A. Together below 2^-21 n A, then half a step of the output's
type. Copied elements are equal."""
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
    """got against x turned; both CPU tensors [T][H][D]."""
    rot = {k: v for k, v in kw.items() if k != "layout"}
    w, amp = O.rope_frequencies(**{"base": 10000.0, **rot})
    want, size = O.rope(x.double().numpy(), pos.numpy(), w, amp, kw.get("layout", "half"))
    rd = 2 * len(w)
    tol = size * amp * 2.0 ** -21 + np.abs(want) * torch.finfo(x.dtype).eps / 2
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25                     # half a step among the subnormal numbers
    bad = np.abs(got.double().numpy() - want)[..., :rd] > tol[..., :rd]
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3])
    assert torch.equal(got[..., rd:], x[..., rd:])


PLANS = [
    dict(rotary_dim=128), dict(rotary_dim=128, layout="interleaved"),
    dict(rotary_dim=64, base=500000.0, scaling="bands", factor=8.0, original_len=8192),
    dict(rotary_dim=32, layout="interleaved", scaling="linear", factor=4.0),
    dict(rotary_dim=20, scaling="base", factor=4.0),
    dict(rotary_dim=20, layout="interleaved", scaling="yarn", factor=16.0, original_len=4096),
    dict(rotary_dim=2), dict(rotary_dim=8, layout="interleaved"), dict(rotary_dim=24),
]


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("plan", range(len(PLANS)))
def test_rope_matches_formula(plan, D, dt):
    kw = PLANS[plan]
    if kw["rotary_dim"] > D:
        kw = {**kw, "rotary_dim": D}
    p = b.RopePlan(**kw)
    for T, Hq, Hk in ((1, 1, 1), (3, 8, 2), (300, 5, 5), (700, 4, 1)):
        q, k = randn((T, Hq, D), dt, T), randn((T, Hk, D), dt, T + 1)
        pos = torch.from_numpy(np.random.default_rng(T).integers(0, 1 << 20, T).astype(np.int32))
        pos[0] = 0
        if T > 2:
            pos[1], pos[2] = 2 ** 31 - 1, -5
        qo, ko = b.rope(q.cuda(), k.cuda(), pos.cuda(), p)
        close(qo.cpu(), q, pos, kw)
        close(ko.cpu(), k, pos, kw)


def test_far_positions_keep_their_angles():
    # whole range of int32: the angle is reduced without rounding
    kw = dict(rotary_dim=128)
    pos = torch.from_numpy(np.random.default_rng(0).integers(-2 ** 31, 2 ** 31, 2000).astype(np.int32))
    q = randn((2000, 1, 128), "f32", 3)
    qo, _ = b.rope(q.cuda(), q.cuda(), pos.cuda(), b.RopePlan(**kw))
    # the fractions of a turn are off by up to 2^-52 of a turn a position (double), 2^-21 turns at 2^31
    w, amp = O.rope_frequencies(base=10000.0, **kw)
    want, size = O.rope(q.double().numpy(), pos.numpy(), w, amp, "half")
    tol = size * (2.0 ** -21 + 2 * np.pi * 2.0 ** -21)
    assert (np.abs(qo.cpu().double().numpy() - want) <= tol + np.abs(want) * 2.0 ** -24).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("layout,rd", [("half", 64), ("interleaved", 64), ("half", 20)])
def test_in_place_and_strided_views(layout, rd, dt):
    T, Hq, Hk, D = 37, 6, 2, 64
    kw = dict(rotary_dim=rd, layout=layout)
    qkv = randn((T, (Hq + 2 * Hk) * D + 16), dt, 0).cuda()
    before = qkv.clone()
    q = qkv[:, : Hq * D].unflatten(1, (Hq, D))
    k = qkv[:, Hq * D: (Hq + Hk) * D].unflatten(1, (Hk, D))
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 3
    qo, ko = b.rope(q, k, pos, b.RopePlan(**kw))                    # strided in, dense out
    b.rope(q, k, pos, b.RopePlan(**kw), q_out=q, k_out=k)           # in place
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])
    close(qo.cpu(), before[:, : Hq * D].unflatten(1, (Hq, D)).cpu(), pos.cpu(), kw)


@pytest.mark.parametrize("dt", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("T,Hq,Hk,D,rd,layout", [(1, 4, 1, 64, 64, "half"), (64, 32, 8, 128, 128, "half"),
                                                 (501, 3, 3, 64, 20, "interleaved"),
                                                 (700, 10, 5, 128, 64, "interleaved")])
def test_rope_append_equals_rope_then_append(T, Hq, Hk, D, rd, layout, B, dt):
    rng = np.random.default_rng([T, B])
    q, k, v = (randn((T, h, D), dt, i).cuda() for i, h in enumerate((Hq, Hk, Hk)))
    NB = -(-T // B) + 2
    slots = rng.permutation(NB * B)[:T]
    slots[rng.random(T) < 0.1] = -1
    slots = torch.from_numpy(slots).cuda()
    pos = torch.from_numpy(rng.integers(0, 40000, T).astype(np.int32)).cuda()
    plan = b.RopePlan(rd, layout=layout)
    pools = [torch.full((NB, Hk, B, D), 3.5, dtype=DT[dt], device="cuda") for _ in range(4)]
    qo = b.rope_append(q, k, v, pos, slots, plan, pools[0], pools[1])
    q2, k2 = b.rope(q, k, pos, plan)
    b.append(k2, v, slots, pools[2], pools[3])
    assert torch.equal(qo, q2)
    assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
    assert b.get_error() == 0
    close(q2.cpu(), q.cpu(), pos.cpu(), dict(rotary_dim=rd, layout=layout))


def test_rope_append_flags_slots_past_the_pool():
    q = randn((3, 2, 64), "bf16", 0).cuda()
    kp, vp = (torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.tensor([5, 64, 1 << 40], device="cuda")
    pos = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    qo = b.rope_append(q, q, q, pos, slots, b.RopePlan(64), kp, vp)
    assert b.get_error() == b.DEVERR_SLOT
    close(qo.cpu(), q.cpu(), pos.cpu(), dict(rotary_dim=64))
    assert vp[0, :, 5].equal(q[0]) and int((vp != 0).any(-1).sum()) == 2


def test_other_stream_and_graph():
    q = randn((9, 2, 64), "f16", 0).cuda()
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    plan = b.RopePlan(64)
    want, _ = b.rope(q, q, pos, plan)
    out, ko = torch.zeros_like(q), torch.zeros_like(q)
    call = b.prepared_rope(q, q, pos, plan, q_out=out, k_out=ko)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for shift in (0, 7):
        pos.copy_(torch.arange(9, device="cuda") + shift)
        g.replay()
        assert torch.equal(out, b.rope(q, q, pos, plan)[0])
