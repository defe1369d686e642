"""Edges of the step operators' calls: slots past the pool wherever they lie in a block, one-shot calls
on another stream than the current one."""
import pytest
import torch

from paged_kv_cache_47_gb300 import binding as b

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [8, 16, 32])
@pytest.mark.parametrize("off", [0, 3, -1])
def test_block_means_flags_every_slot_past_the_pool(off, B):
    NB = 4
    k = torch.randn(NB, 2, B, 64, device="cuda").bfloat16()
    means = torch.full((NB, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([5, NB * B + off % B], device="cuda")
    b.block_means(slots, k, means)
    assert b.get_error() == b.DEVERR_SLOT and (means == 9).all()


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("call", ["q4", "sparse", "select", "gather", "rope", "rope_append"])
def test_one_shot_calls_allocate_on_their_stream(call, raw):
    """The current stream is busy and its allocator's free memory is not zero: a call on another
    stream has its outputs and its zero-filled workspace from there."""
    S, Hk, G, D, B, n = 5, 2, 4, 128, 16, 60
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(S, Hk * G, D, device="cuda", generator=g).bfloat16()
    k, v = (torch.randn(S * n, Hk, B, D, device="cuda", generator=g).bfloat16() for _ in range(2))
    means = k.float().mean(2).bfloat16()
    tab = torch.randperm(S * n, device="cuda", generator=g).int().view(S, n)
    lens = torch.full((S,), n * B - 3, dtype=torch.int32, device="cuda")
    cache = b.Q4Cache.empty(S * n, Hk, B, D)
    rows = [x.transpose(1, 2).reshape(-1, Hk, D).contiguous() for x in (k, v)]
    slots = torch.arange(S * n * B, device="cuda")
    b.append_q4(*rows, slots, cache)
    plan, pos = b.RopePlan(D), torch.arange(S, dtype=torch.int32, device="cuda")
    calls = {
        "q4": lambda **kw: b.decode_attention_q4(q, cache, tab, lens, 0.09, **kw),
        "sparse": lambda **kw: b.decode_attention_sparse(q, k, v, means, tab, lens, 0.09, 20, **kw),
        "select": lambda **kw: b.select_blocks(q, k, means, tab, lens, 20, **kw)[0],
        "gather": lambda **kw: b.gather_q4(slots[:99], cache, **kw)[1],
        "rope": lambda **kw: b.rope(q, q, pos, plan, **kw)[0],
        "rope_append": lambda **kw: b.rope_append(q, q[:, :Hk], q[:, Hk: 2 * Hk], pos, slots[:S], plan, k.clone(), v.clone(), **kw),
    }
    want = calls[call]()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):                       # (this stream's first allocations)
        calls[call]()
    torch.cuda.synchronize()
    for size in (1 << 10, 1 << 14, 1 << 17, 1 << 20, 1 << 22, 1 << 24):
        for x in [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]:
            del x
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                   # a tenth of a second of the current stream
    if call == "rope_append":                        # (its pools are copies made for the call)
        torch.cuda.synchronize()
    got = []
    for _ in range(3):
        x = calls[call](stream=s.cuda_stream if raw else s)
        with torch.cuda.stream(s):
            got.append(x.clone())
    s.synchronize()
    for x in got:
        assert torch.equal(x, want)
    assert b.get_error() == 0
    torch.cuda.synchronize()
