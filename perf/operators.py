"""Operators of a paged KV-cache decode step, as cases to measure: plain forms and the library's calls.

Four groups, in the order in which a serving loop calls them:

  tables   finished requests give their blocks back, the others get blocks and slots for their new
           tokens, all on the GPU (`tables_release`, then `tables_append`)
  rope     rotary positions of q and k, k and v written to their slots (`rope_append`)
  store    K/V rows quantized to 4 bits at their slots, and read back as values (`append_q4`, `gather_q4`)
  q4       decode attention over a 4-bit cache (`decode_attention_q4`)
  sparse   block means of the step's finished blocks, then decode attention over the blocks that the
           means select for each sequence and kv head (`block_means`, `decode_attention_sparse`)

Layouts are those of the library: pools [blocks][kv heads][block size][head size], tables
[sequences][blocks] int32, lengths [sequences] int32, slots int64.
"""
import functools
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}
GROUP = 32          # elements that share one scale and one minimum in the 4-bit cache


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of the benchmark's batch: 64 requests, a token each, a few finished and begun
        {"name": "tables_step", "kind": "tables", "S": 64, "B": 16, "M": 256, "lo": 512, "hi": 4080,
         "add_lo": 1, "add_hi": 1, "done": 0.05, "new_lo": 1, "new_hi": 1},
        # an admission wave: 997 requests, a fifth of them replaced by prompts of up to 2000 tokens
        {"name": "tables_admission", "kind": "tables", "S": 997, "B": 16, "M": 300, "lo": 0, "hi": 2700,
         "add_lo": 0, "add_hi": 8, "done": 0.2, "new_lo": 1, "new_hi": 2000},
        # the benchmark's decode step: 64 tokens, 32 q and 8 kv heads
        {"name": "rope_step", "kind": "rope", "T": 64, "Hq": 32, "Hk": 8, "D": 128, "rd": 128, "B": 16,
         "dt": "bf16", "layout": "half", "scaling": "bands", "base": 500000.0, "far": 131072, "packed": True},
        # a wave of prompts over as many kv heads as q heads, half of each head rotated, in
        # neighbouring pairs, odd token count, some tokens of a padded batch without a slot
        {"name": "rope_prompts", "kind": "rope", "T": 8191, "Hq": 40, "Hk": 40, "D": 128, "rd": 64, "B": 16,
         "dt": "f16", "layout": "interleaved", "scaling": "yarn", "base": 10000.0, "far": 65536, "packed": False},
        # new rows of one decode step into the 4-bit cache
        {"name": "store_step", "kind": "store", "T": 64, "Hk": 8, "D": 128, "B": 16, "dt": "bf16"},
        # a wave of prompts into the 4-bit cache
        {"name": "store_prompts", "kind": "store", "T": 16383, "Hk": 8, "D": 128, "B": 32, "dt": "f16"},
        # one interactive request: latency
        {"name": "q4_one", "kind": "q4", "S": 1, "Hq": 32, "Hk": 8, "D": 128, "B": 16, "dt": "bf16",
         "lo": 1000, "hi": 1000},
        # the benchmark's batch over a 4-bit cache
        {"name": "q4_batch", "kind": "q4", "S": 64, "Hq": 32, "Hk": 8, "D": 128, "B": 16, "dt": "bf16",
         "lo": 512, "hi": 4096},
        # one q head for each kv head, 256 short contexts
        {"name": "q4_heads", "kind": "q4", "S": 256, "Hq": 40, "Hk": 40, "D": 128, "B": 16, "dt": "f16",
         "lo": 128, "hi": 2048},
        # eight long agent contexts, 8 q heads to a kv head
        {"name": "q4_long", "kind": "q4", "S": 8, "Hq": 64, "Hk": 8, "D": 128, "B": 32, "dt": "bf16",
         "lo": 32768, "hi": 131072},
        # the benchmark's batch, about a quarter of its blocks read
        {"name": "sparse_batch", "kind": "sparse", "S": 64, "Hq": 32, "Hk": 8, "D": 128, "B": 16, "dt": "bf16",
         "lo": 512, "hi": 4096, "top": 32, "first": 1, "last": 4},
        # eight long agent contexts, 4096 tokens chosen of up to 131072
        {"name": "sparse_long", "kind": "sparse", "S": 8, "Hq": 64, "Hk": 8, "D": 128, "B": 16, "dt": "bf16",
         "lo": 32768, "hi": 131072, "top": 240, "first": 4, "last": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["tables", "rope", "store", "q4", "sparse"])
    B = rng.choice([8, 16, 32])
    if kind == "tables":
        S = _log(rng, 1, 997)
        hi = _log(rng, 1, 2000)
        new_hi = _log(rng, 1, 2000)
        return {"kind": kind, "S": S, "B": B, "M": -(-(hi + new_hi + 8) // B) + rng.randint(0, 40), "lo": 0,
                "hi": hi, "add_lo": rng.randint(0, 1), "add_hi": rng.randint(1, 8),
                "done": rng.choice([0.0, 0.1, 0.5]), "new_lo": 0, "new_hi": new_hi}
    D = rng.choice([64, 128])
    if kind == "rope":
        Hk = rng.choice([1, 2, 5, 8, 40])
        return {"kind": kind, "T": _log(rng, 1, 8000), "Hq": Hk * rng.choice([1, 4, 7]) if Hk < 40 else 40, "Hk": Hk,
                "D": D, "rd": rng.choice([D, D // 2, D // 4, 20]), "B": B, "dt": rng.choice(["f16", "bf16", "f32"]),
                "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "base", "bands", "yarn"]),
                "base": rng.choice([10000.0, 500000.0]), "far": _log(rng, 100, 1 << 20),
                "packed": rng.choice([False, True])}
    dt = rng.choice(["f16", "bf16"])
    if kind == "store":
        return {"kind": kind, "T": _log(rng, 1, 16000), "Hk": rng.choice([1, 2, 5, 8]), "D": D, "B": B, "dt": dt}
    Hk = rng.choice([1, 2, 3, 8])
    Hq = Hk * rng.choice([1, 3, 4, 8, 12] if Hk < 8 else [1, 4, 5, 8])
    hi = _log(rng, 1, 40000)
    S = max(1, min(_log(rng, 1, 300), 250000 // hi))
    case = {"kind": kind, "S": S, "Hq": Hq, "Hk": Hk, "D": D, "B": B, "dt": dt, "lo": hi // rng.choice([2, 4, 20]),
            "hi": hi}
    if kind == "sparse":
        if rng.random() < 0.2:
            case["dt"] = "f32"
        case |= {"top": _log(rng, 1, 240), "first": rng.randint(0, 4), "last": rng.randint(1, 12)}
    return case


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _lengths(case, rng):
    return rng.integers(case["lo"], case["hi"] + 1, size=case["S"]).astype(np.int64)


def _tables(case, rng):
    """Lengths, tables of randomly scattered blocks, and the pool's size: room for every request at its longest."""
    lens = _lengths(case, rng)
    n = -(-lens // case["B"])
    M = max(1, int(n.max())) + 1
    NB = case["S"] * -(-case["hi"] // case["B"]) + 3
    perm = rng.permutation(NB)[: int(n.sum())]
    tab = np.full((case["S"], M), -1, np.int32)
    tab[np.arange(M)[None, :] < n[:, None]] = perm
    return lens, n, tab, NB


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _randn(shape, dt, g, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(DT[dt])


def _new_tokens(case):
    """Tokens that a step of `case` adds, about."""
    turn = round(case["S"] * case["done"])
    return (max(0, case["S"] - 2 * turn) * (case["add_lo"] + case["add_hi"])
            + min(turn, case["S"] - turn) * (case["new_lo"] + case["new_hi"])) / 2


def prepare(case, seed):
    rng = np.random.default_rng([int(seed), 7])
    g = _gen(seed)
    st = {"case": case}
    kind = case["kind"]
    if kind == "tables":
        S, B, M = case["S"], case["B"], case["M"]
        # as many requests finish as new ones begin, in rows that were empty; the others go on
        turn = int(round(S * case["done"]))
        done, fresh = np.arange(S) < turn, np.arange(S) >= max(turn, S - turn)
        spread = lambda lo, hi, m: rng.permutation(np.linspace(lo, hi, m).round().astype(np.int64))  # noqa: E731
        lens = np.where(fresh, 0, rng.integers(case["lo"], case["hi"] + 1, size=S))
        add = np.where(done, 0, spread(case["add_lo"], case["add_hi"], S))
        add[fresh] = spread(case["new_lo"], case["new_hi"], int(fresh.sum()))
        order = rng.permutation(S)
        done, lens, add = done[order], lens[order], add[order]
        n = -(-lens // B)
        NB = S * M
        perm = rng.permutation(NB).astype(np.int32)
        tab = np.full((S, M), -1, np.int32)
        tab[np.arange(M)[None, :] < n[:, None]] = perm[: int(n.sum())]
        spare = NB - int(n.sum())
        free = np.full(NB, -1, np.int32)
        free[:spare] = perm[int(n.sum()):]
        # the token buffers have room for the largest step of such a program
        tokens = S * case["add_hi"] + turn * case["new_hi"] if S < 8 else int(1.02 * _new_tokens(case)) + 8
        st |= {"NB": NB, "tables": _dev(tab), "lens": _dev(lens.astype(np.int32)), "done": _dev(done),
               "add": _dev(add.astype(np.int32)), "free": _dev(free),
               "num_free": torch.tensor([spare], dtype=torch.int32, device="cuda"), "max_tokens": max(1, tokens)}
        return st
    if kind == "rope":
        T, Hq, Hk, D, B = (case[k] for k in ("T", "Hq", "Hk", "D", "B"))
        if case["packed"]:      # q, k and v are parts of one projection's output
            qkv = _randn((T, (Hq + 2 * Hk) * D), case["dt"], g)
            q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
        else:
            q, k, v = (_randn((T, h, D), case["dt"], g) for h in (Hq, Hk, Hk))
        NB = -(-T // B) + 3
        slots = rng.permutation(NB * B)[:T].astype(np.int64)
        if not case["packed"]:
            slots[rng.random(T) < 0.02] = -1
        pos = rng.integers(0, case["far"], size=T).astype(np.int32)
        st |= {"q": q, "k": k, "v": v, "slots": _dev(slots), "pos": _dev(pos),
               "k_pool": torch.zeros(NB, Hk, B, D, dtype=DT[case["dt"]], device="cuda"),
               "v_pool": torch.zeros(NB, Hk, B, D, dtype=DT[case["dt"]], device="cuda"),
               "q_out": torch.empty(T, Hq, D, dtype=DT[case["dt"]], device="cuda")}
        return st
    Hk, D, B = case["Hk"], case["D"], case["B"]
    NG = D // GROUP
    if kind == "store":
        T = case["T"]
        NB = -(-T // B) + 3
        k = _randn((T, Hk, D), case["dt"], g) * (1 + 9 * (torch.arange(D, device="cuda") % 41 == 0)).to(DT[case["dt"]])
        v = _randn((T, Hk, D), case["dt"], g)
        st |= {"k": k, "v": v, "slots": _dev(rng.permutation(NB * B)[:T].astype(np.int64))}
        st |= _empty_q4(NB, Hk, B, D)
        return st
    lens, n, tab, NB = _tables(case, rng)
    st |= {"tables": _dev(tab), "lens": _dev(lens.astype(np.int32)), "NB": NB, "scale": 1 / math.sqrt(D),
           "q": _randn((case["S"], case["Hq"], D), case["dt"], g)}
    # positions that no context holds: what a pool has there is not to be used
    used = np.zeros(NB, np.int64)
    valid = np.clip(lens[:, None] - np.arange(tab.shape[1])[None, :] * B, 0, B)
    used[tab[tab >= 0]] = valid[tab >= 0]
    dead = _dev(np.arange(B)[None, :] >= used[:, None])          # [NB][B]
    if kind == "q4":
        st |= _empty_q4(NB, Hk, B, D)
        st["k_codes"].random_(0, 256, generator=g)
        st["v_codes"].random_(0, 256, generator=g)
        for name, rows in (("k", True), ("v", False)):
            s = torch.rand(NB, Hk, B, NG, device="cuda", generator=g) * 0.3 + 0.15
            m = -7.5 * s + torch.randn(NB, Hk, B, NG, device="cuda", generator=g) * 0.3
            p = torch.cat([s, m], -1).masked_fill_(dead[:, None, :, None], math.nan).half()
            st[name + "_params"].copy_(p if rows else p.transpose(2, 3))
        return st
    k_pool, v_pool = (_randn((NB, Hk, B, D), case["dt"], g) for _ in range(2))
    # neighbouring tokens are alike: each block's keys lean to one direction
    k_pool.mul_(0.7).add_(_randn((NB, Hk, 1, D), case["dt"], g, 0.7))
    means = _means(k_pool)
    for p in (k_pool, v_pool):
        p.masked_fill_(dead[:, None, :, None], math.nan)
    full = _dev((used == B))
    means.masked_fill_(~full[:, None, None], math.nan)
    last = tab[np.arange(case["S"]), np.maximum(n - 1, 0)].astype(np.int64)
    slots = np.where(lens > 0, last * B + (lens - 1) % B, -1)
    means[_dev(last[(lens > 0) & (lens % B == 0)])] = math.nan        # the pass computes these
    st |= {"k_pool": k_pool, "v_pool": v_pool, "k_means": means, "slots": _dev(slots)}
    return st


def _empty_q4(NB, Hk, B, D):
    NG = D // GROUP
    new = functools.partial(torch.zeros, device="cuda")
    return {"k_codes": new(NB, Hk, B, D // 2, dtype=torch.uint8), "v_codes": new(NB, Hk, B, D // 2, dtype=torch.uint8),
            "k_params": new(NB, Hk, B, 2 * NG, dtype=torch.float16),
            "v_params": new(NB, Hk, 2 * NG, B, dtype=torch.float16)}


# ------------------------------------------------------------------------------- the library's calls
def _rope_args(case):
    more = {"none": {}, "linear": {"factor": 4.0}, "base": {"factor": 4.0},
            "bands": {"factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0, "original_len": 8192},
            "yarn": {"factor": 16.0, "beta_fast": 32.0, "beta_slow": 1.0, "original_len": 4096}}[case["scaling"]]
    return {"rotary_dim": case["rd"], "base": case["base"], "layout": case["layout"], "scaling": case["scaling"], **more}


def _calls(st):
    """The library's calls of one pass, prepared as a serving loop prepares them, and their outputs."""
    from paged_kv_cache_47_gb300 import binding as b

    case = st["case"]
    kind = case["kind"]
    i32 = functools.partial(torch.empty, dtype=torch.int32, device="cuda")
    if kind == "tables":
        S = case["S"]
        mid, last, freed, left = i32(S), i32(S), i32(1), i32(1)
        slots = torch.empty(st["max_tokens"], dtype=torch.int64, device="cuda")
        pos, offs = i32(st["max_tokens"]), i32(S + 1)
        ws = b.alloc_tables_workspace()
        calls = (b.prepared_tables_release(st["tables"], st["lens"], st["done"], st["free"], st["num_free"], case["B"],
                                           workspace=ws, context_lens_out=mid, num_free_out=freed),
                 b.prepared_tables_append(st["tables"], mid, st["add"], st["free"], freed, case["B"], slots, pos, offs,
                                          workspace=ws, context_lens_out=last, num_free_out=left))
        return calls, {"tables": st["tables"], "free": st["free"], "lens": last, "num_free": left, "slots": slots,
                       "positions": pos, "offsets": offs}
    if kind == "rope":
        plan = b.RopePlan(**_rope_args(case))
        call = b.prepared_rope_append(st["q"], st["k"], st["v"], st["pos"], st["slots"], plan, st["k_pool"],
                                      st["v_pool"], q_out=st["q_out"])
        return (call,), {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    if kind == "sparse":
        sel = i32(case["S"], case["Hk"], case["top"] + case["first"] + case["last"]), i32(case["S"], case["Hk"])
        ws = b.alloc_sparse_workspace(st["k_pool"], case["S"], case["Hq"], st["tables"].shape[1])
        out = torch.empty_like(st["q"])
        calls = (b.prepared_block_means(st["slots"], st["k_pool"], st["k_means"]),
                 b.prepared_decode_attention_sparse(
                     st["q"], st["k_pool"], st["v_pool"], st["k_means"], st["tables"], st["lens"], st["scale"],
                     top_blocks=case["top"], first_blocks=case["first"], last_blocks=case["last"], out=out,
                     sel_tables=sel[0], sel_lens=sel[1], workspace=ws))
        return calls, {"out": out, "sel_tables": sel[0], "sel_lens": sel[1], "k_means": st["k_means"]}
    cache = b.Q4Cache(st["k_codes"], st["v_codes"], st["k_params"], st["v_params"], DT[case["dt"]])
    if kind == "store":
        k, v = torch.empty_like(st["k"]), torch.empty_like(st["v"])
        calls = (b.prepared_append_q4(st["k"], st["v"], st["slots"], cache),
                 b.prepared_gather_q4(st["slots"], cache, k, v))
        return calls, {"k": k, "v": v}
    out = torch.empty_like(st["q"])
    call = b.prepared_decode_attention_q4(st["q"], cache, st["tables"], st["lens"], st["scale"], out=out,
                                          workspace=b.alloc_q4_workspace(cache, case["Hq"]))
    return (call,), {"out": out}


def _own(st):
    if "calls" not in st:       # what a program makes once and keeps: plans, workspaces, outputs, arguments
        st["calls"] = _calls(st)
    calls, outputs = st["calls"]
    [call() for call in calls]
    return outputs


# -------------------------------------------------------------------------------------- plain forms
def _plain_tables(st):
    B, M, NB = st["case"]["B"], st["case"]["M"], st["NB"]
    tab, lens, done = st["tables"].long(), st["lens"].long(), st["done"]
    S = tab.shape[0]
    nf, free = st["num_free"].long(), st["free"].long()
    # release: the blocks of finished requests go on the stack of free blocks, in table order
    held = torch.where(done, (lens + B - 1) // B, 0)
    at = nf + torch.cumsum(held, 0) - held
    j = torch.arange(M, device="cuda")
    put = j < held[:, None]
    free = torch.cat([free, free.new_empty(1)])
    free[torch.where(put, at[:, None] + j, NB)] = tab
    free = free[:NB]
    nf = nf + held.sum()
    lens = torch.where(done, 0, lens)
    # append: blocks from the top of the stack, request after request
    add = st["add"].long()
    have, after = (lens + B - 1) // B, (lens + add + B - 1) // B
    take = torch.cumsum(after - have, 0) - (after - have)
    k = nf - 1 - (take - have)[:, None] - j
    fresh = (j >= have[:, None]) & (j < after[:, None])
    tab = torch.where(fresh, free[k.clamp(0, NB - 1)], tab)
    offs = torch.cat([add.new_zeros(1), torch.cumsum(add, 0)])
    i = torch.arange(st["max_tokens"], device="cuda")
    s = torch.searchsorted(offs[1:], i, right=True).clamp(max=S - 1)
    real = i < offs[-1]
    pos = torch.where(real, lens[s] + i - offs[s], 0)
    slots = torch.where(real, tab[s, (pos // B).clamp(max=M - 1)] * B + pos % B, -1)
    st["tables"].copy_(tab)
    st["free"].copy_(free)
    return {"tables": st["tables"], "free": st["free"], "lens": (lens + add).int(),
            "num_free": (nf - (after - have).sum()).int(), "slots": slots, "positions": pos.int(),
            "offsets": offs.int()}


def _frequencies(case):
    """Radians a position of each rotated pair, and the factor on cos and sin, in 64 bits."""
    a = _rope_args(case)
    rd, base, f = a["rotary_dim"], a["base"], a.get("factor", 1.0)
    if a["scaling"] == "base":
        base = base * f ** (rd / (rd - 2))
    i = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    w = base ** (-2 * i / rd)
    if a["scaling"] == "linear":
        return w / f, 1.0
    if a["scaling"] == "bands":
        n, lo, hi = a["original_len"], a["low_freq_factor"], a["high_freq_factor"]
        turns = n * w / (2 * math.pi)
        mix = ((turns - lo) / (hi - lo)).clamp(0, 1)
        return w * mix + w / f * (1 - mix), 1.0
    if a["scaling"] == "yarn":
        at = lambda turns: rd * math.log(a["original_len"] / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(at(a["beta_fast"]))), min(rd - 1, math.ceil(at(a["beta_slow"])))
        mix = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return w * (1 - mix) + w / f * mix, 0.1 * math.log(f) + 1
    return w, 1.0


def _rotate(x, cos, sin, case):
    rd = case["rd"]
    y = x.float()
    r = y[..., :rd]
    if case["layout"] == "half":
        a, b = r[..., :rd // 2], r[..., rd // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([r, y[..., rd:]], -1).to(x.dtype)


def _plain_rope(st):
    case = st["case"]
    w, amp = _frequencies(case)
    angle = (st["pos"].double()[:, None] * w)[:, None]
    cos, sin = (torch.cos(angle) * amp).float(), (torch.sin(angle) * amp).float()
    st["q_out"].copy_(_rotate(st["q"], cos, sin, case))
    B = case["B"]
    keep = torch.nonzero(st["slots"] >= 0)[:, 0]
    slot = st["slots"][keep]
    st["k_pool"][slot // B, :, slot % B] = _rotate(st["k"], cos, sin, case)[keep]
    st["v_pool"][slot // B, :, slot % B] = st["v"][keep]
    return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _quantize(x):
    """Codes 0..15 (as fp32), scale and minimum (fp16) of each group of 32 elements."""
    g = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = g.amin(-1), g.amax(-1)
    m = lo.clamp(-65504, 65504).half()
    s = ((hi - lo) / 15).clamp(max=65504).half()
    c = ((g - m.float()[..., None]) / s.float()[..., None]).round().clamp(0, 15)
    return torch.where(s[..., None] > 0, c, 0.0), s, m


def _pack(c, rows):
    """Codes [..., groups, 32] as the bytes of a cached row: K keeps 8 elements of a group together, V 4."""
    n = 8 if rows else 4
    c = c.unflatten(-1, (-1, n)).transpose(-3, -2).reshape(*c.shape[:-2], -1, 2).to(torch.uint8)
    return c[..., 0] | (c[..., 1] << 4)


def _unpack(codes, rows):
    """Codes [..., groups, 32] as fp32."""
    n = 8 if rows else 4
    D = codes.shape[-1] * 2
    c = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], GROUP // n, D // GROUP, n)
    return c.transpose(-3, -2).reshape(*codes.shape[:-1], D // GROUP, GROUP).float()


def _plain_store(st):
    B = st["case"]["B"]
    blk, off = st["slots"] // B, st["slots"] % B
    NG = st["case"]["D"] // GROUP
    (kc, ks, km), (vc, vs, vm) = _quantize(st["k"]), _quantize(st["v"])
    st["k_codes"][blk, :, off] = _pack(kc, True)
    st["v_codes"][blk, :, off] = _pack(vc, False)
    st["k_params"][blk, :, off] = torch.cat([ks, km], -1)
    st["v_params"][blk, :, :, off] = torch.cat([vs, vm], -1)
    kp, vp = st["k_params"][blk, :, off].float(), st["v_params"][blk, :, :, off].float()
    k = _unpack(st["k_codes"][blk, :, off], True) * kp[..., :NG, None] + kp[..., NG:, None]
    v = _unpack(st["v_codes"][blk, :, off], False) * vp[..., :NG, None] + vp[..., NG:, None]
    return {"k": k.flatten(-2).to(st["k"].dtype), "v": v.flatten(-2).to(st["k"].dtype)}


def _attend(q, k, v, live, scale):
    """q [S][Hk][G][D], k and v [S][Hk][N][D], live [S][1 or Hk][N]."""
    z = torch.matmul(q, k.transpose(-1, -2)) * scale
    z = z.masked_fill_(~live[:, :, None], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True).clamp(min=-3e38))
    return torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-37)


def _plain_q4(st):
    case = st["case"]
    S, Hk, D, B = case["S"], case["Hk"], case["D"], case["B"]
    NG = D // GROUP
    tab = st["tables"].clamp(min=0).long()
    live = (torch.arange(tab.shape[1] * B, device="cuda") < st["lens"][:, None])[:, None]
    kp = st["k_params"][tab].float()
    k = (_unpack(st["k_codes"][tab], True) * kp[..., :NG, None]).add_(kp[..., NG:, None]).flatten(-2)
    k = k.transpose(1, 2).reshape(S, Hk, -1, D).masked_fill_(~live[..., None], 0)
    vp = st["v_params"][tab].transpose(-1, -2).float()
    v = (_unpack(st["v_codes"][tab], False) * vp[..., :NG, None]).add_(vp[..., NG:, None]).flatten(-2)
    v = v.transpose(1, 2).reshape(S, Hk, -1, D).masked_fill_(~live[..., None], 0)
    q = st["q"].float().unflatten(1, (Hk, -1))
    return {"out": _attend(q, k, v, live, st["scale"]).flatten(1, 2).to(st["q"].dtype)}


def _means(k):
    """Mean key of each block [..., B, D]: rows added in order in 32 bits, rounded once."""
    return (functools.reduce(torch.add, k.float().unbind(-2)) / k.shape[-2]).to(k.dtype)


def _scores(q, means):
    """Score of each block for a kv head: the largest of its q heads' products with the mean key.
    The order of the additions is part of the definition, so that equal inputs select equal blocks: eight
    neighbouring elements one after another, then neighbouring sums in pairs."""
    x = functools.reduce(torch.add, (q * means).unflatten(-1, (-1, 8)).unbind(-1))
    pair = lambda x, _: x[..., 0::2] + x[..., 1::2]  # noqa: E731
    return functools.reduce(pair, range(int(math.log2(x.shape[-1]))), x)[..., 0].amax(-1)


def _choose(score, n, top, first, last):
    """Which blocks [S][N][Hk] are read: the first and last ones, and the best of those between."""
    j = torch.arange(score.shape[1], device="cuda")[None, :, None]
    n = n[:, None, None]
    between = (j >= first) & (j < n - last)
    order = torch.where(between, torch.where(score.isnan(), math.inf, score), -math.inf)
    order = torch.sort(order, dim=1, descending=True, stable=True)[1]
    rank = torch.empty_like(order).scatter_(1, order, j.expand_as(order).contiguous())
    return (j < n) & (~between | (rank < top))


def _plain_sparse(st):
    case = st["case"]
    S, Hk, D, B = case["S"], case["Hk"], case["D"], case["B"]
    W = case["top"] + case["first"] + case["last"]
    NB, lens = st["NB"], st["lens"].long()
    ready = torch.nonzero((st["slots"] >= 0) & (st["slots"] % B == B - 1))[:, 0]
    blk = st["slots"][ready] // B
    st["k_means"][blk] = _means(st["k_pool"][blk])
    tab = st["tables"].clamp(min=0).long()
    q = st["q"].float().unflatten(1, (Hk, -1))
    score = _scores(q[:, None], st["k_means"][tab].float()[:, :, :, None])
    n = (lens + B - 1) // B
    chosen = _choose(score, n, case["top"], case["first"], case["last"]).transpose(1, 2)     # [S][Hk][N]
    count = chosen.sum(-1)
    N = chosen.shape[-1]
    logical = torch.sort(torch.where(chosen, torch.arange(N, device="cuda"), N), -1)[0]
    logical = torch.nn.functional.pad(logical, (0, max(0, W - N)), value=N)[..., :W]
    head = torch.arange(Hk, device="cuda")[None, :, None]
    ids = tab[torch.arange(S, device="cuda")[:, None, None], logical.clamp(max=N - 1)]
    sel = torch.where(logical < N, ids * Hk + head, -1)
    sel_lens = torch.where(count > 0, (count - 1) * B + (lens - (n - 1) * B)[:, None], 0)
    live = torch.arange(W * B, device="cuda") < sel_lens[..., None]
    pick = lambda p: p.flatten(0, 1)[sel.clamp(min=0)].float().flatten(2, 3).masked_fill_(~live[..., None], 0)  # noqa: E731
    out = _attend(q, pick(st["k_pool"]), pick(st["v_pool"]), live, st["scale"])
    return {"out": out.flatten(1, 2).to(st["q"].dtype), "sel_tables": sel.int(), "sel_lens": sel_lens.int(),
            "k_means": st["k_means"]}


def run(st):
    if own:
        return _own(st)
    return {"tables": _plain_tables, "rope": _plain_rope, "store": _plain_store, "q4": _plain_q4,
            "sparse": _plain_sparse}[st["case"]["kind"]](st)


# -------------------------------------------------------------------------------------- work, exact
def work(case):
    kind = case["kind"]
    if kind == "tables":
        new = _new_tokens(case)
        blocks = case["S"] * case["done"] * (case["lo"] + case["hi"]) / 2 / case["B"] + new / case["B"]
        # slots and positions written; released entries read and pushed, new ones popped and written; per request
        # the table entry of its last block, its length in and out twice, its token count and flag
        return {"bytes": 12 * new + 8 * blocks + 30 * case["S"], "flops": 0}
    es = ES[case["dt"]]
    if kind == "rope":
        T, Hq, Hk, D = (case[k] for k in ("T", "Hq", "Hk", "D"))
        return {"bytes": T * (2 * (Hq + 2 * Hk) * D * es + 12), "flops": 3 * T * (Hq + Hk) * case["rd"]}
    Hk, D, B = case["Hk"], case["D"], case["B"]
    if kind == "store":
        rows = 2 * case["T"] * Hk
        row4 = D // 2 + D // GROUP * 4
        return {"bytes": rows * (2 * D * es + 2 * row4) + 16 * case["T"], "flops": 8 * rows * D}
    S, Hq = case["S"], case["Hq"]
    tokens = S * (case["lo"] + case["hi"]) / 2
    io = 2 * S * Hq * D * es + 4 * S
    if kind == "q4":
        return {"bytes": tokens * Hk * 2 * (D // 2 + D // GROUP * 4) + io + 4 * tokens / B, "flops": 4 * tokens * Hq * D}
    mean = (case["lo"] + case["hi"]) / 2
    read = S * min(mean, (case["top"] + case["first"] + case["last"]) * B)
    return {"bytes": tokens / B * Hk * D * es + read * Hk * 2 * D * es + io + 4 * tokens / B,
            "flops": 2 * tokens / B * Hq * D + 4 * read * Hq * D}


def _exact_attend(q, k, v, scale):
    """q [Hk][G][D], k and v [Hk][N][D], in 64 bits."""
    z = torch.einsum("hgd,hnd->hgn", q, k) * scale
    return torch.einsum("hgn,hnd->hgd", torch.softmax(z, -1), v)


def exact(case, seed):
    kind = case["kind"]
    if kind == "tables":
        return None
    st = prepare(case, seed)
    B, D, Hk = case["B"], case["D"], case["Hk"]
    NG = D // GROUP
    f64 = torch.float64
    if kind == "rope":
        w, amp = _frequencies(case)
        angle = st["pos"].to(f64)[:, None] * w[None, :]
        z = torch.polar(torch.full_like(angle, amp), angle)[:, None]
        rd = case["rd"]

        def turn(x):
            y = x.to(f64).clone()
            pairs = (slice(0, rd // 2), slice(rd // 2, rd)) if case["layout"] == "half" else (slice(0, rd, 2), slice(1, rd, 2))
            r = torch.complex(y[..., pairs[0]], y[..., pairs[1]]) * z
            y[..., pairs[0]], y[..., pairs[1]] = r.real, r.imag
            return y

        pools = []
        for rows in (turn(st["k"]), st["v"].to(f64)):
            pool = torch.zeros(st["k_pool"].shape, dtype=f64, device="cuda").transpose(1, 2).reshape(-1, Hk, D)
            pool[st["slots"][st["slots"] >= 0]] = rows[st["slots"] >= 0]
            pools.append(pool.view(-1, B, Hk, D).transpose(1, 2).contiguous())
        return {"q": turn(st["q"]), "k_pool": pools[0], "v_pool": pools[1]}
    if kind == "store":
        out = {}
        for name in ("k", "v"):
            x = st[name].to(f64).reshape(-1, GROUP)
            lo = x.min(1, keepdim=True)[0].half().to(f64)
            s = ((x.max(1, keepdim=True)[0] - x.min(1, keepdim=True)[0]).float() / 15).half().to(f64)
            # the code is decided in 32 bits, by definition
            c = torch.clamp(torch.round((x.float() - lo.float()) / s.float()), 0, 15).to(f64)
            out[name] = (torch.where(s > 0, c, 0.0) * s + lo).reshape(st[name].shape)
        return out
    lens = st["lens"].tolist()
    out = torch.zeros(case["S"], case["Hq"], D, dtype=f64, device="cuda")
    if kind == "q4":
        d = torch.arange(D, device="cuda")
        kn = ((d % 32 // 8) * NG + d // 32) * 8 + d % 8            # nibble of element d in a K row, in a V row
        vn = ((d % 32 // 4) * NG + d // 32) * 4 + d % 4
        for s, L in enumerate(lens):
            if L == 0:
                continue
            blk = st["tables"][s, : -(-L // B)].long()
            both = []
            for codes, params, nib in ((st["k_codes"], st["k_params"], kn), (st["v_codes"], st["v_params"].transpose(2, 3), vn)):
                row = codes[blk].transpose(0, 1).reshape(Hk, -1, D // 2)[:, :L]
                par = params[blk].transpose(0, 1).reshape(Hk, -1, 2 * NG)[:, :L].to(f64)
                c = (row[..., nib // 2] >> (4 * (nib % 2)).to(torch.uint8)) & 15
                both.append(c.to(f64) * par[..., d // 32] + par[..., NG + d // 32])
            out[s] = _exact_attend(st["q"][s].to(f64).view(Hk, -1, D), *both, st["scale"]).reshape(-1, D)
        return {"out": out}
    # sparse: which blocks are read is decided in 32 bits and a fixed order, by definition; the rest in 64
    means = st["k_means"]
    for slot in st["slots"].tolist():
        if slot >= 0 and slot % B == B - 1:
            rows = st["k_pool"][slot // B].cpu().numpy() if case["dt"] == "f32" else st["k_pool"][slot // B].float().cpu().numpy()
            total = rows[:, 0].astype(np.float32)
            for t in range(1, B):
                total = total + rows[:, t]
            means[slot // B] = torch.from_numpy(total / np.float32(B)).to(means.dtype).cuda()
    for s, L in enumerate(lens):
        if L == 0:
            continue
        n = -(-L // B)
        blk = st["tables"][s, :n].long()
        q = st["q"][s].view(Hk, -1, D)
        prod = q.float()[None] * means[blk].float()[:, :, None]                 # [n][Hk][G][D]
        lane = prod[..., 0::8]
        for e in range(1, 8):
            lane = lane + prod[..., e::8]
        while lane.shape[-1] > 1:
            lane = lane[..., 0::2] + lane[..., 1::2]
        score = lane[..., 0].max(-1)[0].T                                       # [Hk][n]
        for h in range(Hk):
            mid = torch.arange(case["first"], max(case["first"], n - case["last"]), device="cuda")
            best = mid[torch.sort(score[h, mid], descending=True, stable=True)[1][: case["top"]]]
            ends = [j for j in range(n) if j < case["first"] or j >= n - case["last"]]
            pick = torch.cat([best, torch.tensor(ends, device="cuda")]).sort()[0]
            tail = L - (n - 1) * B
            k, v = (p[blk[pick], h].reshape(-1, D).to(f64)[: (len(pick) - 1) * B + tail] for p in (st["k_pool"], st["v_pool"]))
            out[s].view(Hk, -1, D)[h] = _exact_attend(q[h: h + 1].to(f64), k[None], v[None], st["scale"])[0]
    return {"out": out, "sel_tables": None, "sel_lens": None, "k_means": None}
