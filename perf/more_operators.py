"""Operators around a decode step that verifies drafted tokens, as cases to measure: plain forms and the library's calls.

Four groups, in the order in which a serving loop calls them:

  plan     masks and positions of the drafted tokens of each request, from their parents (`tree_plan`)
  axes     rotary positions of several axes for q and k, k and v written to their slots (`rope_axes_append`)
  attend   attention of all drafted tokens over the cache, under their tree's mask (`decode_attention_tree`)
  verify   drafted rows in the cache, the branch that the model's answers confirm, its rows moved together,
           blocks behind it given back (`append`, `tree_accept`, `tree_commit`, `tables_truncate`)

A request's drafted tokens are a tree: each has a parent before it, or -1 for the token that is already decided. They
lie at the end of its context in the cache, n of its L tokens. Layouts are those of the library: pools
[blocks][kv heads][block size][head size], tables [requests][blocks] int32, lengths [requests] int32, slots int64, the
requests' drafted tokens one after another with offsets [requests + 1] int32, masks [tokens][words] int64 (bit j: the
request's j-th drafted token is seen).
"""
import functools
import math

import numpy as np
import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ES = {"f32": 4, "f16": 2, "bf16": 2}


# ------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the benchmark's batch, 16 drafted tokens a request
        {"name": "plan_batch", "kind": "plan", "S": 64, "n_lo": 16, "n_hi": 16, "words": 1, "axes": 1, "wide": 0.5,
         "far": 4096},
        # the widest trees for a large batch, positions on three axes
        {"name": "plan_wide", "kind": "plan", "S": 997, "n_lo": 1, "n_hi": 256, "words": 4, "axes": 3, "wide": 0.3,
         "far": 32768},
        # drafted tokens of the benchmark's batch, 32 q and 8 kv heads, three axes whose pairs lie one after another
        {"name": "axes_step", "kind": "axes", "T": 1024, "Hq": 32, "Hk": 8, "D": 128, "rd": 128, "B": 16, "dt": "bf16",
         "layout": "half", "sections": "16,24,24", "order": "sections", "own_base": False, "far": 32768, "packed": True},
        # prompts with pictures over as many kv heads as q heads, pairs dealt out to the axes in turn, some tokens
        # of a padded batch without a slot
        {"name": "axes_prompts", "kind": "axes", "T": 8191, "Hq": 40, "Hk": 40, "D": 128, "rd": 128, "B": 16,
         "dt": "f16", "layout": "half", "sections": "24,20,20", "order": "cycled", "own_base": False, "far": 4096,
         "packed": False},
        # patches of frames: each axis has frequencies of its own, neighbouring pairs
        {"name": "axes_frames", "kind": "axes", "T": 4097, "Hq": 16, "Hk": 16, "D": 64, "rd": 64, "B": 32, "dt": "bf16",
         "layout": "interleaved", "sections": "8,12,12", "order": "sections", "own_base": True, "far": 100,
         "packed": True},
        # one interactive request: latency
        {"name": "attend_one", "kind": "attend", "S": 1, "Hq": 32, "Hk": 8, "D": 128, "B": 16, "dt": "bf16",
         "lo": 1000, "hi": 1000, "n_lo": 16, "n_hi": 16, "words": 1, "wide": 0.5},
        # the benchmark's batch, 16 drafted tokens a request
        {"name": "attend_batch", "kind": "attend", "S": 64, "Hq": 32, "Hk": 8, "D": 128, "B": 16, "dt": "bf16",
         "lo": 512, "hi": 4096, "n_lo": 16, "n_hi": 16, "words": 1, "wide": 0.5},
        # one q head for each kv head, chains of up to 5
        {"name": "attend_chains", "kind": "attend", "S": 128, "Hq": 40, "Hk": 40, "D": 128, "B": 16, "dt": "f16",
         "lo": 128, "hi": 2048, "n_lo": 1, "n_hi": 5, "words": 1, "wide": 0.0},
        # fewer requests with trees of up to 64
        {"name": "attend_trees", "kind": "attend", "S": 32, "Hq": 32, "Hk": 8, "D": 128, "B": 16, "dt": "f16",
         "lo": 512, "hi": 4096, "n_lo": 33, "n_hi": 64, "words": 1, "wide": 0.5},
        # eight long agent contexts, 8 q heads to a kv head
        {"name": "attend_long", "kind": "attend", "S": 8, "Hq": 64, "Hk": 8, "D": 128, "B": 32, "dt": "bf16",
         "lo": 32768, "hi": 131072, "n_lo": 16, "n_hi": 26, "words": 1, "wide": 0.5},
        # the benchmark's batch after its answers are in
        {"name": "verify_batch", "kind": "verify", "S": 64, "Hk": 8, "D": 128, "B": 16, "dt": "bf16", "lo": 100,
         "hi": 1000, "n_lo": 16, "n_hi": 16, "wide": 0.5, "right": 0.7},
        # trees of up to 64 for many requests of a cache with as many kv heads as q heads
        {"name": "verify_wide", "kind": "verify", "S": 199, "Hk": 40, "D": 128, "B": 16, "dt": "f16", "lo": 0,
         "hi": 200, "n_lo": 0, "n_hi": 64, "wide": 0.3, "right": 0.8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["plan", "axes", "attend", "attend", "verify"])
    wide = rng.choice([0.0, 0.3, 0.5, 1.0])
    if kind == "plan":
        n = _log(rng, 1, 256)
        return {"kind": kind, "S": _log(rng, 1, 997), "n_lo": rng.randint(0, n), "n_hi": n, "words": rng.randint(-(-n // 64), 4),
                "axes": rng.randint(1, 4), "wide": wide, "far": _log(rng, 10, 1 << 20)}
    B, D = rng.choice([8, 16, 32]), rng.choice([64, 128])
    if kind == "axes":
        Hk = rng.choice([1, 2, 5, 8, 40])
        rd = rng.choice([D, D // 2, 20])
        axes = rng.randint(1, 4)
        cuts = sorted(rng.sample(range(2, rd // 2 - 1), axes - 1)) if axes > 1 else []
        sections = [b - a for a, b in zip([0] + cuts, cuts + [rd // 2])]
        return {"kind": kind, "T": _log(rng, 1, 8000), "Hq": Hk * rng.choice([1, 4, 7]) if Hk < 40 else 40, "Hk": Hk,
                "D": D, "rd": rd, "B": B, "dt": rng.choice(["f16", "bf16", "f32"]),
                "layout": rng.choice(["half", "interleaved"]), "sections": ",".join(map(str, sections)),
                "order": rng.choice(["sections", "cycled"]), "own_base": rng.choice([False, True]),
                "far": _log(rng, 10, 1 << 20), "packed": rng.choice([False, True])}
    if kind == "verify":
        n = _log(rng, 1, 64)
        return {"kind": kind, "S": _log(rng, 1, 199), "Hk": rng.choice([1, 2, 5, 8, 40]), "D": D, "B": B,
                "dt": rng.choice(["f16", "bf16", "f32"]), "lo": 0, "hi": _log(rng, 1, 200), "n_lo": rng.randint(0, n), "n_hi": n,
                "wide": wide, "right": rng.choice([0.0, 0.5, 0.8, 1.0])}
    Hk = rng.choice([1, 2, 3, 8])
    G = rng.choice([1, 3, 4, 8, 12] if Hk < 8 else [1, 4, 5, 8])
    n = _log(rng, 1, 256 if rng.random() < 0.3 else 64)
    hi = _log(rng, 1, 40000)
    # (at most the listed cases' scores and rows)
    S = max(1, min(_log(rng, 1, 200), 250000 // (hi + n), 200_000_000 // (n * G * Hk * (hi + n))))
    return {"kind": kind, "S": S, "Hq": Hk * G, "Hk": Hk, "D": D, "B": B,
            "dt": "f32" if rng.random() < 0.15 else rng.choice(["f16", "bf16"]), "lo": hi // rng.choice([2, 4, 20]), "hi": hi,
            "n_lo": rng.randint(0, n), "n_hi": n, "words": -(-n // 64), "wide": wide}


# ------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def _randn(shape, dt, g, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(DT[dt])


def _trees(case, rng):
    """Drafted tokens of each request, spread over the case's range, and all their parents: the one before, or with
    chance `wide` any of those before."""
    n = rng.permutation(np.linspace(case["n_hi"], case["n_lo"], case["S"]).round().astype(np.int64))
    offs = np.concatenate([[0], np.cumsum(n)])
    i = np.arange(offs[-1]) - np.repeat(offs[:-1], n)
    any_ = np.minimum((rng.random(len(i)) * i).astype(np.int64), i - 1)
    parents = np.where(rng.random(len(i)) < case["wide"], any_, i - 1)
    return n, offs.astype(np.int32), parents.astype(np.int32)


def _mask_words(n, offs, parents, words):
    """Each token's ancestors and itself, as bits."""
    m = np.zeros((len(parents), words), np.uint64)
    local = np.arange(len(parents)) - np.repeat(offs[:-1], n)
    for k in range(int(n.max(initial=0))):                  # all requests' k-th tokens at once
        at = np.flatnonzero(local == k)
        p = parents[at]
        m[at] = np.where((p >= 0)[:, None], m[at - k + np.maximum(p, 0)], 0)
        m[at, k // 64] |= np.uint64(1 << (k % 64))
    return m.view(np.int64)


def _tables(case, lens, rng):
    """Tables of randomly scattered blocks, the number of blocks of a pool with room for every request at its longest,
    and the blocks to spare."""
    B = case["B"]
    n = -(-lens // B)
    M = -(-(case["hi"] + case["n_hi"]) // B) + 1
    NB = case["S"] * (M - 1) + 3
    perm = rng.permutation(NB)
    tab = np.full((len(lens), M), -1, np.int32)
    tab[np.arange(M)[None, :] < n[:, None]] = perm[: int(n.sum())]
    return tab, NB, perm[int(n.sum()):]


def prepare(case, seed):
    rng = np.random.default_rng([int(seed), 11])
    g = _gen(seed)
    st = {"case": case}
    kind = case["kind"]
    if kind == "axes":
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
        axes = len(case["sections"].split(","))
        pos = rng.integers(0, case["far"], size=(axes, T)).astype(np.int32)
        text = rng.random(T) < 0.5                          # text has one position on all axes
        pos[:, text] = pos[:1, text]
        st |= {"q": q, "k": k, "v": v, "slots": _dev(slots), "pos": _dev(pos),
               "k_pool": torch.zeros(NB, Hk, B, D, dtype=DT[case["dt"]], device="cuda"),
               "v_pool": torch.zeros(NB, Hk, B, D, dtype=DT[case["dt"]], device="cuda"),
               "q_out": torch.empty(T, Hq, D, dtype=DT[case["dt"]], device="cuda")}
        return st
    n, offs, parents = _trees(case, rng)
    T = len(parents)
    st |= {"offs": _dev(offs), "parents": _dev(parents), "max_tree": max(1, case["n_hi"])}
    if kind == "plan":
        lens = n + rng.integers(0, case["far"], size=case["S"])
        st |= {"lens": _dev(lens.astype(np.int32)),
               "deltas": _dev(rng.integers(-int(case["far"]) // 2, int(case["far"]) // 2 + 1, size=case["S"]).astype(np.int32))}
        return st
    lens = n + rng.integers(case["lo"], case["hi"] + 1, size=case["S"])
    Hk, D, B = case["Hk"], case["D"], case["B"]
    tab, NB, spare = _tables(case, lens, rng)
    st |= {"tables": _dev(tab), "lens": _dev(lens.astype(np.int32))}
    if kind == "attend":
        st |= {"q": _randn((T, case["Hq"], D), case["dt"], g), "scale": 1 / math.sqrt(D),
               "masks": _dev(_mask_words(n, offs, parents, case["words"]))}
        pools = [_randn((NB, Hk, B, D), case["dt"], g) for _ in range(2)]
        # positions that no context holds: what a pool has there is not to be used
        used = np.zeros(NB, np.int64)
        valid = np.clip(lens[:, None] - np.arange(tab.shape[1])[None, :] * B, 0, B)
        used[tab[tab >= 0]] = valid[tab >= 0]
        dead = _dev(np.arange(B)[None, :] >= used[:, None])
        for p in pools:
            p.masked_fill_(dead[:, None, :, None], math.nan)
        return st | {"k_pool": pools[0], "v_pool": pools[1]}
    # verify: the model answers with the token of one child, or with another one
    i = np.arange(T) - np.repeat(offs[:-1], n)
    row = np.repeat(offs[:-1], n)
    tokens = rng.permutation(4 * T + 1)[:T].astype(np.int32)          # (all different)
    targets = (tokens.max(initial=0) + 1 + rng.integers(0, 1000, size=T)).astype(np.int32)
    says = (rng.random(T) < case["right"]) & (parents >= 0)
    targets[(row + parents)[says]] = tokens[says]
    pos = np.repeat(lens - n, n) + i
    slots = tab[np.repeat(np.arange(case["S"]), n), pos // B].astype(np.int64) * B + pos % B
    free = np.full(NB, -1, np.int32)
    free[: len(spare)] = spare
    return st | {"tokens": _dev(tokens), "targets": _dev(targets), "slots": _dev(slots), "free": _dev(free),
                 "num_free": torch.tensor([len(spare)], dtype=torch.int32, device="cuda"),
                 "k": _randn((T, Hk, D), case["dt"], g), "v": _randn((T, Hk, D), case["dt"], g),
                 "k_pool": _randn((NB, Hk, B, D), case["dt"], g), "v_pool": _randn((NB, Hk, B, D), case["dt"], g)}


# ------------------------------------------------------------------------------- the library's calls
def _axes_args(case):
    return {"sections": tuple(int(x) for x in case["sections"].split(",")), "order": case["order"],
            "frequencies": "own" if case["own_base"] else "shared", "base": 10000.0, "layout": case["layout"]}


def _calls(st):
    """The library's calls of one pass, prepared as a serving loop prepares them, and their outputs."""
    from paged_kv_cache_47_gb300 import binding as b

    case = st["case"]
    kind = case["kind"]
    i32 = functools.partial(torch.empty, dtype=torch.int32, device="cuda")
    if kind == "plan":
        T = st["parents"].shape[0]
        masks = torch.empty(T, case["words"], dtype=torch.int64, device="cuda")
        pos = i32(case["axes"], T)
        call = b.prepared_tree_plan(st["parents"], st["offs"], st["lens"], masks, pos, position_deltas=st["deltas"])
        return (call,), {"masks": masks, "positions": pos}
    if kind == "axes":
        plan = b.RopeAxesPlan(**_axes_args(case))
        call = b.prepared_rope_axes_append(st["q"], st["k"], st["v"], st["pos"], st["slots"], plan, st["k_pool"],
                                           st["v_pool"], q_out=st["q_out"])
        return (call,), {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}
    if kind == "attend":
        out = torch.empty_like(st["q"])
        ws = b.alloc_tree_workspace(st["k_pool"], case["Hq"], st["max_tree"])
        call = b.prepared_decode_attention_tree(st["q"], st["k_pool"], st["v_pool"], st["tables"], st["lens"],
                                                st["offs"], st["masks"], st["scale"], max_tree=st["max_tree"], out=out,
                                                workspace=ws)
        return (call,), {"out": out}
    S, T = case["S"], st["parents"].shape[0]
    path, count, last, lens, left = i32(T), i32(S), i32(S), i32(S), i32(1)
    calls = (b.PreparedAppend(st["k"], st["v"], st["slots"], st["k_pool"], st["v_pool"]),
             b.prepared_tree_accept(st["parents"], st["tokens"], st["targets"], st["offs"], st["lens"], path, count, last,
                                    lens, max_tree=st["max_tree"]),
             b.prepared_tree_commit(path, count, st["offs"], st["lens"], st["tables"], st["k_pool"], st["v_pool"],
                                    max_tree=st["max_tree"]),
             b.prepared_tables_truncate(st["tables"], st["lens"], lens, st["free"], st["num_free"], case["B"],
                                        workspace=b.alloc_tables_workspace(), context_lens_out=i32(S),
                                        num_free_out=left))
    return calls, {"path": path, "counts": count, "next": last, "lens": lens, "free": st["free"], "num_free": left,
                   "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _own(st):
    if "calls" not in st:       # what a program makes once and keeps: plans, workspaces, outputs, arguments
        st["calls"] = _calls(st)
    calls, outputs = st["calls"]
    for call in calls:
        call(None)
    return outputs


# -------------------------------------------------------------------------------------- plain forms
def _requests(st):
    """Request of each token, its place among the request's tokens, and the number of tokens of each request."""
    offs = st["offs"].long()
    n = offs[1:] - offs[:-1]
    i = torch.arange(st["parents"].shape[0], device="cuda")
    s = torch.searchsorted(offs[1:], i, right=True)
    return s, i - offs[s], n


def _ancestors(st, s, local):
    """[tokens][max_tree] truth values: the request's j-th token is this one or above it. One squaring of the parent
    relation doubles the steps that it spans."""
    N = st["max_tree"]
    S = st["offs"].shape[0] - 1
    up = torch.zeros(S, N, N, device="cuda")
    up[s, local, local] = 1
    has = st["parents"] >= 0
    up[s[has], local[has], st["parents"][has].long()] = 1
    up = functools.reduce(lambda a, _: torch.matmul(a, a).clamp(max=1), range(max(1, N - 1).bit_length()), up)
    return up[s, local] > 0


def _plain_plan(st):
    case = st["case"]
    s, local, n = _requests(st)
    above = _ancestors(st, s, local)
    depth = above.sum(1) - 1
    pos = (st["lens"].long() - n + st["deltas"])[s] + depth
    bits = torch.nn.functional.pad(above, (0, 64 * case["words"] - above.shape[1])).unflatten(1, (-1, 64)).long()
    return {"masks": (bits << torch.arange(64, device="cuda")).sum(-1),
            "positions": pos.int().expand(case["axes"], -1).contiguous()}


def _pairs(case):
    """Axis of each rotated pair, and its radians a position in 64 bits."""
    a = _axes_args(case)
    sections, A = a["sections"], len(a["sections"])
    if a["order"] == "sections":
        axis = [k for k, n in enumerate(sections) for _ in range(n)]
    else:                                        # the next axis that has pairs left
        deal = sorted((j, k) for k, n in enumerate(sections) for j in range(n))
        axis = [k for _, k in deal]
    nth = [axis[:i].count(k) for i, k in enumerate(axis)]
    e = [j / sections[k] if case["own_base"] else i / len(axis) for i, (j, k) in enumerate(zip(nth, axis))]
    return axis, a["base"] ** -torch.tensor(e, dtype=torch.float64, device="cuda")


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


def _plain_axes(st):
    case = st["case"]
    axis, w = _pairs(case)
    angle = (st["pos"][axis].T.double() * w)[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    st["q_out"].copy_(_rotate(st["q"], cos, sin, case))
    B = case["B"]
    keep = torch.nonzero(st["slots"] >= 0)[:, 0]
    slot = st["slots"][keep]
    st["k_pool"][slot // B, :, slot % B] = _rotate(st["k"], cos, sin, case)[keep]
    st["v_pool"][slot // B, :, slot % B] = st["v"][keep]
    return {"q": st["q_out"], "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def _plain_attend(st):
    case = st["case"]
    S, Hk, D, N = case["S"], case["Hk"], case["D"], st["max_tree"]
    s, local, n = _requests(st)
    tab, lens = st["tables"].clamp(min=0).long(), st["lens"].long()
    t = torch.arange(tab.shape[1] * case["B"], device="cuda")
    live = t < lens[:, None]                                                     # [S][t]
    k, v = (p[tab].transpose(1, 2).flatten(2, 3).float().masked_fill_(~live[:, None, :, None], 0)
            for p in (st["k_pool"], st["v_pool"]))
    q = torch.zeros(S, N, case["Hq"], D, device="cuda")
    q[s, local] = st["q"].float()
    q = q.unflatten(2, (Hk, -1)).transpose(1, 2)                                 # [S][Hk][N][G][D]
    # which positions each token sees: all before the drafted ones, and those of its mask
    bits = torch.zeros(S, N, 64 * case["words"], dtype=torch.bool, device="cuda")
    bits[s, local] = ((st["masks"][:, :, None] >> torch.arange(64, device="cuda")) & 1).bool().flatten(1)
    j = t - (lens - n)[:, None]
    sees = bits.gather(2, j.clamp(0, bits.shape[2] - 1)[:, None].expand(-1, N, -1))
    sees = ((j < 0)[:, None] | sees) & live[:, None]                             # [S][N][t]
    z = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).unflatten(2, (N, -1)).mul_(st["scale"])
    z = z.masked_fill_(~sees[:, None, :, None], -math.inf)
    p = z.sub_(z.amax(-1, keepdim=True).clamp(min=-3e38)).exp_().flatten(2, 3)
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-37)
    o = o.unflatten(2, (N, -1)).transpose(1, 2).flatten(2, 3)                     # [S][N][Hq][D]
    return {"out": o[s, local].to(st["q"].dtype)}


def _plain_verify(st):
    case = st["case"]
    S, B, N = case["S"], case["B"], st["max_tree"]
    s, local, n = _requests(st)
    T = s.shape[0]
    offs, lens, tab = st["offs"].long(), st["lens"].long(), st["tables"].long()
    st["k_pool"][st["slots"] // B, :, st["slots"] % B] = st["k"]
    st["v_pool"][st["slots"] // B, :, st["slots"] % B] = st["v"]
    # a token holds where it and all above it are what their parents' answers say
    above = _ancestors(st, s, local)
    par = st["parents"].long()
    right = (par < 0) | (st["tokens"] == st["targets"][offs[s] + par.clamp(min=0)])
    rights = torch.zeros(S, N, dtype=torch.bool, device="cuda")
    rights[s, local] = right
    holds = ~(above & ~rights[s]).any(1)
    depth = above.sum(1)
    # the deepest one, of equals the first
    key = torch.full((S, N), -1, dtype=torch.int64, device="cuda")
    key[s, local] = torch.where(holds, depth * N - local, -1)
    best, last = key.max(1)
    some = best >= 0
    count = torch.where(some, depth[(offs[:-1] + last).clamp(max=max(T - 1, 0))], 0)
    chosen = above[(offs[:-1] + last).clamp(max=max(T - 1, 0))] & some[:, None]           # [S][N]
    rank = chosen.cumsum(1) - 1
    on = chosen[s, local]
    path = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    path[offs[s[on]] + rank[s[on], local[on]]] = local[on]
    answer = torch.where(some, st["targets"][(offs[:-1] + last).clamp(max=max(T - 1, 0))].long(), -1)
    start = lens - n
    kept = start + count
    # rows of the path, moved behind the context
    at, to = start[s[on]] + local[on], start[s[on]] + rank[s[on], local[on]]
    src_b, dst_b = tab[s[on], at // B], tab[s[on], to // B]
    for pool in (st["k_pool"], st["v_pool"]):
        pool[dst_b, :, to % B] = pool[src_b, :, at % B]
    # blocks behind the new lengths, pushed in table order
    nf = st["num_free"].long()
    first, end = (kept + B - 1) // B, (lens + B - 1) // B
    back = end - first
    j = torch.arange(tab.shape[1], device="cuda")
    put = (j >= first[:, None]) & (j < end[:, None])
    place = nf + (torch.cumsum(back, 0) - back)[:, None] + j - first[:, None]
    st["free"][place[put]] = tab[put].int()
    return {"path": path.int(), "counts": count.int(), "next": answer.int(), "lens": kept.int(), "free": st["free"],
            "num_free": (nf + back.sum()).int(), "k_pool": st["k_pool"], "v_pool": st["v_pool"]}


def run(st):
    if own:
        return _own(st)
    return {"plan": _plain_plan, "axes": _plain_axes, "attend": _plain_attend, "verify": _plain_verify}[st["case"]["kind"]](st)


# -------------------------------------------------------------------------------------- work, exact
def work(case):
    kind = case["kind"]
    if kind == "axes":
        T, Hq, Hk, D, es = case["T"], case["Hq"], case["Hk"], case["D"], ES[case["dt"]]
        A = len(case["sections"].split(","))
        return {"bytes": T * (2 * (Hq + 2 * Hk) * D * es + 4 * A + 8), "flops": 3 * T * (Hq + Hk) * case["rd"]}
    S = case["S"]
    n = S * (case["n_lo"] + case["n_hi"]) / 2
    if kind == "plan":
        return {"bytes": n * (4 + 8 * case["words"] + 4 * case["axes"]) + 12 * S, "flops": 0}
    Hk, D, B, es = case["Hk"], case["D"], case["B"], ES[case["dt"]]
    if kind == "verify":
        # rows appended (read and written) and about a third of them moved; parents, tokens, answers, slots and path
        rows = n * (1 + case["right"] / 3)
        return {"bytes": rows * 4 * Hk * D * es + 24 * n + 32 * S, "flops": 0}
    tokens = S * (case["lo"] + case["hi"]) / 2 + n
    io = 2 * n * case["Hq"] * D * es + 8 * n * case["words"] + 8 * S
    return {"bytes": tokens * Hk * 2 * D * es + io + 4 * tokens / B, "flops": 4 * tokens * n / S * case["Hq"] * D}


def exact(case, seed):
    kind = case["kind"]
    if kind in ("plan", "verify"):              # whole numbers, and rows as they are
        return None
    st = prepare(case, seed)
    B, D, Hk = case["B"], case["D"], case["Hk"]
    f64 = torch.float64
    if kind == "axes":
        axis, w = _pairs(case)
        rd = case["rd"]
        angle = torch.stack([st["pos"][a].to(f64) * w[i] for i, a in enumerate(axis)], 1)
        z = torch.polar(torch.ones_like(angle), angle)[:, None]

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
    offs, parents = st["offs"].tolist(), st["parents"].tolist()
    out = torch.zeros(st["q"].shape, dtype=f64, device="cuda")
    for s, L in enumerate(st["lens"].tolist()):
        o0, n = offs[s], offs[s + 1] - offs[s]
        if n == 0:
            continue
        blk = st["tables"][s, : -(-L // B)].long()
        k, v = (p[blk].transpose(0, 1).reshape(Hk, -1, D)[:, :L].to(f64) for p in (st["k_pool"], st["v_pool"]))
        seen = np.zeros((n, L), bool)
        seen[:, : L - n] = True
        for i in range(n):
            j = i
            while j >= 0:                       # itself, its parent, and so on
                seen[i, L - n + j] = True
                j = parents[o0 + j]
        q = st["q"][o0: o0 + n].to(f64).view(n, Hk, -1, D)
        z = torch.einsum("nhgd,htd->nhgt", q, k) * st["scale"]
        z[~_dev(seen)[:, None, None].expand_as(z)] = -math.inf
        out[o0: o0 + n] = torch.einsum("nhgt,htd->nhgd", torch.softmax(z, -1), v).flatten(1, 2)
    return {"out": out}
